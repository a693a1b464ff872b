// What follows the attention of mla_tree_decode: the merge of each (row, head)'s
// parts, weighed by their log-sum-exps, and the output projection
//   out[n,h] = o_lat[n,h] W_uv[h]        ([512] . [512, 128]).
#include "async_copy.cuh"
#include "pair_math.cuh"
#include "tree_parts.cuh"

namespace mla {
namespace {

// The parts of (row n, head h): `count` of them, part i in slot(i), row r of it.
struct RowParts {
  int count, r, share, ubase, ibase, m, j, full, per, tail;

  __device__ __forceinline__ int slot(int i) const {
    if (m == 1) return ubase / share + i + ibase;
    if (i < full * per) {
      const int s = i / per;
      return ubase / share + s * m + j + i % per + ibase + s * m + j;
    }
    const int start = ubase + full * share * m + j * tail;
    return start / share + (i - full * per) + ibase + full * m + j;
  }
};
__device__ __forceinline__ RowParts row_parts(const TreeArgs& a, int n, int h) {
  RowParts p{};
  int lo = 0, hi = a.batch;   // the last sequence that begins at or before row n
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.query_start_loc + mid) <= n) lo = mid; else hi = mid;
  }
  const int q0 = __ldg(a.query_start_loc + lo);
  if (q0 < 0 || n < q0 || n >= __ldg(a.query_start_loc + lo + 1)) return p;
  const int4 pl = a.plan[lo];
  if (pl.w <= 0) return p;
  p.share = reinterpret_cast<const WsHeader*>(a.ws)->share;
  p.ubase = pl.x;
  p.ibase = pl.y;
  p.m = pl.w;
  const int rr = (n - q0) * a.num_heads + h;
  p.j = rr / kTreeBlockRows;
  p.r = rr % kTreeBlockRows;
  const int tiles = pl.z;
  if (p.m == 1) {
    p.count = (p.ubase + tiles - 1) / p.share - p.ubase / p.share + 1;
  } else {
    p.full = tiles / p.share;
    p.per = p.ubase % p.share ? 2 : 1;
    p.tail = tiles % p.share;
    p.count = p.full * p.per;
    if (p.tail) {
      const int start = p.ubase + p.full * p.share * p.m + p.j * p.tail;
      p.count += (start + p.tail - 1) / p.share - start / p.share + 1;
    }
  }
  return p;
}

// Of few (row, head)s, which may have many parts: a (row, head) to a CTA of 16 warps.
// A warp takes 128 columns of every fourth part; lane i has the slot and the weight of
// part i of 32. Rows with one part are in their place already.
__global__ void __launch_bounds__(512) tree_merge_few_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int kAhead = 8, kGroups = 4;
  __shared__ float4 sAcc[kGroups - 1][128];
  const int n = blockIdx.x / a.num_heads, h = blockIdx.x % a.num_heads, tid = threadIdx.x;
  const int group = tid >> 7, c = tid & 127, half = c >> 6, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  const RowParts rp = row_parts(a, n, h);
  if (rp.count == 1) return;
  auto part = [&](int i, int& slot) {
    slot = i < rp.count ? rp.slot(i) : 0;
    return i < rp.count ? a.lse[((int64_t)slot * 2 + half) * kTreeBlockRows + rp.r] : -INFINITY;
  };
  int slot;
  float lse = part(lane, slot), m = lse, den = 0.f;
#pragma unroll 1
  for (int s0 = 32; s0 < rp.count; s0 += 32) m = fmaxf(m, part(s0 + lane, slot));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = m == -INFINITY ? 0.f : m;     // (a row that sees nothing: weights of 0)
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int s0 = 0; s0 < rp.count; s0 += 32) {
    lse = part(s0 + lane, slot);
    const float w = fast_exp2(lse - base);
    den += w;
    const int live = min(32, rp.count - s0);
    float4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = group + u * kGroups, at = __shfl_sync(0xffffffffu, slot, i);
      if (i < live)
        v[u] = __ldcs(reinterpret_cast<const float4*>(a.opart + ((int64_t)at * kTreeBlockRows + rp.r) * kDc) + c);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = group + u * kGroups;
      const float x = __shfl_sync(0xffffffffu, w, i);
      if (i < live) {
        acc.x = fmaf(x, v[u].x, acc.x);
        acc.y = fmaf(x, v[u].y, acc.y);
        acc.z = fmaf(x, v[u].z, acc.z);
        acc.w = fmaf(x, v[u].w, acc.w);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  if (group > 0) sAcc[group - 1][c] = acc;
  __syncthreads();
  if (group > 0) return;
#pragma unroll
  for (int u = 0; u < kGroups - 1; ++u) {
    const float4 x = sAcc[u][c];
    acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  reinterpret_cast<float4*>(a.o_lat + ((size_t)n * a.num_heads + h) * kDc)[c] =
      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
}

// Of 512 (row, head)s or more: 16 to a CTA, whose parts 16 threads find; then a warp for
// each of two, as above but for all of its parts and columns. Bound by latency: a few
// dependent loads a row. With a warp or with eight rows to each step of its own, or
// more CTAs an SM and fewer parts ahead, a call of 64 x 4,096 tokens took 1 to 8 us
// longer (of 100); a CTA a row, as few rows have it, 7 us longer, and 31 us longer
// for 49,280 (row, head)s of short sequences.
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int kAhead = 4;
  __shared__ RowParts sParts[16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int first = blockIdx.x * 16, all = (int)(a.num_q * a.num_heads);
  pdl_wait();
  pdl_launch_dependents();
  bool work = false;
  if (tid < 16) {
    RowParts rp{};
    rp.count = 1;
    if (first + tid < all) rp = row_parts(a, (first + tid) / a.num_heads, (first + tid) % a.num_heads);
    sParts[tid] = rp;
    work = rp.count != 1;
  }
  if (!__syncthreads_or(work)) return;
#pragma unroll 1
  for (int at = warp; at < 16; at += 8) {
    const RowParts rp = sParts[at];
    if (rp.count == 1) continue;
    auto part = [&](int i, int& slot, float& l0, float& l1) {
      slot = 0;
      l0 = l1 = -INFINITY;
      if (i < rp.count) {
        slot = rp.slot(i);
        l0 = a.lse[(int64_t)slot * 2 * kTreeBlockRows + rp.r];
        l1 = a.lse[((int64_t)slot * 2 + 1) * kTreeBlockRows + rp.r];
      }
    };
    int slot;
    float l0, l1, m0 = -INFINITY, m1 = -INFINITY, d0 = 0.f, d1 = 0.f;
#pragma unroll 1
    for (int s0 = 0; s0 < rp.count; s0 += 32) {
      part(s0 + lane, slot, l0, l1);
      m0 = fmaxf(m0, l0);
      m1 = fmaxf(m1, l1);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
      m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
    }
    if (m0 == -INFINITY) m0 = 0.f;
    if (m1 == -INFINITY) m1 = 0.f;
    float4 acc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int s0 = 0; s0 < rp.count; s0 += 32) {
      if (rp.count > 32) part(s0 + lane, slot, l0, l1);
      const float w0 = fast_exp2(l0 - m0), w1 = fast_exp2(l1 - m1);
      d0 += w0;
      d1 += w1;
      const int live = min(32, rp.count - s0);
#pragma unroll 1
      for (int u0 = 0; u0 < live; u0 += kAhead) {
        float4 v[kAhead][4];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int at1 = __shfl_sync(0xffffffffu, slot, (u0 + u) & 31);
          const float4* src = reinterpret_cast<const float4*>(a.opart + ((int64_t)at1 * kTreeBlockRows + rp.r) * kDc) + lane;
          if (u0 + u < live) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[u][k] = __ldcs(src + 32 * k);
          }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const float x0 = __shfl_sync(0xffffffffu, w0, (u0 + u) & 31), x1 = __shfl_sync(0xffffffffu, w1, (u0 + u) & 31);
          if (u0 + u < live) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float x = k < 2 ? x0 : x1;
              acc[k].x = fmaf(x, v[u][k].x, acc[k].x);
              acc[k].y = fmaf(x, v[u][k].y, acc[k].y);
              acc[k].z = fmaf(x, v[u][k].z, acc[k].z);
              acc[k].w = fmaf(x, v[u][k].w, acc[k].w);
            }
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      d0 += __shfl_xor_sync(0xffffffffu, d0, o);
      d1 += __shfl_xor_sync(0xffffffffu, d1, o);
    }
    d0 = d0 == 0.f ? 0.f : 1.f / d0;
    d1 = d1 == 0.f ? 0.f : 1.f / d1;
    float4* dst = reinterpret_cast<float4*>(a.o_lat + (size_t)(first + at) * kDc) + lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float d = k < 2 ? d0 : d1;
      dst[32 * k] = make_float4(acc[k].x * d, acc[k].y * d, acc[k].z * d, acc[k].w * d);
    }
  }
}

// The projection of few rows: CTA = (8 rows, head h). W_uv[h] (128 KB) comes by
// cp.async while the attention ends; the latents are split to two bf16 terms each, so
// that the output is rounded once; then 8 warps, each a quarter of K and half of the
// columns (m16n8k16: rows 0 to 7 the first terms, 8 to 15 the second).
struct Pj {
  static constexpr int rows = 8;
  static constexpr int stride = kDc * 2 + 16;     // bytes of a row of terms, padded against bank conflicts
  static constexpr int w = 0;                     // two halves of 64 columns, 128-byte rows
  static constexpr int a = w + kDc * 256;
  static constexpr int red = a + 2 * rows * stride;  // [4][rows][128]
  static constexpr int bytes = red + 4 * rows * kDv * 4;
};
__global__ void __launch_bounds__(256) tree_proj_kernel(const __grid_constant__ TreeArgs a, const __nv_bfloat16* W_uv,
                                                        __nv_bfloat16* out) {
  extern __shared__ __align__(1024) uint8_t smem_pj[];
  float* sRed = reinterpret_cast<float*>(smem_pj + Pj::red);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, row0 = blockIdx.x * Pj::rows, H = a.num_heads;
  const __nv_bfloat16* src = W_uv + (size_t)h * kDc * kDv;
#pragma unroll 4
  for (int i = tid; i < kDc * 16; i += 256) {
    const int k = i >> 4, c = i & 15;
    cp_async16(smem_pj + Pj::w + (c >> 3) * (kDc * 128) + sw128(k, c & 7), src + (size_t)k * kDv + c * 8);
  }
  cp_async_commit();
  pdl_wait();
  pdl_launch_dependents();
  {
    const int n = row0 + warp;        // a warp a row
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = n < a.num_q ? reinterpret_cast<const float4*>(a.o_lat + ((size_t)n * H + h) * kDc)[lane + 32 * k]
                         : make_float4(0.f, 0.f, 0.f, 0.f);
    auto low = [](uint32_t t) { return __uint_as_float(t << 16); };
    auto high = [](uint32_t t) { return __uint_as_float(t & 0xffff0000u); };
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t t0 = pack_bf16(v[k].x, v[k].y), t1 = pack_bf16(v[k].z, v[k].w);
      uint8_t* at = smem_pj + Pj::a + warp * Pj::stride + (lane + 32 * k) * 8;
      *reinterpret_cast<uint2*>(at) = make_uint2(t0, t1);
      *reinterpret_cast<uint2*>(at + Pj::rows * Pj::stride) =
          make_uint2(pack_bf16(v[k].x - low(t0), v[k].y - high(t0)), pack_bf16(v[k].z - low(t1), v[k].w - high(t1)));
    }
  }
  cp_async_wait_all();
  __syncthreads();
  const int g = lane >> 2, q = lane & 3, kq = warp >> 1, nh = warp & 1;
  const uint8_t* sW = smem_pj + Pj::w + nh * (kDc * 128);
  float acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll 2
  for (int ks = 0; ks < 8; ++ks) {
    const int k = kq * 128 + ks * 16;
    const uint8_t* lo = smem_pj + Pj::a + g * Pj::stride + (k + 2 * q) * 2;
    auto frag = [&](int row, int at) { return *reinterpret_cast<const uint32_t*>(lo + row * Pj::stride + at); };
    const uint32_t a0 = frag(0, 0), a1 = frag(8, 0), a2 = frag(0, 16), a3 = frag(8, 16);
    const int kr = k + (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(smem_u32(sW + sw128(kr, np * 2 + (lane >> 4))), b0, b1, b2, b3);
      mma_16816(acc[2 * np], a0, a1, a2, a3, b0, b1);
      mma_16816(acc[2 * np + 1], a0, a1, a2, a3, b2, b3);
    }
  }
#pragma unroll
  for (int nt = 0; nt < 8; ++nt)
    *reinterpret_cast<float2*>(sRed + (kq * Pj::rows + g) * kDv + nh * 64 + nt * 8 + 2 * q) =
        make_float2(acc[nt][0] + acc[nt][2], acc[nt][1] + acc[nt][3]);
  __syncthreads();
  const int row = row0 + warp, c = lane * 4;
  if (row >= a.num_q) return;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(sRed + (k * Pj::rows + warp) * kDv + c);
    v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
  }
  *reinterpret_cast<uint2*>(out + ((size_t)row * H + h) * kDv + c) =
      make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

}  // namespace

// tree_proj_kernel reads all of W_uv[h] for 8 rows, out_proj_tc for 128. With at most
// three CTAs of the former an SM it is the faster: 24.5 against 32.1 us for a call of 64
// rows of 16 heads, 31.8 against 37.5 for 128; it takes 51.2 against 52.2 for 256, and
// 68.9 against 67.2 for 32 rows of 128 heads.
cudaError_t launch_tree_out(const TreeArgs& a, const void* W_uv, void* out, cudaStream_t st) {
  const int64_t rows = a.num_q * a.num_heads;
  cudaError_t e = rows < 512 ? launch_pdl(tree_merge_few_kernel, dim3((unsigned)rows), dim3(512), 0, st, a)
                             : launch_pdl(tree_merge_kernel, dim3((unsigned)((rows + 15) / 16)), dim3(256), 0, st, a);
  if (e != cudaSuccess) return e;
  if ((a.num_q + Pj::rows - 1) / Pj::rows * a.num_heads > 6 * a.shares) {
    CUtensorMap w_map;
    if (!encode_map_2d(&w_map, W_uv, kDv, (uint64_t)a.num_heads * kDc, 64, 64)) return cudaErrorInvalidValue;
    return launch_out_proj_tc(w_map, a.o_lat, out, a.num_q, a.num_heads, true, st);
  }
  e = cudaFuncSetAttribute(tree_proj_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Pj::bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_proj_kernel, dim3((unsigned)((a.num_q + Pj::rows - 1) / Pj::rows), a.num_heads), dim3(256),
                    Pj::bytes, st, a, (const __nv_bfloat16*)W_uv, (__nv_bfloat16*)out);
}

}  // namespace mla
