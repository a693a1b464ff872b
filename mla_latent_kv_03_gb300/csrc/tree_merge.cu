// What follows the attention of mla_tree_decode: the merge of each (row, head)'s
// parts, weighed by their log-sum-exps, and the output projection
//   out[n,h] = o_lat[n,h] W_uv[h]        ([512] . [512, 128]).
#include "async_copy.cuh"
#include "pair_math.cuh"
#include "tcgen05.cuh"
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

// The merge and the projection in one, for many (row, head)s: CTA = (R rows, head
// h). A warp finds the parts of every eighth row, loads and weighs them, and
// splits each to two bf16 terms, so that the output is rounded once. The products have
// the output's columns as the 128 rows of the accumulator and the terms as its 2 R
// columns: W_uv[h], 64 k-rows a stage by TMA, is the first operand as it lies in memory.
// Bound by the parts' bytes from the L2 and by latency: behind the attention it adds
// 13 us to a call of 64 x 4,096 tokens and 8 rows; a merge that wrote the latents, and a
// projection that read them, added 26.
template <int R>
struct Pt {
  static constexpr int stages = 3;
  static constexpr int chunk = 2 * R * 128;       // 64 latents of the rows' first, then of their second terms
  static constexpr int wstage = 64 * 256;         // two slabs of 64 columns
  static constexpr int w = 0;
  static constexpr int terms = w + stages * wstage;
  static constexpr int bars = terms + 8 * chunk;  // full[stages], free[stages], done
  static constexpr int misc = bars + (2 * stages + 1) * 8;
  static constexpr int bytes = misc + 16;
  static constexpr uint32_t cols = 2 * R < 32 ? 32 : 2 * R;
};
template <int R>
__global__ void __launch_bounds__(256, 2)
    tree_merge_proj_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ TreeArgs a, __nv_bfloat16* out) {
  using M = Pt<R>;
  constexpr int kAhead = 4;
  extern __shared__ __align__(1024) uint8_t smem_pt[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_pt + M::bars);
  uint64_t* free_ = full + M::stages;
  uint64_t* done = free_ + M::stages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_pt + M::misc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, row0 = blockIdx.x * R, H = a.num_heads;
  auto load_w = [&](int c) {
    uint64_t* bar = full + c % M::stages;
    uint8_t* dst = smem_pt + M::w + c % M::stages * M::wstage;
    mbar_arrive_expect_tx(bar, M::wstage);
    tma_load_2d(dst, &w_map, 0, h * kDc + 64 * c, bar);
    tma_load_2d(dst + M::wstage / 2, &w_map, 64, h * kDc + 64 * c, bar);
  };
  if (tid == 0) {
    for (int i = 0; i < 2 * M::stages + 1; ++i) mbar_init(full + i, 1);
    fence_mbar_init();
    for (int c = 0; c < M::stages; ++c) load_w(c);     // (W_uv does not depend on earlier kernels)
  }
  if (warp == 0) tc::alloc(tmem_slot, M::cols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();
  // A row's two terms: latents 4 lane + 128 k and on, in chunk 2 k + lane / 16.
  auto put = [&](int r, const float4 (&x)[4]) {
    auto low = [](uint32_t t) { return __uint_as_float(t << 16); };
    auto high = [](uint32_t t) { return __uint_as_float(t & 0xffff0000u); };
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t t0 = pack_bf16(x[k].x, x[k].y), t1 = pack_bf16(x[k].z, x[k].w);
      uint8_t* at = smem_pt + M::terms + (2 * k + (lane >> 4)) * M::chunk + sw128(r, (lane & 15) >> 1) + (lane & 1) * 8;
      *reinterpret_cast<uint2*>(at) = make_uint2(t0, t1);
      *reinterpret_cast<uint2*>(at + R * 128) =
          make_uint2(pack_bf16(x[k].x - low(t0), x[k].y - high(t0)), pack_bf16(x[k].z - low(t1), x[k].w - high(t1)));
    }
  };
  auto add = [](float4 (&acc)[4], const float4 (&v)[4], float x0, float x1) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = k < 2 ? x0 : x1;
      acc[k].x = fmaf(x, v[k].x, acc[k].x);
      acc[k].y = fmaf(x, v[k].y, acc[k].y);
      acc[k].z = fmaf(x, v[k].z, acc[k].z);
      acc[k].w = fmaf(x, v[k].w, acc[k].w);
    }
  };
  // This warp's rows are row0 + warp + 8 j; kLanes lanes find the parts of each.
  constexpr int kLanes = 32 / (R / 8);
  const RowParts mine = row_parts(a, row0 + warp + 8 * (lane / kLanes), h);
  const int i = lane % kLanes;
  const bool few = mine.count <= kLanes, have = few && i < mine.count;
  const float4* src = reinterpret_cast<const float4*>(a.o_lat);
  float l0 = -INFINITY, l1 = -INFINITY;
  if (have && mine.count == 1) {
    src += ((size_t)(row0 + warp + 8 * (lane / kLanes)) * H + h) * (kDc / 4);
    l0 = l1 = 0.f;
  } else if (have) {
    const int64_t slot = mine.slot(i);
    src = reinterpret_cast<const float4*>(a.opart) + (slot * kTreeBlockRows + mine.r) * (kDc / 4);
    l0 = a.lse[slot * 2 * kTreeBlockRows + mine.r];
    l1 = a.lse[(slot * 2 + 1) * kTreeBlockRows + mine.r];
  }
  float m0 = l0, m1 = l1;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
  float w0 = fast_exp2(l0 - (m0 == -INFINITY ? 0.f : m0)), w1 = fast_exp2(l1 - (m1 == -INFINITY ? 0.f : m1));
  float d0 = w0, d1 = w1;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    d0 += __shfl_xor_sync(0xffffffffu, d0, o);
    d1 += __shfl_xor_sync(0xffffffffu, d1, o);
  }
  w0 = d0 == 0.f ? 0.f : w0 / d0;         // (a row that sees nothing: weights of 0)
  w1 = d1 == 0.f ? 0.f : w1 / d1;
  // all parts of all rows one behind another, kAhead on their way at a time
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  uint32_t todo = __ballot_sync(0xffffffffu, have);
  const uint32_t none = __ballot_sync(0xffffffffu, mine.count == 0 && i == 0), many = __ballot_sync(0xffffffffu, !few && i == 0);
#pragma unroll 1
  for (uint32_t rows = none; rows; rows &= rows - 1) put(warp + 8 * ((__ffs(rows) - 1) / kLanes), acc);
#pragma unroll 1
  while (todo) {
    float4 v[kAhead][4];
    uint32_t left = todo;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int from = left ? __ffs(left) - 1 : 0;
      const float4* p = reinterpret_cast<const float4*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), from));
      if (left) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[u][k] = __ldcs(p + lane + 32 * k);
      }
      left &= left - 1;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (!todo) break;
      const int from = __ffs(todo) - 1;
      todo &= todo - 1;
      add(acc, v[u], __shfl_sync(0xffffffffu, w0, from), __shfl_sync(0xffffffffu, w1, from));
      if (!todo || (__ffs(todo) - 1) / kLanes != from / kLanes) {     // the row's last part
        put(warp + 8 * (from / kLanes), acc);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
  }
  // rows of more parts: 32 at a time
#pragma unroll 1
  for (uint32_t rows = many; rows; rows &= rows - 1) {
    const int owner = __ffs(rows) - 1, r = warp + 8 * (owner / kLanes);
    const RowParts rp = row_parts(a, row0 + r, h);
    auto part = [&](int n, int& slot, float& x0, float& x1) {
      slot = 0;
      x0 = x1 = -INFINITY;
      if (n < rp.count) {
        slot = rp.slot(n);
        x0 = a.lse[(int64_t)slot * 2 * kTreeBlockRows + rp.r];
        x1 = a.lse[((int64_t)slot * 2 + 1) * kTreeBlockRows + rp.r];
      }
    };
    int slot = 0;
    float x0, x1, n0 = -INFINITY, n1 = -INFINITY, e0 = 0.f, e1 = 0.f;
#pragma unroll 1
    for (int s0 = 0; s0 < rp.count; s0 += 32) {
      part(s0 + lane, slot, x0, x1);
      n0 = fmaxf(n0, x0);
      n1 = fmaxf(n1, x1);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
      n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
    }
    if (n0 == -INFINITY) n0 = 0.f;
    if (n1 == -INFINITY) n1 = 0.f;
#pragma unroll 1
    for (int s0 = 0; s0 < rp.count; s0 += 32) {
      part(s0 + lane, slot, x0, x1);
      x0 = fast_exp2(x0 - n0);
      x1 = fast_exp2(x1 - n1);
      e0 += x0;
      e1 += x1;
      const int live = min(32, rp.count - s0);
#pragma unroll 1
      for (int u0 = 0; u0 < live; u0 += kAhead) {
        float4 v[kAhead][4];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int from = __shfl_sync(0xffffffffu, slot, (u0 + u) & 31);
          const float4* p = reinterpret_cast<const float4*>(a.opart + ((int64_t)from * kTreeBlockRows + rp.r) * kDc) + lane;
          if (u0 + u < live) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[u][k] = __ldcs(p + 32 * k);
          }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (u0 + u < live)
            add(acc, v[u], __shfl_sync(0xffffffffu, x0, (u0 + u) & 31), __shfl_sync(0xffffffffu, x1, (u0 + u) & 31));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      e0 += __shfl_xor_sync(0xffffffffu, e0, o);
      e1 += __shfl_xor_sync(0xffffffffu, e1, o);
    }
    e0 = e0 == 0.f ? 0.f : 1.f / e0;
    e1 = e1 == 0.f ? 0.f : 1.f / e1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float d = k < 2 ? e0 : e1;
      acc[k] = make_float4(acc[k].x * d, acc[k].y * d, acc[k].z * d, acc[k].w * d);
    }
    put(r, acc);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  bool ok = true;
  if (warp == 0) {
    constexpr uint32_t kId = tc::idesc_bf16(128, 2 * R, true, false);
    const uint64_t wdesc = tc::smem_desc(smem_u32(smem_pt + M::w), M::wstage / 2, 1024, tc::kSwizzle128);
    const uint64_t tdesc = tc::smem_desc(smem_u32(smem_pt + M::terms), 16, 1024, tc::kSwizzle128);
    const bool leader = tc::elect_one();
    int loaded = M::stages, c = 0;
#pragma unroll 1
    for (; c < 8; ++c) {
      const int at = c % M::stages;
      if (c > 0 && loaded < 8) {      // the stage of the chunk before takes the next
        if (!(ok = mbar_wait(free_ + (c - 1) % M::stages, ((c - 1) / M::stages) & 1))) break;
        if (lane == 0) load_w(loaded);
        ++loaded;
      }
      if (!(ok = mbar_wait(full + at, (c / M::stages) & 1))) break;
      tc::fence_after_sync();
      if (leader) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc::mma_bf16(tmem, wdesc + (uint64_t)((at * M::wstage + k * 16 * 128) >> 4),
                       tdesc + (uint64_t)((c * M::chunk + k * 32) >> 4), kId, c > 0 || k > 0);
        tc::commit(free_ + at);
      }
      __syncwarp();
    }
    if (leader) tc::commit(done);
    __syncwarp();
    if (!ok)       // never leave with copies in flight
      for (; c < loaded; ++c) mbar_wait(full + c % M::stages, (c / M::stages) & 1);
  }
  ok = __syncthreads_and(mbar_wait(done, 0) && ok);
  tc::fence_after_sync();
  // thread = output column, the rows behind one another
  if (warp < 4) {
    __nv_bfloat16* dst = out + ((size_t)row0 * H + h) * kDv + warp * 32 + lane;
    const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16);
    uint32_t v[32], y[32];
    tc::ld32(at, v);
    if (R == 32) tc::ld32(at + 32, y);
    tc::wait_ld();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float second = __uint_as_float(R == 32 ? y[r] : v[(R + r) & 31]);
      const float x = ok ? __uint_as_float(v[r]) + second : NAN;     // (no result: not passed for one)
      if (row0 + r < a.num_q) dst[(size_t)r * H * kDv] = __float2bfloat16_rn(x);
    }
    tc::fence_before_sync();
  }
  if (!ok && tid == 0) set_status(a.status, MLA_DEV_TIMEOUT);
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::dealloc(tmem, M::cols);
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

// Few (row, head)s with many parts want a CTA each for the merge; more of them are merged
// where they are projected. In graphs, us, a merge of its own / in one: 1 x 8 rows of 16
// heads over 4,096 tokens 23.0 / 43.6, over 30,000 31.2 / 53.2; 512 (row, head)s (4 x 8
// rows) 25.8 / 29.5; 1,024 (8 x 8 rows) 39.1 / 35.1, (2 x 4 of 128 heads) 47.3 / 43.4;
// 4,096 96.1 / 56.6. Of few parts a row: 1 x 6 rows of 16 heads over 64 tokens 14.9 / 17.1,
// over 333 17.8 / 19.4, over 1,024 17.3 / 20.5; 512 (row, head)s (4 x 8 rows) over 64 17.0 /
// 18.7, over 333 21.2 / 21.2, over 1,024 21.9 / 26.0. Rows of a CTA: the most that leave a CTA an SM (W_uv[h] is read for
// each). 32 / 16 / 8: 64 x 8 rows of 16 heads 87.6 / 93.9 / 106; 8 x 4 of 128 heads
// 174.8 / 162.9 / 169.5; 12 x 2 of 32 heads 22.5 / 21.3 / 20.5. (64 rows with 512
// threads: 88.5 for the first, 127 against 121 for 11 x 70 rows of 64 heads.)
cudaError_t launch_tree_out(const TreeArgs& a, const void* W_uv, void* out, cudaStream_t st) {
  const int64_t rows = a.num_q * a.num_heads;
  if (rows >= 768) {
    CUtensorMap w_map;
    if (!encode_map_2d(&w_map, W_uv, kDv, (uint64_t)a.num_heads * kDc, 64, 64)) return cudaErrorInvalidValue;
    auto both = [&](auto kernel, int per, int smem) {
      const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      return r != cudaSuccess ? r
                              : launch_pdl(kernel, dim3((unsigned)((a.num_q + per - 1) / per), a.num_heads),
                                           dim3(256), smem, st, w_map, a, (__nv_bfloat16*)out);
    };
    auto ctas = [&](int per) { return (a.num_q + per - 1) / per * a.num_heads; };
    return ctas(32) >= 2 * a.shares   ? both(tree_merge_proj_kernel<32>, 32, Pt<32>::bytes)
           : ctas(16) >= 2 * a.shares ? both(tree_merge_proj_kernel<16>, 16, Pt<16>::bytes)
                                      : both(tree_merge_proj_kernel<8>, 8, Pt<8>::bytes);
  }
  cudaError_t e = launch_pdl(tree_merge_few_kernel, dim3((unsigned)rows), dim3(512), 0, st, a);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(tree_proj_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Pj::bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_proj_kernel, dim3((unsigned)((a.num_q + Pj::rows - 1) / Pj::rows), a.num_heads), dim3(256),
                    Pj::bytes, st, a, (const __nv_bfloat16*)W_uv, (__nv_bfloat16*)out);
}

}  // namespace mla
