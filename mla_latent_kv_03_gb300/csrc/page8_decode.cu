// mla_page8_decode and mla_page8_decode_mass: split-KV attention of absorbed
// queries over pages of e4m3 codes with one scale per page, the merge of the
// splits, the output projection, and (mass) the attention weight of every
// cached token accumulated at its slot.
//
// For query row n, head h and token t of page p with scale S_p:
//   s_t = softmax_scale * log2(e) * (S_p q_lat . code_t + q_rope . k_t)   (base 2)
//   o   = sum_t 2^(s_t - lse) S_p code_t,     lse = log2 sum_t 2^(s_t)
// The work is cut as in the other decodes (plan_kernel: units of one row, 16
// heads and 64 tokens in equal contiguous shares), the parts are merged by the
// CTA that finishes a (row, 16 heads) last.
#include <cuda_fp8.h>

#include "async_copy.cuh"
#include "internal.h"
#include "merge.cuh"
#include "page8.cuh"
#include "sched.cuh"

namespace mla {
namespace {

constexpr int kSub = 16;  // tokens per inner step

struct P8Args {
  const __nv_bfloat16* q_abs;
  const uint8_t* cache8;
  const float* scales;
  int64_t num_blocks;
  const int32_t* block_table;
  int32_t max_blocks;
  int32_t block_size;
  int32_t num_heads;
  int32_t groups;
  int32_t num_ctas;
  int64_t num_q;
  float scale_log2;
  uint8_t* ws;
  float* o_lat;       // [num_q, H, 512]
  float* lse;         // [num_q, H], base 2
  float* scores;      // [num_q, groups, max tokens, 16], base 2; NULL without mass
};

// The decode workspace: the split plan and partials of ws_layout, then
// the merged latents, their log-sum-exps and (with mass) the scores.
struct P8Ws {
  size_t o_lat, lse, scores, total;
};
P8Ws p8_ws(int64_t num_q, int H, int num_ctas, int64_t max_tokens, bool mass) {
  P8Ws L;
  L.o_lat = align_up(ws_layout(num_q, H / kHG, num_ctas).total, 256);
  L.lse = align_up(L.o_lat + (size_t)num_q * H * kDc * 4, 256);
  L.scores = align_up(L.lse + (size_t)num_q * H * 4, 256);
  L.total = mass ? align_up(L.scores + (size_t)num_q * H * max_tokens * 4, 256) : L.scores;
  return L;
}

__device__ __forceinline__ float page_scale(float s) {
  return fmaxf(s, __uint_as_float((uint32_t)(kP8MinExp + 127) << 23));
}

__global__ void __launch_bounds__(256) page8_decode_kernel(P8Args a) {
  extern __shared__ float smem_f[];
  float* sQ = smem_f;                         // [16][576]
  float* sK = sQ + kHG * kRow;                // [16][577], dequantised
  float* sP = sK + kSub * (kRow + 1);         // [16][16]
  float* sA = sP + kHG * kSub;                // [16] alpha
  float* sL = sA + kHG;                       // [16] final l
  float* sM = sL + kHG;                       // [16] final m
  float* sMerge = sM + kHG;                   // fused-merge scratch
  int* sFlag = reinterpret_cast<int*>(sMerge + 2 * kHG + kMergeChunk * kHG);
  int64_t* sOff = reinterpret_cast<int64_t*>(sFlag + 2);  // [kSub] cache row, -1: none
  float* sS = reinterpret_cast<float*>(sOff + kSub);      // [kSub] page scales
  const int tid = threadIdx.x;
  const int h = tid >> 4, j = tid & 15;       // score role: head h, token j
  const int d0 = tid * 2;                     // output role: columns d0, d0 + 1 of all heads
  WsHeader* hdr = reinterpret_cast<WsHeader*>(a.ws);
  const WsLayout L = ws_layout(a.num_q, a.groups, a.num_ctas);
  float* lse_out = reinterpret_cast<float*>(a.ws + L.lse);
  float* o_out = reinterpret_cast<float*>(a.ws + L.opart);
  pdl_wait();
  pdl_launch_dependents();

  SchedWalker sw;
  const bool has_work = sw.init(a.ws, a.num_q, a.groups, a.num_ctas, blockIdx.x);
  zero_unvisited_rows(sw.row_info, sw.plan_ok, a.num_q, a.num_heads, a.o_lat, tid, 256);
  if (!has_work) return;
  Segment seg;
  while (sw.next(seg)) {
    const int t = seg.n * a.groups + seg.g;
    const int64_t slot = (int64_t)blockIdx.x + t;
    __syncthreads();
    const __nv_bfloat16* qsrc = a.q_abs + ((size_t)seg.n * a.num_heads + seg.g * kHG) * kRow;
    for (int i = tid; i < kHG * kRow; i += 256) sQ[i] = __bfloat162float(qsrc[i]);
    float m = -INFINITY, l = 0.f;
    float o[kHG][2];
#pragma unroll
    for (int r = 0; r < kHG; ++r) o[r][0] = o[r][1] = 0.f;
    const int end = min(seg.pos + 1, seg.k1 * kTile);
    for (int tok0 = seg.k0 * kTile; tok0 < end; tok0 += kSub) {
      __syncthreads();
      if (tid < kSub) {
        const int tok = tok0 + tid;
        int64_t off = -1;
        float sc = 0.f;
        if (tok < end) {
          const int blk = a.block_table[(size_t)seg.b * a.max_blocks + tok / a.block_size];
          if (blk >= 0 && blk < a.num_blocks) {
            off = (int64_t)blk * a.block_size + tok % a.block_size;
            sc = page_scale(a.scales[blk]);
          } else {
            set_status(&hdr->status, MLA_DEV_BAD_BLOCK);
          }
        }
        sOff[tid] = off;
        sS[tid] = sc;
      }
      __syncthreads();
      // 16 rows of 40 16-byte pieces: 32 of codes, 8 of rope values
      for (int i = tid; i < kSub * 40; i += 256) {
        const int r = i / 40, c = i % 40;
        const int64_t off = sOff[r];
        uint4 v = make_uint4(0, 0, 0, 0);
        if (off >= 0) v = *reinterpret_cast<const uint4*>(a.cache8 + off * kRow8 + c * 16);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        float* d = sK + r * (kRow + 1);
        if (c < 32) {
          const float sc = sS[r];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            __nv_fp8_e4m3 code;
            code.__x = (uint8_t)(u[k >> 2] >> (8 * (k & 3)));
            d[c * 16 + k] = off >= 0 ? (float)code * sc : 0.f;
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            d[kDc + (c - 32) * 8 + k] = __uint_as_float((k & 1) ? u[k >> 1] & 0xffff0000u : u[k >> 1] << 16);
        }
      }
      __syncthreads();
      const int tok = tok0 + j;
      const bool live = tok < end && sOff[j] >= 0;
      float s0 = 0.f, s1 = 0.f;
      for (int c = 0; c < kRow; c += 2) {
        s0 = fmaf(sQ[h * kRow + c], sK[j * (kRow + 1) + c], s0);
        s1 = fmaf(sQ[h * kRow + c + 1], sK[j * (kRow + 1) + c + 1], s1);
      }
      const float s = live ? (s0 + s1) * a.scale_log2 : -INFINITY;
      if (a.scores && live)
        a.scores[((size_t)t * a.max_blocks * a.block_size + tok) * kHG + h] = s;
      float mx = s;
#pragma unroll
      for (int o2 = 8; o2 > 0; o2 >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
      const float mn = fmaxf(m, mx);
      const float mu = mn == -INFINITY ? 0.f : mn;
      const float alpha = fast_exp2(m - mu);
      const float p = fast_exp2(s - mu);
      float ps = p;
#pragma unroll
      for (int o2 = 8; o2 > 0; o2 >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o2);
      l = l * alpha + ps;
      m = mn;
      sP[h * kSub + j] = p;
      if (j == 0) sA[h] = alpha;
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kHG; ++r) {
        const float al = sA[r];
        float acc0 = o[r][0] * al, acc1 = o[r][1] * al;
        for (int jj = 0; jj < kSub; ++jj) {
          const float pj = sP[r * kSub + jj];
          acc0 = fmaf(pj, sK[jj * (kRow + 1) + d0], acc0);
          acc1 = fmaf(pj, sK[jj * (kRow + 1) + d0 + 1], acc1);
        }
        o[r][0] = acc0;
        o[r][1] = acc1;
      }
    }
    __syncthreads();
    if (j == 0) { sL[h] = l; sM[h] = m; }
    __syncthreads();
    const int u_first = seg.ustart + seg.g * seg.tiles;
    const int c_first = u_first / sw.share, c_last = (u_first + seg.tiles - 1) / sw.share;
    const bool direct = c_first == c_last;
    float* o_tile = a.o_lat + ((size_t)seg.n * a.num_heads + seg.g * kHG) * kDc;
    float* dst = direct ? o_tile : o_out + (size_t)slot * kHG * kDc;
#pragma unroll
    for (int r = 0; r < kHG; ++r) {
      // (a NaN sum stays NaN)
      const float lr = sL[r];
      const float inv = lr == 0.f ? 0.f : 1.f / lr;
      *reinterpret_cast<float2*>(dst + (size_t)r * kDc + d0) = make_float2(o[r][0] * inv, o[r][1] * inv);
    }
    if (tid < kHG) {
      const float lr = sL[tid], lse = lr == 0.f ? -INFINITY : sM[tid] + log2f(lr);
      if (direct)
        a.lse[(size_t)t * kHG + tid] = lse;
      else
        lse_out[(size_t)slot * kHG + tid] = lse;
    }
    if (!direct) {
      int* arrive = reinterpret_cast<int*>(a.ws + L.arrive);
      __threadfence();  // publish protocol: see count_arrival
      __syncthreads();
      if (tid == 0) sFlag[0] = count_arrival(&arrive[t]) == c_last - c_first;
      __syncthreads();
      if (sFlag[0]) {
        merge_qtile<256>(lse_out, o_out, (int64_t)c_first + t, c_last - c_first + 1, 1, o_tile, tid,
                         sMerge, [] { __syncthreads(); });
        // merge_qtile leaves the maxima and inverse weight sums in its scratch
        if (tid < kHG) a.lse[(size_t)t * kHG + tid] = sMerge[tid] - log2f(sMerge[kHG + tid]);
        if (tid == 0) arrive[t] = 0;  // every part has arrived: ready for the next launch
      }
      __syncthreads();
    }
  }
}

// mass[slot(t)] = decay * mass[slot(t)] + sum over the sequence's rows and all
// heads of 2^(score - lse), rows and heads in order: one thread per token.
struct MassArgs {
  const float* scores;
  const float* lse;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  const int32_t* block_table;
  int32_t max_blocks, block_size, groups;
  int64_t num_q, num_blocks;
  float decay;
  float* mass;
};
__global__ void __launch_bounds__(256) page8_mass_kernel(MassArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, t = blockIdx.x * 256 + threadIdx.x;
  const int len = a.seq_lens[b], q0 = a.query_start_loc[b], q1 = a.query_start_loc[b + 1];
  const int ql = q1 - q0;
  const int64_t max_tokens = (int64_t)a.max_blocks * a.block_size;
  if (q0 < 0 || q1 > a.num_q || ql <= 0 || ql > len || (int64_t)len > max_tokens) return;
  if (t >= len) return;
  const int32_t p = a.block_table[(size_t)b * a.max_blocks + t / a.block_size];
  if (p < 0 || p >= a.num_blocks) return;
  float sum = 0.f;
  for (int n = max(q0, q0 + t - (len - ql)); n < q1; ++n) {  // rows at or behind token t
    for (int g = 0; g < a.groups; ++g) {
      const size_t tile = (size_t)n * a.groups + g;
      const float4* s = reinterpret_cast<const float4*>(a.scores + (tile * max_tokens + t) * kHG);
      const float4* e = reinterpret_cast<const float4*>(a.lse + tile * kHG);
#pragma unroll
      for (int k = 0; k < kHG / 4; ++k) {
        const float4 x = s[k], y = e[k];
        sum += fast_exp2(x.x - y.x) + fast_exp2(x.y - y.y) + fast_exp2(x.z - y.z) + fast_exp2(x.w - y.w);
      }
    }
  }
  float* m = a.mass + (size_t)p * a.block_size + t % a.block_size;
  *m = a.decay > 0.f ? fmaf(a.decay, *m, sum) : sum;
}

mla_status p8_decode(const mla_config* cfg, const void* q_abs, const void* cache8,
                     const float* page_scales, int64_t num_blocks, const int32_t* block_table,
                     int32_t max_blocks, const int32_t* seq_lens, const int32_t* query_start_loc,
                     int32_t batch, int64_t num_q, const void* W_uv, float* mass, float decay,
                     bool with_mass, void* workspace, size_t ws_bytes, void* out, void* stream) {
  if (validate_config(cfg) == MLA_OK && cfg->dtype != MLA_BF16) return MLA_ERR_UNSUPPORTED;
  mla_status s = decode_paged_checks(cfg, q_abs, cache8, num_blocks, block_table, max_blocks,
                                     seq_lens, query_start_loc, batch, num_q);
  if (s != MLA_OK) return s;
  if (with_mass && !(decay >= 0.f && decay <= 1.f)) return MLA_ERR_INVALID_ARGUMENT;
  if (!workspace || !p8_aligned(workspace, 256)) return MLA_ERR_INVALID_ARGUMENT;
  if (num_q == 0) return MLA_OK;
  if (!page_scales || !W_uv || !out || (with_mass && !mass)) return MLA_ERR_INVALID_ARGUMENT;
  if (!p8_aligned(page_scales, 4) || !p8_aligned(W_uv, 16) || !p8_aligned(out, 16) ||
      !p8_aligned(mass, 4))
    return MLA_ERR_INVALID_ARGUMENT;
  if (with_mass && batch > 65535) return MLA_ERR_UNSUPPORTED;
  const size_t need = mla_page8_decode_workspace_size(cfg, num_q, batch, max_blocks, with_mass);
  if (need == 0) return MLA_ERR_UNSUPPORTED;
  if (ws_bytes < need) return MLA_ERR_WORKSPACE_TOO_SMALL;
  const int C = split_ctas(cfg), H = cfg->num_heads, bs = cfg->block_size;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const P8Ws L = p8_ws(num_q, H, C, (int64_t)max_blocks * bs, with_mass);
  const PlanArgs pa{seq_lens, query_start_loc, batch, (int32_t)num_q, H / kHG, C, bs, max_blocks,
                    workspace};
  cudaError_t e = launch_plan(pa, st);
  if (e != cudaSuccess) return MLA_ERR_CUDA;
  P8Args a{(const __nv_bfloat16*)q_abs, (const uint8_t*)cache8, page_scales, num_blocks,
           block_table, max_blocks, bs, H, H / kHG, C, num_q,
           (float)(cfg->softmax_scale * 1.4426950408889634), ws,
           reinterpret_cast<float*>(ws + L.o_lat), reinterpret_cast<float*>(ws + L.lse),
           with_mass ? reinterpret_cast<float*>(ws + L.scores) : nullptr};
  const size_t smem =
      (size_t)(kHG * kRow + kSub * (kRow + 1) + kHG * kSub + 3 * kHG + 2 * kHG + kMergeChunk * kHG + 2) * 4 +
      kSub * 12;
  e = cudaFuncSetAttribute(page8_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = launch_pdl(page8_decode_kernel, dim3(C), dim3(256), smem, st, a);
  if (e != cudaSuccess) return MLA_ERR_CUDA;
  if (with_mass) {
    const MassArgs ma{a.scores, a.lse, seq_lens, query_start_loc, block_table, max_blocks, bs,
                      H / kHG, num_q, num_blocks, decay, mass};
    const int64_t tokens = (int64_t)max_blocks * bs;
    if (tokens > 0) {
      e = launch_pdl(page8_mass_kernel, dim3((unsigned)((tokens + 255) / 256), (unsigned)batch),
                     dim3(256), 0, st, ma);
      if (e != cudaSuccess) return MLA_ERR_CUDA;
    }
  }
  return mla_out_proj(cfg, a.o_lat, W_uv, out, num_q, stream);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_page8_decode_workspace_size(const mla_config* cfg, int64_t num_q, int32_t batch,
                                       int32_t max_blocks_per_seq, int32_t with_mass) {
  if (validate_config(cfg) != MLA_OK || cfg->dtype != MLA_BF16 || num_q < 0 ||
      num_q > 48 * 1024 || batch < 0 || max_blocks_per_seq < 0 ||
      max_blocks_per_seq > ((int64_t)1 << 31) / cfg->block_size)
    return 0;
  const int C = split_ctas(cfg);
  if (C <= 0) return 0;
  return p8_ws(num_q, cfg->num_heads, C, (int64_t)max_blocks_per_seq * cfg->block_size,
               with_mass != 0)
      .total;
}

mla_status mla_page8_decode(const mla_config* cfg, const void* q_abs, const void* cache8,
                            const float* page_scales, int64_t num_blocks,
                            const int32_t* block_table, int32_t max_blocks_per_seq,
                            const int32_t* seq_lens, const int32_t* query_start_loc,
                            int32_t batch, int64_t num_q, const void* W_uv, void* workspace,
                            size_t ws_bytes, void* out, void* stream) {
  return p8_decode(cfg, q_abs, cache8, page_scales, num_blocks, block_table, max_blocks_per_seq,
                   seq_lens, query_start_loc, batch, num_q, W_uv, nullptr, 0.f, false, workspace,
                   ws_bytes, out, stream);
}

mla_status mla_page8_decode_mass(const mla_config* cfg, const void* q_abs, const void* cache8,
                                 const float* page_scales, int64_t num_blocks,
                                 const int32_t* block_table, int32_t max_blocks_per_seq,
                                 const int32_t* seq_lens, const int32_t* query_start_loc,
                                 int32_t batch, int64_t num_q, const void* W_uv, float* mass,
                                 float decay, void* workspace, size_t ws_bytes, void* out,
                                 void* stream) {
  return p8_decode(cfg, q_abs, cache8, page_scales, num_blocks, block_table, max_blocks_per_seq,
                   seq_lens, query_start_loc, batch, num_q, W_uv, mass, decay, true, workspace,
                   ws_bytes, out, stream);
}

}  // extern "C"
