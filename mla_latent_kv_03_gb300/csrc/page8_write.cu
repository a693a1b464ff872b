// mla_page8_cache_write: RMSNorm of the latent, RoPE of the shared key, and
// the write of both into pages of e4m3 codes with one power-of-two scale to a
// page.
//
// A page's scale goes by all of its rows that a call writes, so a page is the
// unit of work: one CTA finds the page's tokens, normalises their latents
// (kept in registers between the two uses), takes the largest magnitude,
// grows the scale if it must, recodes the page's other rows if it grew, and
// writes the new rows. Nothing depends on the order in which CTAs run: one CTA
// owns the page, and a slot named twice goes to the later token.
//
// Which tokens fall into a page is found in one of two ways.
//  - Up to kScanTokens tokens (a decode step): CTA t owns the page of token t
//    if no earlier token has that page; it reads the whole slot mapping, a few
//    kilobytes from L2. One launch.
//  - More tokens (prompts): a first kernel numbers the touched pages, a second
//    notes each slot's last token, and the page CTAs walk the numbered list.
// A power of two as the scale makes the growth exact for every code that does
// not become subnormal, and makes the rounded values independent of the scale
// (e4m3 is a floating format), so a token's value does not depend on its
// neighbours in the page.
//
// Bound: HBM, 1,152 bytes read and 640 written per token.
#include "async_copy.cuh"
#include "internal.h"
#include "page8.cuh"
#include "rope_pairs.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kScanTokens = 1024;

struct P8WriteArgs {
  const __nv_bfloat16* c_kv;
  const __nv_bfloat16* k_pe;
  const int32_t* positions;
  const int64_t* slots;
  int num_tokens;
  const __nv_bfloat16* w;
  uint8_t* cache8;
  float* scales;
  int64_t num_blocks;
  float* mass;
  float eps;
  int interleaved;
  uint32_t* status;
};

// The workspace of the numbered form.
struct P8WriteWs {
  size_t count, id_of, list, last, total;
};
P8WriteWs write_ws(int64_t tokens, int64_t num_blocks, int bs) {
  const int64_t pages = tokens < num_blocks ? tokens : num_blocks;
  P8WriteWs L;
  L.count = 0;
  L.id_of = 256;
  L.last = align_up(L.id_of + (size_t)num_blocks * 4, 256);
  L.list = align_up(L.last + (size_t)pages * bs * 4, 256);
  L.total = align_up(L.list + (size_t)pages * 4, 256);
  return L;
}

__device__ __forceinline__ void unpack2(uint32_t v, float& a, float& b) {
  a = __uint_as_float(v << 16);
  b = __uint_as_float(v & 0xffff0000u);
}

// One page: sTok[r] is the token of row r, or -1. All threads call it.
template <int BS>
__device__ __forceinline__ void write_page(const P8WriteArgs& a, const RopeFreq& freq, int64_t page,
                                           const int* sTok, float* sMax) {
  constexpr int kRows = BS / kWarps;  // rows of one warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float old = a.scales[page];
  int tok[kRows];
  uint4 x[kRows][2];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    tok[i] = sTok[warp + kWarps * i];
    if (tok[i] >= 0) {
      const uint4* src = reinterpret_cast<const uint4*>(a.c_kv + (size_t)tok[i] * kDc + lane * 16);
      x[i][0] = __ldg(src);
      x[i][1] = __ldg(src + 1);
    } else {
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    }
  }
  float w[16];
  {
    const uint4* wp = reinterpret_cast<const uint4*>(a.w + lane * 16);
    const uint4 w0 = __ldg(wp), w1 = __ldg(wp + 1);
    const uint32_t u[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) unpack2(u[k], w[2 * k], w[2 * k + 1]);
  }
  // c_hat = x r w, fp32; the largest magnitude over the warp's rows
  float rn[kRows], amax = 0.f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint32_t u[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w,
                           x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float v0, v1;
      unpack2(u[k], v0, v1);
      ss = fmaf(v0, v0, ss);
      ss = fmaf(v1, v1, ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    rn[i] = 1.0f / sqrtf(ss * (1.0f / kDc) + a.eps);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float v0, v1;
      unpack2(u[k], v0, v1);
      amax = fmaxf(amax, fmaxf(fabsf(v0 * rn[i] * w[2 * k]), fabsf(v1 * rn[i] * w[2 * k + 1])));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (lane == 0) sMax[warp] = amax;
  __syncthreads();
  amax = sMax[0];
#pragma unroll
  for (int k = 1; k < kWarps; ++k) amax = fmaxf(amax, sMax[k]);
  const float scale = fmaxf(old, p8_scale_for(amax));
  if (threadIdx.x == 0 && scale != old) a.scales[page] = scale;
  const float inv = 1.0f / scale;
  const bool grew = old > 0.f && scale > old;
  const float f = grew ? old / scale : 1.f;

#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t slot = page * BS + warp + kWarps * i;
    uint8_t* dst = a.cache8 + slot * kRow8;
    uint4* codes = reinterpret_cast<uint4*>(dst + lane * 16);
    if (tok[i] < 0) {
      if (grew) *codes = p8_recode16(*codes, f);
      continue;
    }
    const uint32_t u[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w,
                           x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
    uint32_t q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v0, v1, v2, v3;
      unpack2(u[2 * k], v0, v1);
      unpack2(u[2 * k + 1], v2, v3);
      q[k] = (uint32_t)__nv_cvt_float2_to_fp8x2(
                 make_float2(v0 * rn[i] * w[4 * k] * inv, v1 * rn[i] * w[4 * k + 1] * inv),
                 __NV_SATFINITE, __NV_E4M3) |
             ((uint32_t)__nv_cvt_float2_to_fp8x2(
                  make_float2(v2 * rn[i] * w[4 * k + 2] * inv, v3 * rn[i] * w[4 * k + 3] * inv),
                  __NV_SATFINITE, __NV_E4M3)
              << 16);
    }
    *codes = make_uint4(q[0], q[1], q[2], q[3]);
    const int i1 = rope_i1(a.interleaved, lane), i2 = rope_i2(a.interleaved, lane);
    const __nv_bfloat16* kp = a.k_pe + (size_t)tok[i] * kDr;
    const float x1 = __bfloat162float(kp[i1]), x2 = __bfloat162float(kp[i2]);
    float cs, sn;
    rope_cos_sin(a.positions[tok[i]], freq.hi[lane], freq.lo[lane], &cs, &sn);
    __nv_bfloat16* kr = reinterpret_cast<__nv_bfloat16*>(dst + kDc);
    kr[i1] = __float2bfloat16_rn(x1 * cs - x2 * sn);
    kr[i2] = __float2bfloat16_rn(x2 * cs + x1 * sn);
    if (a.mass && lane == 0) a.mass[slot] = 0.f;
  }
}

template <int BS>
__global__ void __launch_bounds__(kThreads) p8_write_scan_kernel(P8WriteArgs a,
                                                                 const __grid_constant__ RopeFreq freq) {
  __shared__ int sTok[BS];
  __shared__ float sMax[kWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x;
  const int64_t slot = a.slots[t], num_slots = a.num_blocks * BS;
  if (slot < 0) return;
  if (slot >= num_slots) {
    if (threadIdx.x == 0) set_status(a.status, MLA_DEV_BAD_SLOT);
    return;
  }
  const int64_t page = slot / BS;
  for (int r = threadIdx.x; r < BS; r += kThreads) sTok[r] = -1;
  __syncthreads();
  bool earlier = false;
  for (int j = threadIdx.x; j < a.num_tokens; j += kThreads) {
    const int64_t s = a.slots[j];
    if (s >= 0 && s < num_slots && s / BS == page) {
      earlier |= j < t;
      atomicMax(&sTok[s % BS], j);
    }
  }
  if (__syncthreads_or(earlier)) return;  // an earlier token's CTA owns the page
  write_page<BS>(a, freq, page, sTok, sMax);
}

// Numbers the pages that the call's tokens touch: id_of[page] = number + 1.
__global__ void __launch_bounds__(kThreads) p8_number_pages_kernel(P8WriteArgs a, int bs, int* count,
                                                                   int* id_of, int* list) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x * kThreads + threadIdx.x;
  if (t >= a.num_tokens) return;
  const int64_t slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.num_blocks * bs) {
    set_status(a.status, MLA_DEV_BAD_SLOT);
    return;
  }
  const int64_t page = slot / bs;
  if (t > 0) {  // the token before it asks for the same page
    const int64_t before = a.slots[t - 1];
    if (before >= 0 && before / bs == page) return;
  }
  if (atomicCAS(&id_of[page], 0, -1) == 0) {
    const int id = atomicAdd(count, 1);
    list[id] = (int)page;
    id_of[page] = id + 1;
  }
}

__global__ void __launch_bounds__(kThreads) p8_last_token_kernel(P8WriteArgs a, int bs,
                                                                 const int* id_of, int* last) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x * kThreads + threadIdx.x;
  if (t >= a.num_tokens) return;
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.num_blocks * bs) return;
  atomicMax(&last[(size_t)(id_of[slot / bs] - 1) * bs + slot % bs], t + 1);
}

template <int BS>
__global__ void __launch_bounds__(kThreads) p8_write_pages_kernel(P8WriteArgs a,
                                                                  const __grid_constant__ RopeFreq freq,
                                                                  const int* count, const int* list,
                                                                  const int* last) {
  __shared__ int sTok[BS];
  __shared__ float sMax[kWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int n = *count;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    __syncthreads();  // the last page's rows and maxima are read
    for (int r = threadIdx.x; r < BS; r += kThreads) sTok[r] = last[(size_t)i * BS + r] - 1;
    __syncthreads();
    write_page<BS>(a, freq, list[i], sTok, sMax);
  }
}

template <int BS>
cudaError_t write_pages(const P8WriteArgs& a, const RopeFreq& freq, uint8_t* ws, cudaStream_t st) {
  if (a.num_tokens <= kScanTokens)
    return launch_pdl(p8_write_scan_kernel<BS>, dim3(a.num_tokens), dim3(kThreads), 0, st, a, freq);
  const P8WriteWs L = write_ws(a.num_tokens, a.num_blocks, BS);
  int* count = reinterpret_cast<int*>(ws + L.count);
  int* id_of = reinterpret_cast<int*>(ws + L.id_of);
  int* last = reinterpret_cast<int*>(ws + L.last);
  int* list = reinterpret_cast<int*>(ws + L.list);
  cudaError_t e = cudaMemsetAsync(ws, 0, L.list, st);  // count, id_of and last
  const dim3 grid((unsigned)((a.num_tokens + kThreads - 1) / kThreads));
  if (e == cudaSuccess)
    e = launch_pdl(p8_number_pages_kernel, grid, dim3(kThreads), 0, st, a, BS, count, id_of, list);
  if (e == cudaSuccess)
    e = launch_pdl(p8_last_token_kernel, grid, dim3(kThreads), 0, st, a, BS, (const int*)id_of, last);
  if (e != cudaSuccess) return e;
  const int64_t pages = a.num_tokens < a.num_blocks ? a.num_tokens : a.num_blocks;
  return launch_pdl(p8_write_pages_kernel<BS>, dim3((unsigned)(pages < 65536 ? pages : 65536)),
                    dim3(kThreads), 0, st, a, freq, (const int*)count, (const int*)list,
                    (const int*)last);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_page8_write_workspace_size(const mla_config* cfg, int64_t num_tokens, int64_t num_blocks) {
  if (validate_config(cfg) != MLA_OK || cfg->dtype != MLA_BF16 || num_tokens < 0 ||
      num_tokens > ((int64_t)1 << 30) || num_blocks < 0 ||
      num_blocks > ((int64_t)1 << 31) / cfg->block_size)
    return 0;
  // the one-launch form needs none; what is asked for is never zero, which
  // stands for a refusal
  return num_tokens <= kScanTokens ? 256 : write_ws(num_tokens, num_blocks, cfg->block_size).total;
}

mla_status mla_page8_cache_write(const mla_config* cfg, const void* c_kv, const void* k_pe,
                                 const int32_t* positions, const int64_t* slot_mapping,
                                 int64_t num_tokens, const void* rms_weight, void* cache8,
                                 float* page_scales, int64_t num_blocks, float* mass,
                                 void* workspace, size_t ws_bytes, uint32_t* dev_status,
                                 void* stream) {
  mla_status s = validate_config(cfg);
  if (s != MLA_OK) return s;
  if (cfg->dtype != MLA_BF16) return MLA_ERR_UNSUPPORTED;
  if (num_tokens < 0 || num_tokens > ((int64_t)1 << 30) || num_blocks < 0)
    return MLA_ERR_INVALID_ARGUMENT;
  if (num_blocks > ((int64_t)1 << 31) / cfg->block_size) return MLA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MLA_OK;
  if (!c_kv || !k_pe || !positions || !slot_mapping || !rms_weight || !cache8 || !page_scales ||
      !workspace)
    return MLA_ERR_INVALID_ARGUMENT;
  if (!p8_aligned(c_kv, 16) || !p8_aligned(k_pe, 16) || !p8_aligned(rms_weight, 16) ||
      !p8_aligned(cache8, 16) || !p8_aligned(positions, 4) || !p8_aligned(slot_mapping, 8) ||
      !p8_aligned(page_scales, 4) || !p8_aligned(mass, 4) || !p8_aligned(dev_status, 4) ||
      !p8_aligned(workspace, 256))
    return MLA_ERR_INVALID_ARGUMENT;
  if (ws_bytes < mla_page8_write_workspace_size(cfg, num_tokens, num_blocks))
    return MLA_ERR_WORKSPACE_TOO_SMALL;
  P8WriteArgs a{(const __nv_bfloat16*)c_kv, (const __nv_bfloat16*)k_pe, positions, slot_mapping,
                (int)num_tokens, (const __nv_bfloat16*)rms_weight, (uint8_t*)cache8, page_scales,
                num_blocks, mass, cfg->rms_eps, cfg->rope_interleaved, dev_status};
  const RopeFreq freq = make_rope_freq((double)cfg->rope_base);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = cfg->block_size == 16   ? write_pages<16>(a, freq, ws, st)
                        : cfg->block_size == 32 ? write_pages<32>(a, freq, ws, st)
                                                : write_pages<64>(a, freq, ws, st);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
