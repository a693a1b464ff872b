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
//  - More tokens (prompts): a first kernel lists the touched pages and notes each
//    slot's last token, and the page CTAs walk the list. In a cache of many more
//    slots than tokens the last tokens go by the page's number in the list, which
//    a second kernel finds there, so that the workspace stays small.
// A power of two as the scale makes the growth exact for every code that does
// not become subnormal, and makes the rounded values independent of the scale
// (e4m3 is a floating format), so a token's value does not depend on its
// neighbours in the page.
//
// Bound: HBM, 1,152 bytes read and 640 written per token. 262,144 tokens of 64
// sequences on one GB300: 74 us for 470 MB, 6.4 TB/s (0.94 of a copy's rate), 85 us
// with the listing before it (a kernel and a memset); a step of 64 tokens
// takes 6.1 us alone with a cold L2, 3.7 us behind another kernel.
#include <cmath>
#include <type_traits>

#include "async_copy.cuh"
#include "internal.h"
#include "page8.cuh"
#include "rope_pairs.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// One launch takes 11.7 / 21.1 us for 1,024 / 2,048 tokens of a page each, 7.1 /
// 9.9 us where 64 lie in a page; the listed form 17.0 / 25.2 and 10.4 / 10.4 us, and
// 5 us more of the host's time. At 4,096: 45.6 and 21.1 against 43.7 and 10.6.
constexpr int64_t kScanTokens = 2048;

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

// The workspace of the listed form.
struct P8WriteWs {
  size_t count, id_of, list, last, total;
};
// Last tokens by slot of the cache, not by number of the page: one kernel less,
// and the workspace is the same where the cache has fewer pages than the call has
// tokens, as here (num_blocks <= tokens / 2). Where the cache is larger its entries
// lie far apart. By slot / by page, us: 64 x 4,096 tokens in one slot a token 85.1 /
// 86.8; 2,051 in 8 slots a token 6.8 / 8.6; 8,192 in 64 10.7 / 11.6; 65,536 in 20
// 32.9 / 30.6, in 64 35.2 / 33.2.
bool by_slot(int64_t tokens, int64_t num_blocks, int bs) { return num_blocks * bs <= 8 * tokens; }
P8WriteWs write_ws(int64_t tokens, int64_t num_blocks, int bs) {
  const int64_t pages = tokens < num_blocks && !by_slot(tokens, num_blocks, bs) ? tokens : num_blocks;
  P8WriteWs L;
  L.count = 0;
  L.id_of = 256;
  L.last = align_up(L.id_of + (size_t)num_blocks * 4, 256);
  L.list = align_up(L.last + (size_t)pages * bs * 4, 256);
  L.total = align_up(L.list + (size_t)pages * 4, 256);
  return L;
}

__device__ __forceinline__ float2 unpack2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// Shared memory of a page: its tokens' latents and rope keys as given, and what
// the warps exchange.
template <int BS>
struct PageSm {
  static constexpr int x = 0;                       // [BS][512] bf16
  static constexpr int k = x + BS * kDc * 2;        // [BS][64] bf16
  static constexpr int tok = k + BS * kDr * 2;      // [2][BS] token of a row, or -1
  static constexpr int mx = tok + 2 * BS * 4;       // [8] largest magnitude of a warp
  static constexpr int bytes = mx + kWarps * 4;
};

// The frequencies in turns: inv_freq_i / (2 pi) modulo 1, in units of 2^-64. A
// position times that, modulo 2^64, is the angle for every int32 position: whole
// turns fall away in the integer product, and what the double's 53 bits leave out
// is below 2^-24 turns at 2^31.
struct PageFreq {
  uint64_t turns[32];
};
PageFreq make_page_freq(double base) {
  PageFreq f;
  for (int i = 0; i < 32; ++i) {
    const double t = std::pow(base, -2.0 * i / 64.0) * 0.15915494309189533577;  // 1 / (2 pi)
    f.turns[i] = (uint64_t)std::ldexp(t - std::floor(t), 64);
  }
  return f;
}

// cos and sin of a position's angle: its upper 32 bits in turns, split into the
// nearest quarter and a rest of [-pi/4, pi/4), then the Taylor series to r^9 and
// r^8 (remainders below 2e-9 and 3e-8), a third of the instructions of sincosf.
__device__ __forceinline__ void page_cos_sin(int pos, uint64_t turns, float* c, float* s) {
  const uint32_t a = (uint32_t)(((uint64_t)(int64_t)pos * turns) >> 32);
  const uint32_t q = (a + 0x20000000u) >> 30;
  const float r = (float)(int32_t)(a - (q << 30)) * 1.46291807926716e-9f;  // 2 pi / 2^32
  const float z = r * r;
  const float sp = fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f);
  const float cp = fmaf(z, fmaf(z, fmaf(z, 1.f / 40320.f, -1.f / 720.f), 1.f / 24.f), -0.5f);
  const float sn = fmaf(r * z, sp, r), cs = fmaf(z, cp, 1.f);
  const float u = q & 1 ? cs : sn, v = q & 1 ? sn : cs;
  *s = q & 2 ? -u : u;
  *c = (q + 1) & 2 ? -v : v;
}

// The pages of one CTA, one after another, all threads. Warp w has rows w,
// w + 8, ... of a page: all their bytes are on their way at once (cp.async); a
// row is read from shared memory for the norm and again for the codes, so that
// few registers hold many rows in flight (three CTAs an SM at 64 rows), and as
// soon as a row's codes are made its place takes the same row of the next page.
//   c_hat = (x w) r,  r = 1 / sqrt(mean(x^2) + eps)
// x w is exact in fp32 (two bf16 factors), so c_hat is one rounding away from
// r, the largest |c_hat| of a row is r times its largest |x w|, and dividing by
// the scale is a power of two folded into r. Lane l has elements 8 l ... 8 l + 7
// and 256 + those.
template <int BS>
struct PageWriter {
  using S = PageSm<BS>;
  static constexpr int kRows = BS / kWarps;
  const P8WriteArgs& a;
  uint8_t* sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t mine = 0;  // bit i: row warp + 8 i of the page in shared memory has a token
  int pos[kRows];

  // Row i of a page from its token list.
  __device__ __forceinline__ bool fetch(int i, const int* sTok, int& p) {
    const int row = warp + kWarps * i, tok = sTok[row];
    if (tok < 0) return false;
    const __nv_bfloat16* src = a.c_kv + (size_t)tok * kDc + lane * 8;
    cp_async16(sm + S::x + row * (kDc * 2) + lane * 16, src);
    cp_async16(sm + S::x + row * (kDc * 2) + 512 + lane * 16, src + kDc / 2);
    if (lane < 8) cp_async16(sm + S::k + row * (kDr * 2) + lane * 16, a.k_pe + (size_t)tok * kDr + lane * 8);
    p = a.positions[tok];
    return true;
  }
  __device__ __forceinline__ void fetch_page(const int* sTok) {
    mine = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) mine |= (uint32_t)fetch(i, sTok, pos[i]) << i;
    cp_async_commit();
  }
  __device__ __forceinline__ void load_row(int row, uint32_t (&u)[8]) const {
    const uint4 x0 = *reinterpret_cast<const uint4*>(sm + S::x + row * (kDc * 2) + lane * 16);
    const uint4 x1 = *reinterpret_cast<const uint4*>(sm + S::x + row * (kDc * 2) + 512 + lane * 16);
    u[0] = x0.x; u[1] = x0.y; u[2] = x0.z; u[3] = x0.w;
    u[4] = x1.x; u[5] = x1.y; u[6] = x1.z; u[7] = x1.w;
  }

  // Writes `page`, whose rows were fetched. nextTok: the token list of the page
  // to fetch meanwhile, complete at the barrier inside (after publish(), which
  // every thread calls before it), or NULL.
  template <typename F>
  __device__ __forceinline__ void write(const PageFreq& freq, int64_t page, const int* nextTok, F publish) {
    float* sMax = reinterpret_cast<float*>(sm + S::mx);
    const float old = a.scales[page];
    const uint4 w0 = __ldg(reinterpret_cast<const uint4*>(a.w + lane * 8));
    const uint4 w1 = __ldg(reinterpret_cast<const uint4*>(a.w + kDc / 2 + lane * 8));
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    cp_async_wait_all();
    __syncwarp();
    // (a row without a token reads what is there, and its results are dropped:
    // without branches the rows' latencies overlap)
    float r[kRows], mx[kRows], amax = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      uint32_t u[8];
      load_row(warp + kWarps * i, u);
      float2 s0 = make_float2(0.f, 0.f), s1 = s0;
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 v0 = unpack2(u[k]), v1 = unpack2(u[k + 1]);
        s0 = fma_f32x2(v0, v0, s0);
        s1 = fma_f32x2(v1, v1, s1);
        const float2 p0 = mul_f32x2(v0, unpack2(w[k])), p1 = mul_f32x2(v1, unpack2(w[k + 1]));
        m = fmaxf(m, fmaxf(fmaxf(fabsf(p0.x), fabsf(p0.y)), fmaxf(fabsf(p1.x), fabsf(p1.y))));
      }
      mx[i] = m;
      r[i] = (s0.x + s1.x) + (s0.y + s1.y);
    }
    // the rows' sums over the warp: every exchange halves the rows a lane holds,
    // so the lanes of (bits 4, 3, 2 of the lane) end with one row's sum each
#pragma unroll
    for (int h = kRows / 2, o = 16; h > 0; h >>= 1, o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int j = 0; j < h; ++j) {
        const float send = up ? r[j] : r[j + h], keep = up ? r[j + h] : r[j];
        r[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
#pragma unroll
    for (int o = 16 / kRows; o > 0; o >>= 1) r[0] += __shfl_xor_sync(0xffffffffu, r[0], o);
    // one Newton step takes the reciprocal root to about half a rounding
    const float ms = fmaf(r[0], 1.0f / kDc, a.eps), r0 = rsqrtf(ms);
    const float root = ms > 0.f && ms < INFINITY ? fmaf(r0 * 0.5f, fmaf(-ms * r0, r0, 1.f), r0) : r0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      r[i] = __shfl_sync(0xffffffffu, root, i * (32 / kRows));
      amax = fmaxf(amax, (mine >> i) & 1 ? mx[i] * r[i] : 0.f);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) sMax[warp] = amax;
    publish();
    __syncthreads();
    amax = sMax[0];
#pragma unroll
    for (int k = 1; k < kWarps; ++k) amax = fmaxf(amax, sMax[k]);
    const float scale = fmaxf(old, p8_scale_for(amax));
    if (threadIdx.x == 0 && scale != old) a.scales[page] = scale;
    const float inv = 1.0f / scale;
    const bool grew = old > 0.f && scale > old;
    const float f = grew ? old / scale : 1.f;
    const uint64_t turns = freq.turns[lane];
    const int i1 = rope_i1(a.interleaved, lane), i2 = rope_i2(a.interleaved, lane);
    uint32_t next = 0;
    // (the page whose every row is written has no branches but the copies')
    auto rows = [&](auto all) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int row = warp + kWarps * i;
        const int64_t slot = page * BS + row;
        uint8_t* dst = a.cache8 + slot * kRow8;
        const bool has = decltype(all)::value || ((mine >> i) & 1);
        uint32_t u[8];
        load_row(row, u);
        const __nv_bfloat16* kp = reinterpret_cast<const __nv_bfloat16*>(sm + S::k + row * (kDr * 2));
        const float x1 = __bfloat162float(kp[i1]), x2 = __bfloat162float(kp[i2]);
        const int p = pos[i];
        if (nextTok) {
          __syncwarp();  // every lane has the row in registers
          next |= (uint32_t)fetch(i, nextTok, pos[i]) << i;
        }
        if (!has) {
          if (grew) {
            uint4* codes = reinterpret_cast<uint4*>(dst + lane * 16);
            *codes = p8_recode16(*codes, f);
          }
          continue;
        }
        const float2 rs = make_float2(r[i] * inv, r[i] * inv);
        uint32_t q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = mul_f32x2(mul_f32x2(unpack2(u[2 * k]), unpack2(w[2 * k])), rs);
          const float2 hi = mul_f32x2(mul_f32x2(unpack2(u[2 * k + 1]), unpack2(w[2 * k + 1])), rs);
          q[k] = (uint32_t)__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3) |
                 ((uint32_t)__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3) << 16);
        }
        *reinterpret_cast<uint2*>(dst + lane * 8) = make_uint2(q[0], q[1]);
        *reinterpret_cast<uint2*>(dst + kDc / 2 + lane * 8) = make_uint2(q[2], q[3]);
        float cs, sn;
        page_cos_sin(p, turns, &cs, &sn);
        __nv_bfloat16* kr = reinterpret_cast<__nv_bfloat16*>(dst + kDc);
        kr[i1] = __float2bfloat16_rn(x1 * cs - x2 * sn);
        kr[i2] = __float2bfloat16_rn(x2 * cs + x1 * sn);
        if (a.mass && lane == 0) a.mass[slot] = 0.f;
      }
    };
    if (mine == (1u << kRows) - 1)
      rows(std::true_type{});
    else
      rows(std::false_type{});
    cp_async_commit();
    mine = next;
  }
};

template <int BS>
__global__ void __launch_bounds__(kThreads, 3) p8_write_scan_kernel(P8WriteArgs a,
                                                                    const __grid_constant__ PageFreq freq) {
  extern __shared__ __align__(16) uint8_t sm_page[];
  int* sTok = reinterpret_cast<int*>(sm_page + PageSm<BS>::tok);
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
  PageWriter<BS> pw{a, sm_page};
  pw.fetch_page(sTok);
  pw.write(freq, page, nullptr, [] {});
}

// Numbers the pages that the call's tokens touch: id_of[page] = number + 1. last:
// of each slot, or NULL.
__global__ void __launch_bounds__(kThreads) p8_number_pages_kernel(P8WriteArgs a, int bs, int* count,
                                                                   int* id_of, int* list, int* last) {
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
  if (last) atomicMax(&last[slot], t + 1);
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
__global__ void __launch_bounds__(kThreads, 3) p8_write_pages_kernel(P8WriteArgs a,
                                                                     const __grid_constant__ PageFreq freq,
                                                                     const int* count, const int* list,
                                                                     const int* last, int slot_last) {
  extern __shared__ __align__(16) uint8_t sm_page[];
  int* sTok = reinterpret_cast<int*>(sm_page + PageSm<BS>::tok);
  pdl_wait();
  pdl_launch_dependents();
  const int n = *count, r = threadIdx.x;
  int i = blockIdx.x;
  if (i >= n) return;
  // page numbers are fetched three pages ahead, token lists two, rows one
  auto tokens_of = [&](int number, int page) { return last[(size_t)(slot_last ? page : number) * BS + r] - 1; };
  int page = list[i], next_page = i + gridDim.x < n ? list[i + gridDim.x] : 0;
  if (r < BS) sTok[r] = tokens_of(i, page);
  __syncthreads();
  PageWriter<BS> pw{a, sm_page};
  pw.fetch_page(sTok);
  for (int buf = 1; i < n; i += gridDim.x, buf ^= 1) {
    const int next = i + gridDim.x;
    int next_tok = 0;
    if (next < n && r < BS) next_tok = tokens_of(next, next_page);
    const int after = next + (int)gridDim.x < n ? list[next + gridDim.x] : 0;
    pw.write(freq, page, next < n ? sTok + buf * BS : nullptr, [&] {
      if (next < n && r < BS) sTok[buf * BS + r] = next_tok;
    });
    __syncthreads();  // the maxima are read
    page = next_page;
    next_page = after;
  }
}

int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return 1;
  return sms;
}

template <int BS>
cudaError_t write_pages(const P8WriteArgs& a, const PageFreq& freq, uint8_t* ws, cudaStream_t st) {
  const int smem = PageSm<BS>::bytes;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if (a.num_tokens <= kScanTokens) {
    const cudaError_t r = cudaFuncSetAttribute(p8_write_scan_kernel<BS>, attr, smem);
    return r != cudaSuccess
               ? r
               : launch_pdl(p8_write_scan_kernel<BS>, dim3(a.num_tokens), dim3(kThreads), smem, st, a, freq);
  }
  cudaError_t e = cudaFuncSetAttribute(p8_write_pages_kernel<BS>, attr, smem);
  if (e != cudaSuccess) return e;
  const P8WriteWs L = write_ws(a.num_tokens, a.num_blocks, BS);
  int* count = reinterpret_cast<int*>(ws + L.count);
  int* id_of = reinterpret_cast<int*>(ws + L.id_of);
  int* last = reinterpret_cast<int*>(ws + L.last);
  int* list = reinterpret_cast<int*>(ws + L.list);
  const bool slot_last = by_slot(a.num_tokens, a.num_blocks, BS);
  e = cudaMemsetAsync(ws, 0, L.list, st);  // count, id_of and last
  const dim3 grid((unsigned)((a.num_tokens + kThreads - 1) / kThreads));
  if (e == cudaSuccess)
    e = launch_pdl(p8_number_pages_kernel, grid, dim3(kThreads), 0, st, a, BS, count, id_of, list,
                   slot_last ? last : nullptr);
  if (e == cudaSuccess && !slot_last)
    e = launch_pdl(p8_last_token_kernel, grid, dim3(kThreads), 0, st, a, BS, (const int*)id_of, last);
  if (e != cudaSuccess) return e;
  const int64_t pages = a.num_tokens < a.num_blocks ? a.num_tokens : a.num_blocks;
  const int64_t most = (int64_t)device_sms() * 3;  // as many CTAs as run at once
  return launch_pdl(p8_write_pages_kernel<BS>, dim3((unsigned)(pages < most ? pages : most)),
                    dim3(kThreads), smem, st, a, freq, (const int*)count, (const int*)list,
                    (const int*)last, (int)slot_last);
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
  const PageFreq freq = make_page_freq((double)cfg->rope_base);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = cfg->block_size == 16   ? write_pages<16>(a, freq, ws, st)
                        : cfg->block_size == 32 ? write_pages<32>(a, freq, ws, st)
                                                : write_pages<64>(a, freq, ws, st);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
