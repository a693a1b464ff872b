// Eviction from a paged cache by accumulated attention weight:
// mla_evict_select (which tokens of each sequence stay) and mla_page8_compact
// (their rows moved, in order, into other pages).
#include "async_copy.cuh"
#include "internal.h"
#include "page8.cuh"

namespace mla {
namespace {

// ---------------------------------------------------------------------------
// select. The middle tokens (behind the sinks, before the recent ones) are
// ranked by mass: as an unsigned key that orders like the float (NaN lowest,
// -0 = +0), a radix select finds the key T of the last token that stays, 8
// bits at a time from the top, and how many tokens of key T stay; one ordered
// pass then writes every token above T and the first ones of key T.
// One CTA per sequence.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

struct SelectArgs {
  const float* mass;
  int64_t num_blocks;
  const int32_t* block_table;
  int32_t max_blocks;
  const int32_t* seq_lens;
  int32_t block_size, sinks, recent, budget;
  int32_t* keep;
  int32_t* new_lens;
  uint32_t* status;
};

__device__ __forceinline__ uint32_t mass_key(float m) {
  if (isnan(m)) return 0u;
  const uint32_t u = __float_as_uint(m + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(SelectArgs a) {
  __shared__ int hist[256];
  __shared__ int sWarp[kSelWarps], sWarp2[kSelWarps];
  __shared__ int sPick, sNeed;
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = a.seq_lens[b], bs = a.block_size;
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;
  int32_t* keep = a.keep + (size_t)b * a.budget;
  const bool bad = len < 0 || (int64_t)len > (int64_t)a.max_blocks * bs;
  if (bad && tid == 0) set_status(a.status, MLA_DEV_BAD_SEQ);
  const int n = bad ? 0 : len;
  const int kept = min(n, a.budget);
  if (tid == 0) a.new_lens[b] = kept;
  for (int i = kept + tid; i < a.budget; i += kSelThreads) keep[i] = -1;
  if (n <= a.budget) {
    for (int i = tid; i < n; i += kSelThreads) keep[i] = i;
    return;
  }
  const int m0 = a.sinks, m1 = n - a.recent;  // the middle tokens
  auto key_of = [&](int t) {
    const int32_t p = bt[t / bs];
    if (p < 0 || p >= a.num_blocks) return 0u;
    return mass_key(a.mass[(size_t)p * bs + t % bs]);
  };
  for (int i = tid; i < (n + bs - 1) / bs; i += kSelThreads)
    if (bt[i] < 0 || bt[i] >= a.num_blocks) set_status(a.status, MLA_DEV_BAD_BLOCK);
  int need = a.budget - a.sinks - a.recent;  // middle tokens that stay
  uint32_t prefix = 0, mask = 0;
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int t = m0 + tid; t < m1; t += kSelThreads) {
        const uint32_t k = key_of(t);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255, left = need;
        while (hist[d] < left) left -= hist[d--];
        sPick = d;
        sNeed = left;
      }
      __syncthreads();
      prefix |= (uint32_t)sPick << shift;
      mask |= 255u << shift;
      need = sNeed;
    }
  }
  // `need` tokens of key `prefix` stay, the first ones
  int out = 0, ties = 0;
  for (int t0 = 0; t0 < n; t0 += kSelThreads) {
    const int t = t0 + tid;
    bool stay = t < n && (t < m0 || t >= m1), tie = false;
    if (t < n && !stay && a.budget > a.sinks + a.recent) {
      const uint32_t k = key_of(t);
      stay = k > prefix;
      tie = k == prefix;
    }
    const uint32_t tb = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) sWarp[warp] = __popc(tb);
    __syncthreads();
    int before = ties, all = 0;
    for (int k = 0; k < kSelWarps; ++k) {
      if (k < warp) before += sWarp[k];
      all += sWarp[k];
    }
    if (tie && before + __popc(tb & ((1u << lane) - 1)) < need) stay = true;
    ties += all;
    const uint32_t sb = __ballot_sync(0xffffffffu, stay);
    if (lane == 0) sWarp2[warp] = __popc(sb);
    __syncthreads();
    int at = out, total = 0;
    for (int k = 0; k < kSelWarps; ++k) {
      if (k < warp) at += sWarp2[k];
      total += sWarp2[k];
    }
    if (stay) keep[at + __popc(sb & ((1u << lane) - 1))] = t;
    out += total;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// compact. One CTA per destination page: the largest scale among the pages its
// rows come from, then one warp per row (16 bytes of codes a lane, the rope
// part by 8 lanes). Rows whose page has that scale are copied as they are;
// the others are recoded. Source and destination pages are distinct, so the
// CTAs share nothing they write.
// Bound: HBM, each kept row read once and written once.
// ---------------------------------------------------------------------------
constexpr int kCmpThreads = 256;

struct CompactArgs {
  uint8_t* cache8;
  float* scales;
  float* mass;
  int64_t num_blocks;
  const int32_t* block_table;
  int32_t max_blocks;
  const int32_t* keep;
  const int32_t* new_lens;
  int32_t budget;
  const int32_t* dst_table;
  int32_t dst_max;
  uint32_t* status;
};

template <int BS>
__global__ void __launch_bounds__(kCmpThreads) page8_compact_kernel(CompactArgs a) {
  __shared__ int64_t sSlot[BS];
  __shared__ float sScale[BS];
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, j = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.new_lens[b];
  if (n < 0 || n > a.budget || (int64_t)n > (int64_t)a.dst_max * BS) {
    if (tid == 0 && j == 0) set_status(a.status, MLA_DEV_BAD_SEQ);
    return;
  }
  if (j * BS >= n) return;
  const int rows = min(BS, n - j * BS);
  const int32_t dp = a.dst_table[(size_t)b * a.dst_max + j];
  if (dp < 0 || dp >= a.num_blocks) {
    if (tid == 0) set_status(a.status, MLA_DEV_BAD_BLOCK);
    return;
  }
  if (tid < BS) {
    int64_t slot = -1;
    float sc = 0.f;
    if (tid < rows) {
      const int t = a.keep[(size_t)b * a.budget + j * BS + tid];
      if (t < 0 || (int64_t)t >= (int64_t)a.max_blocks * BS) {
        set_status(a.status, MLA_DEV_BAD_SLOT);
      } else {
        const int32_t p = a.block_table[(size_t)b * a.max_blocks + t / BS];
        if (p < 0 || p >= a.num_blocks) {
          set_status(a.status, MLA_DEV_BAD_BLOCK);
        } else {
          slot = (int64_t)p * BS + t % BS;
          sc = a.scales[p];
        }
      }
    }
    sSlot[tid] = slot;
    sScale[tid] = sc;
  }
  __syncthreads();
  float top = 0.f;
#pragma unroll
  for (int r = 0; r < BS; ++r) top = fmaxf(top, sScale[r]);
  if (tid == 0) a.scales[dp] = top;
  for (int r = warp; r < rows; r += kCmpThreads / 32) {
    const int64_t slot = sSlot[r];
    if (slot < 0) continue;
    const uint8_t* src = a.cache8 + slot * kRow8;
    uint8_t* dst = a.cache8 + ((int64_t)dp * BS + r) * kRow8;
    uint4 c = *reinterpret_cast<const uint4*>(src + lane * 16);
    uint4 k = make_uint4(0, 0, 0, 0);
    if (lane < 8) k = *reinterpret_cast<const uint4*>(src + kDc + lane * 16);
    if (sScale[r] != top) c = p8_recode16(c, sScale[r] / top);
    *reinterpret_cast<uint4*>(dst + lane * 16) = c;
    if (lane < 8) *reinterpret_cast<uint4*>(dst + kDc + lane * 16) = k;
    if (a.mass && lane == 0) a.mass[(int64_t)dp * BS + r] = a.mass[slot];
  }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

mla_status mla_evict_select(const mla_config* cfg, const float* mass, int64_t num_blocks,
                            const int32_t* block_table, int32_t max_blocks_per_seq,
                            const int32_t* seq_lens, int32_t batch, int32_t sinks, int32_t recent,
                            int32_t budget, int32_t* keep, int32_t* new_lens,
                            uint32_t* dev_status, void* stream) {
  mla_status s = validate_config(cfg);
  if (s != MLA_OK) return s;
  if (num_blocks < 0 || max_blocks_per_seq < 0 || batch < 0 || sinks < 0 || recent < 0 ||
      budget < 1 || (int64_t)sinks + recent > budget)
    return MLA_ERR_INVALID_ARGUMENT;
  if (num_blocks > ((int64_t)1 << 31) / cfg->block_size ||
      max_blocks_per_seq > ((int64_t)1 << 30) / cfg->block_size)
    return MLA_ERR_UNSUPPORTED;
  if (batch == 0) return MLA_OK;
  if (!mass || !block_table || !seq_lens || !keep || !new_lens) return MLA_ERR_INVALID_ARGUMENT;
  if (!p8_aligned(mass, 4) || !p8_aligned(block_table, 4) || !p8_aligned(seq_lens, 4) ||
      !p8_aligned(keep, 4) || !p8_aligned(new_lens, 4) || !p8_aligned(dev_status, 4))
    return MLA_ERR_INVALID_ARGUMENT;
  const SelectArgs a{mass, num_blocks, block_table, max_blocks_per_seq, seq_lens, cfg->block_size,
                     sinks, recent, budget, keep, new_lens, dev_status};
  const cudaError_t e = launch_pdl(evict_select_kernel, dim3((unsigned)batch), dim3(kSelThreads), 0,
                                   reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

mla_status mla_page8_compact(const mla_config* cfg, void* cache8, float* page_scales, float* mass,
                             int64_t num_blocks, const int32_t* block_table,
                             int32_t max_blocks_per_seq, const int32_t* keep,
                             const int32_t* new_lens, int32_t batch, int32_t budget,
                             const int32_t* dst_block_table, int32_t dst_max_blocks,
                             uint32_t* dev_status, void* stream) {
  mla_status s = validate_config(cfg);
  if (s != MLA_OK) return s;
  if (cfg->dtype != MLA_BF16) return MLA_ERR_UNSUPPORTED;
  if (num_blocks < 0 || max_blocks_per_seq < 0 || dst_max_blocks < 0 || batch < 0 || budget < 1)
    return MLA_ERR_INVALID_ARGUMENT;
  if (num_blocks > ((int64_t)1 << 31) / cfg->block_size ||
      max_blocks_per_seq > ((int64_t)1 << 30) / cfg->block_size ||
      dst_max_blocks > ((int64_t)1 << 30) / cfg->block_size || batch > 65535)
    return MLA_ERR_UNSUPPORTED;
  if (batch == 0 || dst_max_blocks == 0) return MLA_OK;
  if (!cache8 || !page_scales || !block_table || !keep || !new_lens || !dst_block_table)
    return MLA_ERR_INVALID_ARGUMENT;
  if (!p8_aligned(cache8, 16) || !p8_aligned(page_scales, 4) || !p8_aligned(mass, 4) ||
      !p8_aligned(block_table, 4) || !p8_aligned(keep, 4) || !p8_aligned(new_lens, 4) ||
      !p8_aligned(dst_block_table, 4) || !p8_aligned(dev_status, 4))
    return MLA_ERR_INVALID_ARGUMENT;
  const CompactArgs a{(uint8_t*)cache8, page_scales, mass, num_blocks, block_table,
                      max_blocks_per_seq, keep, new_lens, budget, dst_block_table, dst_max_blocks,
                      dev_status};
  const int bs = cfg->block_size;
  const dim3 grid((unsigned)dst_max_blocks, (unsigned)batch);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      bs == 16   ? launch_pdl(page8_compact_kernel<16>, grid, dim3(kCmpThreads), 0, st, a)
      : bs == 32 ? launch_pdl(page8_compact_kernel<32>, grid, dim3(kCmpThreads), 0, st, a)
                 : launch_pdl(page8_compact_kernel<64>, grid, dim3(kCmpThreads), 0, st, a);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
