// Eviction from a paged cache by accumulated attention weight:
// mla_evict_select (which tokens of each sequence stay) and mla_page8_compact
// (their rows moved, in order, into other pages).
#include <type_traits>

#include "async_copy.cuh"
#include "cluster.cuh"
#include "internal.h"
#include "page8.cuh"

namespace mla {
namespace {

// ---------------------------------------------------------------------------
// select. The middle tokens (behind the sinks, before the recent ones) are
// ranked by mass, as an unsigned key that orders like the float (NaN lowest,
// -0 = +0). A radix select finds the key T of the last token that stays, 8 bits
// at a time from the top, and how many tokens of key T stay; then every token
// above T and the first ones of key T are written in order.
//
// A cluster of 1 to 16 CTAs takes a sequence, each CTA a contiguous piece of it,
// and each warp a contiguous piece of that, so order is a matter of prefix
// counts: over a warp's 32-token steps by ballots, over warps and CTAs by their
// totals. The keys are read once, into shared memory (kKeys a CTA; a piece
// beyond that is read again from the cache in every pass). The CTAs of a
// cluster meet once a pass: each copies its histogram to all (bulk copies counted
// on the receiver's mbarrier; a barrier of the cluster would order global memory
// too, which takes longer than the counting) and adds up what it gets.
// The second pass also lists the keys of the first digit, so that the last two
// need not go through all; and what the count of the classes found is kept for the
// writing, 2 bits a token.
// Bound: latency. One pass over 4 bytes a token, a histogram, a meeting and a scan
// for each of the four digits, and the two steps at the end: 9.0 us for 64
// sequences of 4,096 tokens on one GB300 (2 CTAs each), 18 us for 3 of up to
// 131,072 (16 each), of which reading the masses at HBM's rate would be 0.2 us.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCl = 16;                    // CTAs of a cluster
constexpr int kSms = 152;                     // of the device
constexpr int kKeys = 40 * 1024;              // keys a CTA holds
constexpr int kList = 256;                    // keys of the first digit that a warp lists
constexpr int kSelSmem = (kKeys + kSelWarps * kList) * 4;
constexpr int kSelPiece = 1024;               // tokens a CTA takes before another joins

struct SelectArgs {
  const float* mass;
  int64_t num_blocks;
  const int32_t* block_table;
  int32_t max_blocks;
  const int32_t* seq_lens;
  int32_t bs_shift, sinks, recent, budget, cluster;
  int32_t held;   // keys of a CTA in shared memory
  int32_t* keep;
  int32_t* new_lens;
  uint32_t* status;
};

__device__ __forceinline__ uint32_t mass_key(float m) {
  if (isnan(m)) return 0u;
  const uint32_t u = __float_as_uint(m + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// PER_SM: CTAs that run on an SM. With one, the registers are free for twice as
// many tokens at a time.
template <int PER_SM>
__global__ void __launch_bounds__(kSelThreads, PER_SM) evict_select_kernel(SelectArgs a) {
  constexpr int kBatch = PER_SM == 1 ? 16 : 8;
  extern __shared__ uint32_t sKey[];
  __shared__ __align__(16) int hist[2][256];    // this CTA's digits
  __shared__ __align__(16) int got[2][kMaxCl][256];  // every CTA's
  __shared__ __align__(16) int gotTotal[kMaxCl][4];
  __shared__ uint64_t bar[3];                   // of got and of gotTotal
  __shared__ __align__(16) int sTotal[4];       // tokens above T and of key T in this CTA
  __shared__ int sAbove[kSelWarps], sTies[kSelWarps];
  __shared__ int sPick, sNeed;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int CL = a.cluster, b = blockIdx.x / CL, rank = blockIdx.x % CL;
  const int len = a.seq_lens[b];
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;
  int32_t* keep = a.keep + (size_t)b * a.budget;
  const bool bad = len < 0 || (int64_t)len > ((int64_t)a.max_blocks << a.bs_shift);
  if (bad && tid == 0) set_status(a.status, MLA_DEV_BAD_SEQ);
  const int n = bad ? 0 : len, kept = min(n, a.budget);
  if (tid == 0 && rank == 0) a.new_lens[b] = kept;
  if (n <= a.budget) {  // (the whole cluster)
    for (int i = rank * kSelThreads + tid; i < a.budget; i += CL * kSelThreads) keep[i] = i < n ? i : -1;
    return;
  }
  // (every CTA's barriers are there before the first counts reach them)
  if (tid < 256) hist[0][tid] = 0;
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(&bar[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // this CTA's tokens [c0, c1); warp w's are 32 * steps of them
  const int steps = (n + CL * kSelThreads - 1) / (CL * kSelThreads);
  const int c0 = (int)min((int64_t)rank * steps * kSelThreads, (int64_t)n);
  const int c1 = (int)min((int64_t)c0 + (int64_t)steps * kSelThreads, (int64_t)n);
  const int m0 = a.sinks, m1 = n - a.recent;    // the middle tokens
  auto load_key = [&](int t) {
    const int32_t p = bt[t >> a.bs_shift];
    return p >= 0 && p < a.num_blocks
               ? mass_key(a.mass[((size_t)p << a.bs_shift) + (t & ((1 << a.bs_shift) - 1))])
               : 0u;
  };
  // U tokens of a thread at a time: their pages together, then their masses
  bool bad_page = false;
  auto load_keys = [&](int t0, auto batch) {
    constexpr int U = decltype(batch)::value;
    int32_t p[U];
    float m[U];
#pragma unroll
    for (int u = 0; u < U; ++u) p[u] = t0 + u * kSelThreads < c1 ? bt[(t0 + u * kSelThreads) >> a.bs_shift] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * kSelThreads;
      const bool fine = p[u] >= 0 && p[u] < a.num_blocks;
      bad_page |= t < c1 && !fine;
      m[u] = __int_as_float(0x7fffffff);
      if (t < c1 && fine) m[u] = a.mass[((size_t)p[u] << a.bs_shift) + (t & ((1 << a.bs_shift) - 1))];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = t0 - c0 + u * kSelThreads;
      if (t0 + u * kSelThreads < c1 && i < a.held) sKey[i] = mass_key(m[u]);
    }
  };
  for (int t0 = c0 + tid; t0 < c1;) {
    if (c1 - t0 > 2 * kSelThreads) {
      load_keys(t0, std::integral_constant<int, kBatch>{});
      t0 += kBatch * kSelThreads;
    } else {
      load_keys(t0, std::integral_constant<int, 2>{});
      t0 += 2 * kSelThreads;
    }
  }
  if (bad_page) set_status(a.status, MLA_DEV_BAD_BLOCK);
  __syncwarp();
  auto key = [&](int t) { return t - c0 < a.held ? sKey[t - c0] : load_key(t); };
  const int want = a.budget - a.sinks - a.recent;  // middle tokens that stay
  int need = want;
  uint32_t prefix = 0, mask = 0;
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  uint32_t* list = sKey + a.held + warp * kList;
  int listed = kList + 1;
  for (int pass = 0; pass < 4 && want > 0; ++pass) {
    const int shift = 24 - 8 * pass;
    auto count_digit = [&](uint32_t k, bool there) {
      const bool in = there && (k & mask) == prefix;
      const uint32_t d = in ? (k >> shift) & 255u : 256u;
      int all;
      __match_all_sync(0xffffffffu, d, &all);
      if (all) {  // a warp of equal digits counts once: equal keys do not queue up
        if (in && lane == 0) atomicAdd(&hist[pass & 1][d], 32);
      } else if (in) {
        atomicAdd(&hist[pass & 1][d], 1);
      }
      return in;
    };
    if (pass > 1 && listed <= kList) {
      for (int i = 0; i < listed; i += 32) count_digit(list[i + lane], i + lane < listed);
    } else {
      // The second pass lists the warp's keys of the first digit, which are few
      // in most distributions: if they fit, the passes after it need no others.
      if (pass == 1) listed = 0;
      const int hi = min(c1, m1);
      for (int t0 = max(c0, m0); t0 < hi; t0 += kSelThreads) {
        const int t = t0 + tid;
        const uint32_t k = t < hi ? key(t) : 0u;
        const bool in = count_digit(k, t < hi);
        if (pass == 1) {
          const uint32_t some = __ballot_sync(0xffffffffu, in);
          const int at = listed + __popc(some & ((1u << lane) - 1));
          if (in && at < kList) list[at] = k;
          listed += __popc(some);
        }
      }
    }
    if (CL > 1) fence_proxy_async_smem();
    __syncthreads();
    if (CL > 1 && warp == 0) {
      if (lane == 0) mbar_arrive_expect_tx(&bar[pass & 1], CL * (int)sizeof(hist[0]));
      __syncwarp();
      if (lane < CL) {
        cl::bulk_to_peer(cl::map(smem_u32(got[pass & 1][rank]), lane), smem_u32(hist[pass & 1]), sizeof(hist[0]),
                         cl::map(smem_u32(&bar[pass & 1]), lane));
        cl::bulk_commit();
      }
      __syncwarp();
    }
    // the cluster's count of digit 255 - tid, and of the digits above it
    int count = 0, above = 0;
    if (tid < 256) {
      if (CL > 1) {
        if (!mbar_wait(&bar[pass & 1], pass >> 1)) set_status(a.status, MLA_DEV_TIMEOUT);
#pragma unroll
        for (int r = 0; r < kMaxCl; ++r)
          if (r < CL) count += got[pass & 1][r][255 - tid];
      } else {
        count = hist[pass & 1][255 - tid];
      }
      // (its last copies have been read: every CTA has sent the counts that follow them)
      hist[(pass + 1) & 1][tid] = 0;
      above = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, above, o);
        if (lane >= o) above += u;
      }
      if (lane == 31) sAbove[warp] = above;
      above -= count;
    }
    __syncthreads();
    if (tid < 256) {
#pragma unroll
      for (int w = 0; w < 7; ++w) above += w < warp ? sAbove[w] : 0;
      if (above < need && need <= above + count) {  // (one thread)
        sPick = 255 - tid;
        sNeed = need - above;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sPick << shift;
    mask |= 255u << shift;
    need = sNeed;
  }
  // how many tokens of each warp stay for sure, and how many have key T
  const int w0 = c0 + warp * steps * 32;
  auto classify = [&](int t, bool& above, bool& tie) {
    above = t < c1 && (t < m0 || t >= m1);
    tie = false;
    if (t < c1 && !above && want > 0) {
      const uint32_t k = key(t);
      above = k > prefix;
      tie = k == prefix;
    }
  };
  // (as far as the lists' place holds it, it is not found again)
  uint2* found = reinterpret_cast<uint2*>(list);
  const int places = kList / 2;
  int above_n = 0, ties_n = 0;
  for (int s = 0; s < steps; ++s) {
    bool above, tie;
    classify(w0 + s * 32 + lane, above, tie);
    const uint32_t am = __ballot_sync(0xffffffffu, above), tm = __ballot_sync(0xffffffffu, tie);
    if (lane == 0 && s < places) found[s] = make_uint2(am, tm);
    above_n += __popc(am);
    ties_n += __popc(tm);
  }
  if (lane == 0) sAbove[warp] = above_n, sTies[warp] = ties_n;
  __syncthreads();
  int above_at = sAbove[lane], ties_at = sTies[lane];  // (kSelWarps is 32)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, above_at, o), v = __shfl_up_sync(0xffffffffu, ties_at, o);
    if (lane >= o) above_at += u, ties_at += v;
  }
  if (CL > 1 && warp == 0) {
    if (lane == 31) {
      sTotal[0] = above_at, sTotal[1] = ties_at;
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(&bar[2], CL * (int)sizeof(sTotal));
    }
    __syncwarp();
    if (lane < CL) {
      cl::bulk_to_peer(cl::map(smem_u32(gotTotal[rank]), lane), smem_u32(sTotal), sizeof(sTotal),
                       cl::map(smem_u32(&bar[2]), lane));
      cl::bulk_commit();
    }
    __syncwarp();
  }
  above_at = __shfl_sync(0xffffffffu, above_at - sAbove[lane], warp);
  ties_at = __shfl_sync(0xffffffffu, ties_at - sTies[lane], warp);
  if (CL > 1) {
    if (!mbar_wait(&bar[2], 0)) set_status(a.status, MLA_DEV_TIMEOUT);
    for (int r = 0; r < rank; ++r) above_at += gotTotal[r][0], ties_at += gotTotal[r][1];
  }
  for (int s = 0; s < steps; ++s) {
    const int t = w0 + s * 32 + lane;
    uint2 f;
    if (s < places) {
      f = found[s];
    } else {
      bool above, tie;
      classify(t, above, tie);
      f.x = __ballot_sync(0xffffffffu, above), f.y = __ballot_sync(0xffffffffu, tie);
    }
    const uint32_t am = f.x, tm = f.y;
    const bool above = am >> lane & 1, tie = tm >> lane & 1;
    const uint32_t below = (1u << lane) - 1;
    const int ties_before = ties_at + __popc(tm & below);
    const int at = above_at + __popc(am & below) + min(need, ties_before);
    // (at lies in the budget, unless a wait has run out)
    if ((above || (tie && ties_before < need)) && (uint32_t)at < (uint32_t)a.budget) keep[at] = t;
    above_at += __popc(am);
    ties_at += __popc(tm);
  }
  // What the others send has arrived; what this CTA sends has to be read.
  if (warp == 0) cl::bulk_wait_read<0>();
}

// CTAs that share a sequence of up to `tokens`: another as long as each has more
// than kSelPiece tokens and all of them run at once (clusters of 8 and 16 place
// badly beyond 96 CTAs, and 16 pay later), and up to 8 wherever the keys would
// not fit otherwise. Measured on one GB300, us with 1 / 2 / 4 / 8 / 16 CTAs (the
// choice marked):
//     1 x 3,000     10.9    8.7   *8.0    8.3
//     1 x 16,384    24.6   16.4   13.3   *9.8   10.3
//     6 x 32,768                  16.9   14.0  *11.6
//     8 x 65,536   125.4   46.1   26.5  *17.6   29.7
//    16 x 16,384    24.8   16.5  *13.3   18.7
//    64 x 2,048      7.7   *8.1   15.4   38.9
//    64 x 4,096     11.7   *9.0   16.0   39.6
//   256 x 4,096    *17.8   25.6   38.6   81.0
//     3 x 131,072  296.5  127.5   46.4   27.0  *19.0
//    64 x 131,072  315.4  137.9 *104.1  147.0
int select_cluster(int64_t tokens, int64_t batch) {
  int c = 1;
  while (c < 8 && (tokens > (int64_t)c * kKeys ||
                   (tokens > (int64_t)c * kSelPiece && batch * 2 * c <= (c == 4 ? 96 : kSms))))
    c *= 2;
  return c == 8 && tokens > 16 * kSelPiece && batch * 16 <= 96 ? 16 : c;
}

cudaError_t launch_select(SelectArgs a, int batch, cudaStream_t stream) {
  // (more CTAs than SMs: 256 x 4,096 takes 17.8 us by two an SM, 22.9 by one; fewer:
  // 3 x 131,072 28.9 and 27.0)
  auto kernel = (int64_t)batch * a.cluster > kSms ? evict_select_kernel<2> : evict_select_kernel<1>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelSmem);
  if (e == cudaSuccess && a.cluster > 8)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  // a piece of the longest sequence, in shared memory as far as it fits
  const int64_t tokens = (int64_t)a.max_blocks << a.bs_shift;
  int64_t piece = (tokens + a.cluster * kSelThreads - 1) / (a.cluster * kSelThreads) * kSelThreads;
  if (piece > kKeys) piece = kKeys;
  a.held = (int32_t)piece;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)batch * a.cluster);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (size_t)(piece + kSelWarps * kList) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// ---------------------------------------------------------------------------
// compact. One CTA per destination page: the largest scale among the pages its
// rows come from, then the rows in pieces of 16 bytes (32 of codes, 8 of rope
// values each), every thread's pieces on their way before the first is stored.
// Rows whose page has that scale are copied as they are; the others are
// recoded. Source and destination pages are distinct, so the CTAs share nothing
// they write.
// Bound: HBM, each kept row read once and written once: 29.7 us for 64 sequences
// of 2,048 kept tokens on one GB300, 169 MB at 5.7 TB/s (0.84 of a copy's rate);
// three long sequences of 8,191 in pages of 16 (32 MB) 12.2 us, by latency. Four
// CTAs an SM (64 registers a thread): 33.4 us in the step, three 36.6.
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
__global__ void __launch_bounds__(kCmpThreads, 4) page8_compact_kernel(CompactArgs a) {
  __shared__ int64_t sSlot[BS];
  __shared__ float sScale[BS];
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, j = blockIdx.x, tid = threadIdx.x;
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
  constexpr int kPieces = kRow8 / 16, kPer = (BS * kPieces + kCmpThreads - 1) / kCmpThreads;  // pieces of a row, of a thread
  uint4 c[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = tid + u * kCmpThreads, r = i / kPieces;
    if (r < rows && sSlot[r] >= 0)
      c[u] = __ldcs(reinterpret_cast<const uint4*>(a.cache8 + sSlot[r] * kRow8) + i % kPieces);
  }
  float m = 0.f;
  const bool with_mass = a.mass && tid < rows && sSlot[tid] >= 0;
  if (with_mass) m = a.mass[sSlot[tid]];
  uint4* dst = reinterpret_cast<uint4*>(a.cache8 + (int64_t)dp * BS * kRow8);
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = tid + u * kCmpThreads, r = i / kPieces;
    if (r >= rows || sSlot[r] < 0) continue;
    if (i % kPieces < kDc / 16 && sScale[r] != top) c[u] = p8_recode16(c[u], sScale[r] / top);
    dst[i] = c[u];
  }
  if (with_mass) a.mass[(int64_t)dp * BS + tid] = m;
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
      max_blocks_per_seq > ((int64_t)1 << 30) / cfg->block_size || batch > (1 << 27))
    return MLA_ERR_UNSUPPORTED;
  if (batch == 0) return MLA_OK;
  if (!mass || !block_table || !seq_lens || !keep || !new_lens) return MLA_ERR_INVALID_ARGUMENT;
  if (!p8_aligned(mass, 4) || !p8_aligned(block_table, 4) || !p8_aligned(seq_lens, 4) ||
      !p8_aligned(keep, 4) || !p8_aligned(new_lens, 4) || !p8_aligned(dev_status, 4))
    return MLA_ERR_INVALID_ARGUMENT;
  const int shift = cfg->block_size == 16 ? 4 : cfg->block_size == 32 ? 5 : 6;
  const SelectArgs a{mass, num_blocks, block_table, max_blocks_per_seq, seq_lens, shift, sinks,
                     recent, budget, select_cluster((int64_t)max_blocks_per_seq << shift, batch), 0, keep,
                     new_lens, dev_status};
  const cudaError_t e = launch_select(a, batch, reinterpret_cast<cudaStream_t>(stream));
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
  if (batch == 0) return MLA_OK;
  if (!cache8 || !page_scales || !block_table || !keep || !new_lens || (!dst_block_table && dst_max_blocks > 0))
    return MLA_ERR_INVALID_ARGUMENT;
  if (!p8_aligned(cache8, 16) || !p8_aligned(page_scales, 4) || !p8_aligned(mass, 4) ||
      !p8_aligned(block_table, 4) || !p8_aligned(keep, 4) || !p8_aligned(new_lens, 4) ||
      !p8_aligned(dst_block_table, 4) || !p8_aligned(dev_status, 4))
    return MLA_ERR_INVALID_ARGUMENT;
  const CompactArgs a{(uint8_t*)cache8, page_scales, mass, num_blocks, block_table,
                      max_blocks_per_seq, keep, new_lens, budget, dst_block_table, dst_max_blocks,
                      dev_status};
  const int bs = cfg->block_size;
  // (without destination pages, to flag the sequences that have tokens)
  const dim3 grid((unsigned)(dst_max_blocks > 0 ? dst_max_blocks : 1), (unsigned)batch);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      bs == 16   ? launch_pdl(page8_compact_kernel<16>, grid, dim3(kCmpThreads), 0, st, a)
      : bs == 32 ? launch_pdl(page8_compact_kernel<32>, grid, dim3(kCmpThreads), 0, st, a)
                 : launch_pdl(page8_compact_kernel<64>, grid, dim3(kCmpThreads), 0, st, a);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
