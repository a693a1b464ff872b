// mla_tree_decode: split-KV latent attention of the rows of drafted trees over
// the paged bf16 cache (the merge of the splits and the projection: tree_merge.cu).
//
// Row n of sequence b sees every token t < past = seq_lens[b] - q_len, and of
// the tree's own tokens past + j those whose bit j its mask has:
//   s_t = softmax_scale * log2(e) * (q_abs[n,h] . row_t)        (base 2)
//   out[n,h] = (sum_t 2^(s_t - m) c_t / sum_t 2^(s_t - m)) W_uv[h]
//
// The (row, head) pairs of a sequence are cut into q-blocks of 128, which are
// the M of the tensor-core products; work units are (q-block, 64-token tile).
// The units are cut into equal contiguous shares, one to a cluster of two CTAs.
// Where a sequence has several q-blocks its tokens are taken in strips as long
// as a share, and the q-blocks follow one another within a strip: neighbouring
// clusters then read the same tokens at the same time, which come from HBM once.
// CTA h of a pair owns latent columns [256 h, 256 h + 256) of the cache, and half
// of the rope columns, [512 + 32 h, 512 + 32 h + 32):
//   S_h = Q[:, cols_h] K[:, cols_h]^T    (partial scores, in TMEM, fp32)
//   S   = S_h + the peer's partial       (sent as f16 into this CTA's shared memory)
//   O_h += P V[:, cols_h]                (this CTA's half of the output)
// so every byte of a cache row goes to one shared memory only.
//
// Each CTA takes the softmax of its own sums: its own part is fp32 and the
// peer's rounded to f16 (11 bits, saturating), so the two CTAs' weights differ
// by that rounding, each half of the output is divided by the sum of its own
// weights, and the merge weighs each half by its own log-sum-exp. The weights
// are rounded to bf16 for the product (V is bf16, and the tensor cores take one
// type); the sum adds the rounded weights, so that a row with one large weight
// loses nothing. The f16 half moves a weight by 2^-11 of that half (in units of the
// exponent), the bf16 rounding by 2^-8: beyond halves of 8 the exchange is what
// costs accuracy. fp32 would be twice the exchange, which takes 1,000 cycles of a
// tile's 1,900 for 16 KB, and 32 KB more of shared memory, of which 9 are free.
//
// TMEM (512 columns): O [0, 256), two score buffers of 64 columns, and the
// query's 256 latent columns (bf16 pairs) [384, 512). Its 32 rope columns lie in
// shared memory, with four stages of 64 tokens, two buffers of the peer's scores
// and two of weights.
// Per CTA (384 threads):
//   warp 0      walks the share, lays its segments out for the others, and copies a
//               segment's query and its cache stages into the ring (TMA, SWIZZLE_128B;
//               rope SWIZZLE_64B); block ids are checked
//   warp 1      issues O += P V of a tile; owns the TMEM
//   warp 2      issues the scores of a tile, up to two tiles ahead of its weights
//   warp 3      waits for all that a tile's softmax needs and says so in one word
//               (a poll of an mbarrier takes some 125 cycles, ready or not; the
//               softmax would spend a fifth of its time on four of them a tile)
//   warps 4-7   softmax, a thread a row
//   warps 8-11  send the partial scores to the peer, and move the next segment's
//               query from the ring to TMEM once the last scores are there
//   At a segment's end warps 4-11 write its normalised rows, half of the columns
//   each, and its log-sum-exps: rows whose tokens are all in the segment to their
//   place among the latents, others to a part's slot.
//
// What bounds it: not a rate. 64 sequences of 4,096 tokens take 75 us alone (in graphs;
// 4.0 TB/s of HBM, tensor pipe busy 0.40), 16 sequences of 61 rows over up to 8,000
// tokens 165 (0.46). A tile takes 1,900 cycles on the average, of which its products need 1,140:
// from the copy of a stage to its release are 7,400 cycles (copy 2,700, scores 800,
// exchange 1,300, softmax 1,400, output 850) over four stages, which with the peer's
// scores and the weights fill the shared memory. 32-token tiles in ten stages took 6 to
// 14 % longer, scores exchanged in halves and copies into the L2 ahead of the ring no
// less. A share starts with some 12,000 cycles up to its first weights and a segment
// ends with 10,000, most of them fetches of code that is not in the caches: what is
// done once a segment, and what is done when a wait takes long, is out of line.
// Every wait is bounded; on a timeout the roles leave their loops, the issuers
// wait for their products and the copies' warp for its copies before TMEM is
// freed, and the pair meets at a last barrier.
#include "async_copy.cuh"
#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"
#include "pair_math.cuh"
#include "tcgen05.cuh"
#include "tree_parts.cuh"

namespace mla {
namespace {

constexpr int kBlockRows = kTreeBlockRows, kTok = kTreeTok;
constexpr int kSlab = kTok * 128;              // 64 rows of 64 bf16 columns
constexpr int kRope = kTok * 64;               // 64 rows of 32 rope columns
constexpr int kStage = 4 * kSlab + kRope;      // 36 KB
constexpr int kStages = 4;
constexpr int kXBytes = kBlockRows * kTok * 2; // 16 KB: [8 chunks][128 rows][16 bytes]
constexpr int kPBytes = kBlockRows * 128;      // 16 KB: weights, SWIZZLE_128B
constexpr int kThreads = 384;
constexpr int kSoftWarp0 = 4, kSendWarp0 = 8;
constexpr uint32_t kOCol = 0, kSCol = 256, kQCol = 384, kTmemCols = 512;
constexpr float kRescaleLog2 = 8.f;
constexpr int kTreeMaxRows = 48 * 1024;

enum {
  kFull0 = 0,
  kEmpty0 = kFull0 + kStages,
  kSFull0 = kEmpty0 + kStages,   // [2] partial scores of tile i in S[i % 2]
  kSRead0 = kSFull0 + 2,         // [2] S[i % 2] read (8 warps)
  kPFull0 = kSRead0 + 2,         // [2] weights of tile i in P[i % 2] (4 warps)
  kPVDone0 = kPFull0 + 2,        // [2] O += P V of tile i done
  kXFull0 = kPVDone0 + 2,        // [2] the peer's scores of tile i (bytes from the peer)
  kPeerFree0 = kXFull0 + 2,      // [2] the peer has read its buffer (4 warps of the peer)
  kQRead0 = kPeerFree0 + 2,      // [QuerySlots::kBars] the stage with half of a query read (4 warps)
  kQReady = kQRead0 + QuerySlots::kBars,         // query columns in place (4 warps)
  kSums,                         // the segment's weight sums in shared memory (4 warps)
  kODone,                        // every output product of the segment done
  kOFree,                        // O read out, staging free (8 warps)
  kFinalS,
  kFinalP,
  kNumBars
};

// A stage: per page its 4 column slabs of block_size rows (128 bytes of a row, 64
// columns), then the rope columns of the 64 rows. Byte offset of token t's row in
// its page's first slab, without the swizzle:
__device__ __forceinline__ int token_at(int t, int bs_shift) {
  return ((t >> bs_shift) << (bs_shift + 9)) + (t & ((1 << bs_shift) - 1)) * 128;
}

struct Smem {
  static constexpr int stage = 0;
  static constexpr int x = stage + kStages * kStage;
  static constexpr int p = x + 2 * kXBytes;
  static constexpr int rope = p + 2 * kPBytes;            // [128 rows][32 columns], SWIZZLE_64B
  static constexpr int sum = rope + kBlockRows * 64;      // [128] 1 / weight sum
  static constexpr int info = sum + kBlockRows * 4;   // [kStages] int2
  static constexpr int bars = info + kStages * 8;
  static constexpr int misc = bars + kNumBars * 8;        // tmem base, abort flag, tiles ready, segments laid out
  static constexpr int plan = (misc + 16 + 15) / 16 * 16;  // ShareStart
  static constexpr int segs = (plan + 32 + 12 * (kThreads / 32) + 15) / 16 * 16;   // [4] TreeSeg
  static constexpr int bytes = segs + 4 * 48;
  static constexpr int alloc = bytes + 1024;
};
static_assert(Smem::alloc <= 227 * 1024, "shared memory budget");
static_assert(Smem::bars % 8 == 0 && Smem::stage % 1024 == 0 && kStage % 1024 == 0 && Smem::p % 1024 == 0 &&
                  Smem::rope % 1024 == 0,
              "alignment");

struct TreeSeq {
  int q0, ql, len, n, m;   // rows [q0, q0 + ql); n tiles, m q-blocks (0: nothing to do)
  bool broken;             // query_start_loc does not ascend here, or leaves [0, num_q]
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, bool report) {
  TreeSeq s;
  s.q0 = a.query_start_loc[b];
  const int q1 = a.query_start_loc[b + 1];
  s.ql = q1 - s.q0;
  s.len = a.seq_lens[b];
  s.n = s.m = 0;
  const bool rows_ok = s.q0 >= 0 && q1 <= a.num_q && q1 >= s.q0;
  s.broken = !rows_ok;
  const bool ok = rows_ok && s.ql <= s.len && s.ql <= 64 * a.words &&
                  (int64_t)s.len <= (int64_t)a.max_blocks * a.block_size;
  if (report && !ok) set_status(a.status, MLA_DEV_BAD_SEQ);
  if (ok && s.ql > 0) {
    s.n = (s.len + kTok - 1) / kTok;
    s.m = (s.ql * a.num_heads + kBlockRows - 1) / kBlockRows;
  }
  return s;
}
struct alignas(16) TreeSeg {
  int b, j, k0, k1, item, q0, ql, len, more;   // more: another one follows
};

// Walks the units of one share.
struct TreeWalk {
  int u, u_end, share, b, ubase, ibase;
  TreeSeq s;

  __device__ __forceinline__ bool next(const TreeArgs& a, TreeSeg& g) {
    if (u >= u_end) return false;
#pragma unroll 1
    while (u >= ubase + s.n * s.m) {
      ubase += s.n * s.m;
      ibase += s.m * tree_strips(s.n, s.m, share);
      s = tree_seq(a, ++b, false);
    }
    const int off = u - ubase;
    g.b = b;
    g.q0 = s.q0;
    g.ql = s.ql;
    g.len = s.len;
    if (s.m == 1) {
      g.j = 0;
      g.k0 = off;
      g.k1 = min(s.n, off + u_end - u);
      g.item = ibase;
    } else {
      const TreeUnit at = tree_unit(off, s.n, s.m, share);
      g.j = at.j;
      g.k0 = at.strip * share + at.k;
      g.k1 = g.k0 + min(at.tiles - at.k, u_end - u);
      g.item = ibase + at.strip * s.m + at.j;
    }
    u += g.k1 - g.k0;
    g.more = u < u_end;
    return true;
  }
};

// Of the CTA's threads before this one, the sum of v; and of all.
__device__ __noinline__ int2 block_scan(int2 v, int2* scratch, int tid, int2& all) {
  const int lane = tid & 31, warp = tid >> 5;
  int2 sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, sum.x, o), y = __shfl_up_sync(0xffffffffu, sum.y, o);
    if (lane >= o) sum.x += x, sum.y += y;
  }
  if (lane == 31) scratch[warp] = sum;
  __syncthreads();
  sum.x -= v.x;
  sum.y -= v.y;
  all = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int2 x = scratch[w];
    if (w < warp) sum.x += x.x, sum.y += x.y;
    all.x += x.x;
    all.y += x.y;
  }
  return sum;
}

// The split: where share c begins. Every CTA finds it, a thread a sequence (of more
// than the threads, in rounds); the first writes the plan that the merge follows.
struct ShareStart {
  int b, ubase, ibase, q0, ql, len, n, m;
  int sums[kThreads / 32];
  int2 scan[kThreads / 32];
};
__device__ __forceinline__ bool find_share(const TreeArgs& a, int c, ShareStart* st, int tid, TreeWalk& w) {
  const bool first = blockIdx.x == 0;
  TreeSeq s{};
  int sum = 0;
  bool broken = false;
#pragma unroll 1
  for (int b = tid; b < a.batch; b += kThreads) {
    s = tree_seq(a, b, first);
    sum += s.n * s.m;
    broken |= s.broken;
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  if ((tid & 31) == 0) st->sums[tid >> 5] = sum;
  // (rows that two sequences have would not fit the workspace: nothing is done)
  if (__syncthreads_or(broken)) {
    if (first)
      for (int b = tid; b < a.batch; b += kThreads) a.plan[b] = make_int4(0, 0, 0, 0);
    return false;
  }
  int total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) total += st->sums[i];
  const int share = max(1, (total + a.shares - 1) / a.shares);
  const int u0 = (int)min((int64_t)c * share, (int64_t)total);
  int2 base = make_int2(0, 0);
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    if (a.batch > kThreads) {
      s.n = s.m = 0;
      if (b < a.batch) s = tree_seq(a, b, false);
      __syncthreads();         // (the last round's scan is read)
    }
    const int units = s.n * s.m;
    int2 all;
    const int2 at = block_scan(make_int2(units, s.m * tree_strips(s.n, s.m, share)), st->scan, tid, all);
    const int ubase = base.x + at.x, ibase = base.y + at.y;
    if (first && b < a.batch) a.plan[b] = make_int4(ubase, ibase, s.n, s.m);
    if (u0 >= ubase && u0 < ubase + units) {
      st->b = b;
      st->ubase = ubase;
      st->ibase = ibase;
      st->q0 = s.q0;
      st->ql = s.ql;
      st->len = s.len;
      st->n = s.n;
      st->m = s.m;
    }
    base.x += all.x;
    base.y += all.y;
  }
  if (first && tid == 0) {
    WsHeader* hdr = reinterpret_cast<WsHeader*>(a.ws);
    hdr->total_units = total;
    hdr->share = share;
  }
  __syncthreads();
  w.u = u0;
  w.u_end = min(u0 + share, total);
  w.share = share;
  if (w.u >= w.u_end) return false;
  w.b = st->b;
  w.ubase = st->ubase;
  w.ibase = st->ibase;
  w.s.q0 = st->q0;
  w.s.ql = st->ql;
  w.s.len = st->len;
  w.s.n = st->n;
  w.s.m = st->m;
  return true;
}

__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 15u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitTimeoutNs) return false;
    }
  }
}
// By whole warps: try_wait suspends a converged warp until the phase completes and
// wakes it within 82 cycles; with one lane polling for the others it took 190.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || mbar_try_wait(bar, parity) || mbar_try_wait(bar, parity) ||
         wait_long(bar, parity, abort_flag);
}

// Waits until *word > i; false on a timeout or another role's.
__device__ __forceinline__ bool word_passed(const int* word, int i) {
  int x;
  asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(x) : "r"(smem_u32(word)) : "memory");
  return x > i;
}
__device__ __noinline__ bool word_long(const int* word, int i, volatile int* abort_flag) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t n = 1;; ++n) {
    if (word_passed(word, i)) return true;
    if ((n & 63u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitTimeoutNs) return false;
    }
  }
}
__device__ __forceinline__ bool wait_word(const int* word, int i, volatile int* abort_flag) {
  return word_passed(word, i) || word_long(word, i, abort_flag);
}

// Two scores as an f16 pair, saturating; an infinite one is passed on as NaN
// (saturated, it would be a large one).
__device__ __forceinline__ uint32_t pack_score(uint32_t lo, uint32_t hi) {
  const float2 x = make_float2(__uint_as_float(lo), __uint_as_float(hi));
  const float2 y = fma_f32x2(x, make_float2(0.f, 0.f), x);
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y.y), "f"(y.x));
  return r;
}
// lo += the pair's low f16, hi += its high one, in fp32.
__device__ __forceinline__ void add_f16x2(uint32_t pair, float& lo, float& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "add.rn.f32.f16 %0, l, %0;\n\tadd.rn.f32.f16 %1, h, %1;\n\t}"
      : "+f"(lo), "+f"(hi)
      : "r"(pair));
}
__device__ __forceinline__ void add_bf16x2(uint32_t pair, float& lo, float& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "add.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
      : "+f"(lo), "+f"(hi)
      : "r"(pair));
}
// 16 bytes into the peer's shared memory, counted on its barrier.
__device__ __forceinline__ void send16(uint32_t dst, uint32_t bar, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(dst),
      "r"(bar), "r"(a), "r"(b), "r"(c), "r"(d)
      : "memory");
}
// Uses of loaded registers stay behind the wait for the loads.
__device__ __forceinline__ void loaded(uint32_t (&r)[32]) {
#pragma unroll
  for (int k = 0; k < 32; k += 16)
    asm volatile("" : "+r"(r[k]), "+r"(r[k + 1]), "+r"(r[k + 2]), "+r"(r[k + 3]), "+r"(r[k + 4]), "+r"(r[k + 5]),
                 "+r"(r[k + 6]), "+r"(r[k + 7]), "+r"(r[k + 8]), "+r"(r[k + 9]), "+r"(r[k + 10]), "+r"(r[k + 11]),
                 "+r"(r[k + 12]), "+r"(r[k + 13]), "+r"(r[k + 14]), "+r"(r[k + 15]));
}

// A warp's 32 rows of two of the query's column slabs (128 columns) from a stage
// that holds them, [2 slabs][128 rows][128 bytes], into TMEM, and of 64 rows' rope
// columns into their place; the sign of a scale that is not positive goes with them.
__device__ __noinline__ void take_query(const uint8_t* stage, int part, int r, uint32_t tcols, uint8_t* rope_rows,
                                        float scale) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t w[16];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint4 y = *reinterpret_cast<const uint4*>(stage + (c >> 1) * (kBlockRows * 128) + sw128(r, 4 * (c & 1) + u));
      w[4 * u] = signed_query(y.x, scale);
      w[4 * u + 1] = signed_query(y.y, scale);
      w[4 * u + 2] = signed_query(y.z, scale);
      w[4 * u + 3] = signed_query(y.w, scale);
    }
    tc::st16(tcols + 64 * part + 16 * c, w);
  }
  if (r >> 6 == part) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint4 y = *reinterpret_cast<const uint4*>(stage + 4 * kSlab + (r & 63) * 64 + 16 * u);
      *reinterpret_cast<uint4*>(rope_rows + r * 64 + 16 * u) =
          make_uint4(signed_query(y.x, scale), signed_query(y.y, scale), signed_query(y.z, scale), signed_query(y.w, scale));
    }
  }
  fence_proxy_async_smem();
  tc::wait_st();
  tc::fence_before_sync();
  __syncwarp();
}

// Where a segment's rows go: to the merged latents if it has all tokens of its
// q-block (the merge passes such rows over), to its part's slot if not.
__device__ __forceinline__ float* part_rows(const TreeArgs& a, const TreeSeg& g, int share_idx) {
  return g.k0 == 0 && g.k1 * kTok >= g.len
             ? a.o_lat + ((size_t)g.q0 * a.num_heads + (size_t)g.j * kBlockRows) * kDc
             : a.opart + ((size_t)share_idx + g.item) * kBlockRows * kDc;
}

// The normalised columns [128 part, 128 part + 128) of this CTA's half of a
// segment's O, 32 rows, to `dst`, by whole 128-byte lines through `stage` (4 KB).
__device__ __noinline__ void store_rows(uint32_t trow, int part, float inv, int rows, float* dst, uint8_t* stage, int lane) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t o[32];
    tc::ld32(trow + kOCol + 128 * part + 32 * c, o);
    tc::wait_ld();
    loaded(o);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<float4*>(stage + sw128(lane, k)) =
          make_float4(__uint_as_float(o[4 * k]) * inv, __uint_as_float(o[4 * k + 1]) * inv,
                      __uint_as_float(o[4 * k + 2]) * inv, __uint_as_float(o[4 * k + 3]) * inv);
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int r = 4 * u + (lane >> 3);
      const float4 y = *reinterpret_cast<const float4*>(stage + sw128(r, lane & 7));
      if (r < rows) *reinterpret_cast<float4*>(dst + (size_t)r * kDc + 128 * part + 32 * c + 4 * (lane & 7)) = y;
    }
  }
  tc::fence_before_sync();
}

// Rows of a stage that are not there may hold anything: zero, so that a weight of
// 0 stays 0. So do the tree's tokens that are not finite, for the rows that do
// not see them. Two slabs (128 columns) of row `row`.
__device__ __noinline__ void clean_stage(uint8_t* stg, int slab_bytes, int row, bool there, bool of_tree) {
  bool zero = !there;
  if (there && of_tree) {
    uint32_t most = 0;   // the largest exponent and fraction of the low and of the high values
#pragma unroll 4
    for (int c = 0; c < 16; ++c) {
      const uint4 y = *reinterpret_cast<const uint4*>(stg + (c >> 3) * slab_bytes + sw128(row, c & 7));
      most = __vmaxu2(__vmaxu2(most, y.x & 0x7fff7fffu), __vmaxu2(y.y & 0x7fff7fffu, __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu)));
    }
    zero = (most & 0xffffu) >= 0x7f80u || (most >> 16) >= 0x7f80u;
  }
  if (zero) {
#pragma unroll 4
    for (int c = 0; c < 16; ++c)
      *reinterpret_cast<uint4*>(stg + (c >> 3) * slab_bytes + sw128(row, c & 7)) = make_uint4(0, 0, 0, 0);
  }
}

// Bit i: row `j0 + i` of the tree is in the mask (words of 64, `words` of them).
__device__ __noinline__ uint64_t mask_from(const uint64_t* m, int words, int j0) {
  const int w = j0 >> 6, sh = j0 & 63;
  uint64_t x = w < words ? __ldg(m + w) >> sh : 0;
  if (sh && w + 1 < words) x |= __ldg(m + w + 1) << (64 - sh);
  return x;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    tree_decode_kernel(const __grid_constant__ CUtensorMap slab4, const __grid_constant__ CUtensorMap rope_map, const __grid_constant__ CUtensorMap q_map,
                       const __grid_constant__ CUtensorMap qrope_map, const __grid_constant__ TreeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Smem::bars);
  int2* info = reinterpret_cast<int2*>(sm + Smem::info);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Smem::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Smem::misc + 4);
  int* ready = reinterpret_cast<int*>(sm + Smem::misc + 8);   // tiles whose softmax may begin
  int* segments = ready + 1;                                  // segments laid out in `list`
  TreeSeg* list = reinterpret_cast<TreeSeg*>(sm + Smem::segs);
  uint8_t* sStage = sm + Smem::stage;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = (int)cl::rank();
  const int share_idx = blockIdx.x >> 1;
  const int bs = a.block_size, bs_shift = bs == 16 ? 4 : bs == 32 ? 5 : 6;
  const int pages = kTok / bs;                      // of a stage
  const int full_mask = (1 << pages) - 1;

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool eight = i == kSRead0 || i == kSRead0 + 1 || i == kOFree;
      const bool four = (i >= kPFull0 && i < kPVDone0) || (i >= kPeerFree0 && i <= kSums);
      mbar_init(&bars[i], eight ? 8 : four ? 4 : 1);
    }
    for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&bars[kXFull0 + i], kXBytes);
    *abort_flag = 0;
    *ready = 0;
    *segments = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc::alloc(tmem_slot, kTmemCols);
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&slab4);
    prefetch_tensormap(&rope_map);
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&qrope_map);
  }
  tc::fence_before_sync();
  cl::sync();  // both CTAs' barriers exist before either sends
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  TreeWalk sw;
  const bool has_work = find_share(a, share_idx, reinterpret_cast<ShareStart*>(sm + Smem::plan), tid, sw);
  TreeSeg seg;
  auto warp_wait = [&](int bar, uint32_t parity) {
    const bool ok = wait_or_abort(&bars[bar], parity, abort_flag);   // (the same for all lanes)
    __syncwarp();
    return ok;
  };
  // The copies' warp walks the share and lays its segments out for the others, some 50
  // cycles a read; each walking by itself, with its state in local memory behind the
  // stores of the last segment's rows, took 6,000 cycles a segment. A list of four does:
  // a segment has three stages of the ring or more, so when the copies come to segment
  // s + 3, the last tile of s has been through every role, and s - 1 is not read again.
  auto segment = [&](int i) {
    if (!__all_sync(0xffffffffu, wait_word(segments, i, abort_flag))) return false;
    seg = list[i & 3];
    return true;
  };
  auto fail_out = [&]() {
    set_status(a.status, MLA_DEV_TIMEOUT);
    *abort_flag = 1;
  };

  if (has_work && warp == 0) {
    // ------------------------------------------------------------ copies
    // The ring takes a segment's query in two stages (128 latent columns each, and
    // 64 rows' rope columns), then its tiles.
    const uint64_t policy = l2_evict_first_policy();
    const bool leader = tc::elect_one();
    int ri = 0;                                   // stages filled so far
    QuerySlots queries;
    uint32_t phase = 0;                           // per slot: the parity of its next Empty
    int seg_i = 0;
    bool ok = true;
    auto room = [&](int slot) {
      if (ri < kStages) return true;
      if (queries.held(slot)) return warp_wait(kQRead0 + queries.bar(slot), queries.parity(slot));
      const bool free = warp_wait(kEmpty0 + slot, (phase >> slot) & 1);
      phase ^= 1u << slot;
      return free;
    };
    while (ok && sw.next(a, seg)) {
      if (leader) {
        list[seg_i & 3] = seg;
        asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(smem_u32(segments)), "r"(seg_i + 1) : "memory");
      }
      __syncwarp();
      const int32_t* bt = a.block_table + (size_t)seg.b * a.max_blocks;
      for (int part = 0; part < 2 && ok; ++part, ++ri) {
        const int slot = ri % kStages;
        if (!room(slot)) { ok = false; break; }
        queries.put(slot, seg_i, part);
        if (leader) {
          uint64_t* full = &bars[kFull0 + slot];
          uint8_t* dst = sStage + slot * kStage;
          const int row = seg.q0 * a.num_heads + seg.j * kBlockRows;
          mbar_arrive_expect_tx(full, kStage);
          tma_load_2d(dst, &q_map, 256 * h + 128 * part, row, full);
          tma_load_2d(dst + kBlockRows * 128, &q_map, 256 * h + 128 * part + 64, row, full);
          tma_load_2d(dst + 4 * kSlab, &qrope_map, kDc + 32 * h, row + 64 * part, full);
        }
        __syncwarp();
      }
      ++seg_i;
      int cache_base = -(1 << 30), cached = -1;   // lane l holds bt[cache_base + l]
#pragma unroll 1
      for (int k = seg.k0; k < seg.k1 && ok; ++k, ++ri) {
        const int tstart = k * kTok, v = min(kTok, seg.len - tstart), slot = ri % kStages;
        const int p0 = tstart >> bs_shift;
        if (p0 < cache_base || p0 + pages > cache_base + 32) {
          cache_base = p0;
          cached = p0 + lane < a.max_blocks ? bt[p0 + lane] : -1;
        }
        const bool wanted = lane < pages && (lane << bs_shift) < v;     // lane l: page l of the stage
        const int blk = __shfl_sync(0xffffffffu, cached, min(p0 - cache_base + lane, 31));
        const bool there = wanted && blk >= 0 && blk < a.num_blocks;
        if (wanted && !there) set_status(a.status, MLA_DEV_BAD_BLOCK);
        const uint32_t okmask = __ballot_sync(0xffffffffu, there);
        if (!room(slot)) { ok = false; break; }
        queries.clear(slot);
        uint8_t* dst = sStage + slot * kStage;
        if (leader) {
          info[slot] = make_int2(v, (int)okmask);
          mbar_arrive_expect_tx(&bars[kFull0 + slot], __popc(okmask) * bs * (4 * 128 + 64));
        }
        __syncwarp();
#pragma unroll 1
        for (int p = 0; p < pages; ++p) {
          const int y = __shfl_sync(0xffffffffu, blk, p) << bs_shift;
          if (leader && ((okmask >> p) & 1)) {
            tma_load_3d_hint(dst + (p << bs_shift) * 512, &slab4, 0, y, 4 * h, &bars[kFull0 + slot], policy);
            tma_load_2d_hint(dst + 4 * kSlab + (p << bs_shift) * 64, &rope_map, kDc + 32 * h, y, &bars[kFull0 + slot],
                             policy);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      if (!ok) fail_out();
      for (int slot = 0; slot < kStages; ++slot) {   // never leave with copies in flight
        const int fills = ri > slot ? (ri - 1 - slot) / kStages + 1 : 0;
        if (fills > 0 && !mbar_wait(&bars[kFull0 + slot], (fills - 1) & 1)) set_status(a.status, MLA_DEV_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (has_work && warp == 1) {
    // ---------------------------------------------------- output products
    constexpr uint32_t kIdO = tc::idesc_bf16(128, 256, false, true);
    const uint64_t vdesc = tc::smem_desc(smem_u32(sStage), (uint32_t)bs * 128, 1024, tc::kSwizzle128);
    const uint64_t pdesc = tc::smem_desc(smem_u32(sm + Smem::p), 16, 1024, tc::kSwizzle128);
    const bool leader = tc::elect_one();
    int i = 0, ri = 0, seg_i = 0;
    bool ok = true, more = true;
    while (more) {
      if (!(ok = segment(seg_i))) break;
      more = seg.more;
      const int n = seg.k1 - seg.k0;
      ri += 2;
#pragma unroll 1
      for (int t = 0; t < n; ++t, ++i, ++ri) {
        const int slot = ri % kStages, b = i & 1;
        if (!warp_wait(kPFull0 + b, (i >> 1) & 1)) { ok = false; break; }
        if (t == 0 && seg_i > 0 && !warp_wait(kOFree, (seg_i - 1) & 1)) { ok = false; break; }
        tc::fence_after_sync();
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < kTok / 16; ++ks)
            tc::mma_bf16(tmem + kOCol, pdesc + (uint64_t)((b * kPBytes + ks * 32) >> 4),
                         vdesc + (uint64_t)((slot * kStage + token_at(ks * 16, bs_shift)) >> 4), kIdO, t > 0 || ks > 0);
          tc::commit(&bars[kEmpty0 + slot]);
          tc::commit(&bars[kPVDone0 + b]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (leader) tc::commit(&bars[kODone]);
      __syncwarp();
      ++seg_i;
    }
    if (!ok && leader) fail_out();
    if (leader) tc::commit(&bars[kFinalP]);
    __syncwarp();
    if (!mbar_wait(&bars[kFinalP], 0) && leader) set_status(a.status, MLA_DEV_TIMEOUT);
    __syncwarp();
  } else if (has_work && warp == 2) {
    // ------------------------------------------------------------- scores
    constexpr uint32_t kIdS = tc::idesc_bf16(128, kTok, false, false);
    const uint32_t id_page = tc::idesc_bf16(128, bs, false, false);
    const uint64_t kdesc = tc::smem_desc(smem_u32(sStage), 16, 1024, tc::kSwizzle128);
    const uint64_t krdesc = tc::smem_desc(smem_u32(sStage + 4 * kSlab), 16, 512, tc::kSwizzle64);
    const uint64_t qrdesc = tc::smem_desc(smem_u32(sm + Smem::rope), 16, 512, tc::kSwizzle64);
    const bool leader = tc::elect_one();
    int i = 0, ri = 0, seg_i = 0;
    bool ok = true, more = true;
    while (more) {
      if (!(ok = segment(seg_i))) break;
      more = seg.more;
      const int n = seg.k1 - seg.k0;
      ri += 2;
      if (!warp_wait(kQReady, seg_i & 1)) { ok = false; break; }
#pragma unroll 1
      for (int t = 0; t < n; ++t, ++i, ++ri) {
        const int slot = ri % kStages, b = i & 1;
        if (i >= 2 && !warp_wait(kSRead0 + b, ((i - 2) >> 1) & 1)) { ok = false; break; }
        if (!warp_wait(kFull0 + slot, (ri / kStages) & 1)) { ok = false; break; }
        tc::fence_after_sync();
        if (leader) {
          const uint32_t d = tmem + kSCol + (uint32_t)(b * kTok);
          const uint64_t at = (uint64_t)((slot * kStage) >> 4);
          if (pages == 1) {
#pragma unroll
            for (int c = 0; c < 16; ++c)
              tc::mma_bf16_tmem_a(d, tmem + kQCol + (uint32_t)(c * 8),
                                  kdesc + at + (uint64_t)(((c >> 2) * kSlab + (c & 3) * 32) >> 4), kIdS, c > 0);
          } else {
#pragma unroll 1
            for (int pj = 0; pj < 4 * pages; ++pj) {     // page by page, slab by slab
#pragma unroll
              for (int c = 0; c < 4; ++c)
                tc::mma_bf16_tmem_a(d + ((pj >> 2) << bs_shift), tmem + kQCol + (uint32_t)((pj & 3) * 32 + c * 8),
                                    kdesc + at + (uint64_t)(((pj << (bs_shift + 7)) + c * 32) >> 4), id_page,
                                    (pj & 3) > 0 || c > 0);
            }
          }
#pragma unroll
          for (int c = 0; c < 2; ++c)
            tc::mma_bf16(d, qrdesc + (uint64_t)((c * 32) >> 4), krdesc + at + (uint64_t)((c * 32) >> 4), kIdS, true);
          tc::commit(&bars[kSFull0 + b]);
        }
        __syncwarp();
      }
      if (!ok) break;
      ++seg_i;
    }
    if (!ok && leader) fail_out();
    if (leader) tc::commit(&bars[kFinalS]);
    __syncwarp();
    if (!mbar_wait(&bars[kFinalS], 0) && leader) set_status(a.status, MLA_DEV_TIMEOUT);
    __syncwarp();
  } else if (has_work && warp == 3) {
    // ---------------------------------------------------- what a tile needs
    int i = 0, ri = 0, seg_i = 0;
    bool ok = true, more = true;
    while (ok && more) {
      if (!(ok = segment(seg_i++))) break;
      more = seg.more;
      ri += 2;
#pragma unroll 1
      for (int k = seg.k0; k < seg.k1; ++k, ++i, ++ri) {
        const int b = i & 1, slot = ri % kStages;
        ok = (i < 2 || warp_wait(kPVDone0 + b, ((i >> 1) - 1) & 1)) &&   // its weights' buffer
             warp_wait(kFull0 + slot, (ri / kStages) & 1) &&             // what is in the stage
             warp_wait(kSFull0 + b, (i >> 1) & 1) && warp_wait(kXFull0 + b, (i >> 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars[kXFull0 + b], kXBytes);   // for tile i + 2
          asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(smem_u32(ready)), "r"(i + 1) : "memory");
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) fail_out();
  } else if (has_work && warp >= kSendWarp0) {
    // ------------------------------------------------------------ senders
    const int quad = warp - kSendWarp0, r = quad * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t peer = (uint32_t)(h ^ 1);
    const uint32_t x_peer = cl::map(smem_u32(sm + Smem::x), peer) + (uint32_t)r * 16;
    const uint32_t xbar_peer = cl::map(smem_u32(&bars[kXFull0]), peer);
    uint8_t* rope = sm + Smem::rope;
    const float* sSum = reinterpret_cast<const float*>(sm + Smem::sum);
    int i = 0, ri = 0, seg_i = 0;
    int read = 0;                        // segments read
    bool ok = true;
    auto query_in = [&]() {
#pragma unroll 1
      for (int part = 0; part < 2; ++part, ++ri) {
        const int slot = ri % kStages;
        if (!warp_wait(kFull0 + slot, (ri / kStages) & 1)) return false;
        take_query(sStage + slot * kStage, part, r, trow + kQCol, rope, a.scale_log2);
        if (lane == 0) mbar_arrive(&bars[kQRead0 + QuerySlots::bar_of(read - 1, part)]);
      }
      if (lane == 0) mbar_arrive(&bars[kQReady]);
      return true;
    };
    // Once the last tile of a segment is sent, the next one's query comes in and its
    // first tile is sent; the output of the last segment is written after it, when its
    // scores are on their way. (After two tiles it is written 3,000 cycles later.)
    TreeSeg last;
    int t = 0, n = 0, store_at = -1;     // -1: nothing waits to be written
    bool more = true;
    ok = segment(read++) && query_in();
    if (ok) n = seg.k1 - seg.k0;
#pragma unroll 1
    while (ok) {
      if (t == store_at) {
        if (!warp_wait(kODone, seg_i & 1) || !warp_wait(kSums, seg_i & 1)) { ok = false; break; }
        tc::fence_after_sync();
        store_rows(trow, 1, sSum[r], last.ql * a.num_heads - last.j * kBlockRows - quad * 32,
                   part_rows(a, last, share_idx) + (size_t)(quad * 32) * kDc + 256 * h,
                   sm + Smem::p + (4 + quad) * 4096, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kOFree]);
        ++seg_i;
        store_at = -1;
      }
      if (!more) break;
      if (t == n) {
        ri += n;
        last = seg;
        more = seg.more;
        if (more) {
          ok = segment(read++) && query_in();
          n = seg.k1 - seg.k0;
        }
        t = 0;
        store_at = more;
        continue;
      }
      const int b = i & 1;
      // the peer has read tile i - 2 from the buffer
      if (i >= 2 && !warp_wait(kPeerFree0 + b, ((i >> 1) - 1) & 1)) { ok = false; break; }
      if (!warp_wait(kSFull0 + b, (i >> 1) & 1)) { ok = false; break; }
      tc::fence_after_sync();
      uint32_t sv[2][32];
      tc::ld32(trow + kSCol + (uint32_t)(b * kTok), sv[0]);
      tc::ld32(trow + kSCol + (uint32_t)(b * kTok + 32), sv[1]);
      tc::wait_ld();
      loaded(sv[0]);
      loaded(sv[1]);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kSRead0 + b]);
      const uint32_t dst = x_peer + (uint32_t)(b * kXBytes), bar = xbar_peer + (uint32_t)b * 8;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t* v = sv[c >> 2] + 8 * (c & 3);
        send16(dst + c * (kBlockRows * 16), bar, pack_score(v[0], v[1]), pack_score(v[2], v[3]),
               pack_score(v[4], v[5]), pack_score(v[6], v[7]));
      }
      ++t;
      ++i;
    }
    if (!ok && lane == 0) fail_out();
  } else if (has_work) {
    // ------------------------------------------------------------ softmax
    const int quad = warp - kSoftWarp0, r = quad * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t pfree_peer = cl::map(smem_u32(&bars[kPeerFree0]), (uint32_t)(h ^ 1));
    float* sSum = reinterpret_cast<float*>(sm + Smem::sum);
    const float scale = score_scale(a.scale_log2);
    int i = 0, ri = 0, seg_i = 0;
    bool ok = true, more = true;
    while (more) {
      if (!(ok = segment(seg_i))) break;
      more = seg.more;
      ri += 2;
      const int n = seg.k1 - seg.k0, past = seg.len - seg.ql;
      const int row = (seg.j * kBlockRows + r) / a.num_heads;   // of the sequence
      const bool live_row = row < seg.ql;
      const uint64_t* mrow = a.mask + (size_t)(seg.q0 + (live_row ? row : 0)) * a.words;
      float m_used = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int t = 0; t < n; ++t, ++i, ++ri) {
        const int slot = ri % kStages, b = i & 1;
        const int tstart = (seg.k0 + t) * kTok, before = past - tstart;   // tokens from here on that precede the tree
        uint64_t live = ~0ull;
        if (before < kTok) {
          live = 0;
          if (live_row) {
            live = mask_from(mrow, a.words, max(-before, 0));
            if (before > 0) live = live << before | ((1ull << before) - 1);
          }
        }
        if (!wait_word(ready, i, abort_flag)) ok = false;
        if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
        tc::fence_after_sync();
        uint32_t sv[2][32];
        tc::ld32(trow + kSCol + (uint32_t)(b * kTok), sv[0]);
        tc::ld32(trow + kSCol + (uint32_t)(b * kTok + 32), sv[1]);
        const uint8_t* xp = sm + Smem::x + b * kXBytes + r * 16;
        uint4 pv[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) pv[c] = *reinterpret_cast<const uint4*>(xp + c * (kBlockRows * 16));
        const int2 inf = info[slot];
        tc::wait_ld();
        loaded(sv[0]);
        loaded(sv[1]);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kSRead0 + b]);
        float x[64];
#pragma unroll
        for (int j = 0; j < 64; ++j) x[j] = __uint_as_float(sv[j >> 5][j & 31]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          add_f16x2(pv[c].x, x[8 * c], x[8 * c + 1]);
          add_f16x2(pv[c].y, x[8 * c + 2], x[8 * c + 3]);
          add_f16x2(pv[c].z, x[8 * c + 4], x[8 * c + 5]);
          add_f16x2(pv[c].w, x[8 * c + 6], x[8 * c + 7]);
        }
        if (before < kTok || inf.x < kTok || inf.y != full_mask) {      // (the same for all threads)
          uint64_t there = inf.x < kTok ? (1ull << inf.x) - 1 : ~0ull;
          for (int p = 0; p < pages; ++p)
            if (!((inf.y >> p) & 1)) there &= ~((bs == 64 ? ~0ull : (1ull << bs) - 1) << (p << bs_shift));
          live &= there;
          float2 wild2 = make_float2(0.f, 0.f);      // stays 0 if every score is finite
#pragma unroll
          for (int j = 0; j < 64; j += 2)
            wild2 = fma_f32x2(make_float2(x[j], x[j + 1]), make_float2(0.f, 0.f), wild2);
          const bool wild = !(wild2.x + wild2.y == 0.f);
          if (__builtin_expect(wild, 0)) {
            // A token that is not finite makes a row that sees it NaN, whatever its weight.
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if ((((j < 32 ? (uint32_t)live : (uint32_t)(live >> 32)) >> (j & 31)) & 1) && !(fabsf(x[j]) < INFINITY)) l = NAN;
          }
#pragma unroll
          for (int j = 0; j < 64; ++j)
            x[j] = ((j < 32 ? (uint32_t)live : (uint32_t)(live >> 32)) >> (j & 31)) & 1 ? x[j] : -INFINITY;
          // Each thread one token's half of the columns. (A token that is not finite has
          // no row with a finite score.)
          const int tok = r & 63;
          if (wild || there != ~0ull)
            clean_stage(sStage + slot * kStage + ((tok >> bs_shift) << (bs_shift + 9)) + (r >> 6) * 2 * (bs * 128), bs * 128,
                        tok & (bs - 1), (there >> tok) & 1, tstart + tok >= past);
        }
        float mx[22];
#pragma unroll
        for (int j = 0; j < 21; ++j) mx[j] = fmax3(x[3 * j], x[3 * j + 1], x[3 * j + 2]);
        mx[21] = x[63];
#pragma unroll
        for (int j = 0; j < 7; ++j) mx[j] = fmax3(mx[3 * j], mx[3 * j + 1], mx[3 * j + 2]);
        mx[0] = fmax3(mx[0], mx[1], mx[2]);
        mx[3] = fmax3(mx[3], mx[4], mx[5]);
        const float m_cand = fmax3(mx[0], mx[3], fmaxf(mx[6], mx[21])) * scale;
        float alpha = 1.f;
        bool rescale = false;
        if (m_cand > m_used + kRescaleLog2 || (m_used == -INFINITY && m_cand != -INFINITY)) {
          if (m_used != -INFINITY) {
            alpha = fast_exp2(m_used - m_cand);
            rescale = t > 0;
          }
          l *= alpha;
          m_used = m_cand;
        }
        const bool any = __any_sync(0xffffffffu, rescale);
        // (every lane has the peer's scores: they are in the vote's maxima)
        if (lane == 0) cl::arrive_remote_relaxed(pfree_peer + (uint32_t)b * 8);
        if (any) {
          if (!warp_wait(kPVDone0 + (b ^ 1), ((i - 1) >> 1) & 1)) { ok = false; break; }
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[32];
            tc::ld32(trow + kOCol + 32 * c, o);
            tc::wait_ld();
            loaded(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tc::st32(trow + kOCol + 32 * c, o);
          }
          tc::wait_st();
          tc::fence_before_sync();
        }
        const float mneg = m_used == -INFINITY ? 0.f : -m_used;
        const float2 sc2 = make_float2(scale, scale), mn2 = make_float2(mneg, mneg);
        // the senders' staging is in the weights' buffers
        if (t == 0 && seg_i > 0 && !warp_wait(kOFree, (seg_i - 1) & 1)) { ok = false; break; }
        uint8_t* pp = sm + Smem::p + b * kPBytes;
        float sum[4] = {};
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t pk[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 e = fma_f32x2(make_float2(x[8 * c + 2 * k], x[8 * c + 2 * k + 1]), sc2, mn2);
            pk[k] = pack_bf16(fast_exp2(e.x), fast_exp2(e.y));
            add_bf16x2(pk[k], sum[2 * (k & 1)], sum[2 * (k & 1) + 1]);
          }
          *reinterpret_cast<uint4*>(pp + sw128(r, c)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kPFull0 + b]);
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      if (!ok) break;
      // ---- the segment's sums, then its output rows
      const float inv = l == 0.f ? 0.f : 1.f / l;      // (NaN stays NaN)
      sSum[r] = inv;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kSums]);
      const int64_t slot = (int64_t)share_idx + seg.item;
      a.lse[(slot * 2 + h) * kBlockRows + r] = l == 0.f ? -INFINITY : m_used + log2f(l);
      if (!warp_wait(kODone, seg_i & 1)) { ok = false; break; }
      tc::fence_after_sync();
      store_rows(trow, 0, inv, seg.ql * a.num_heads - seg.j * kBlockRows - quad * 32,
                 part_rows(a, seg, share_idx) + (size_t)(quad * 32) * kDc + 256 * h, sm + Smem::p + quad * 4096, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kOFree]);
      ++seg_i;
    }
    if (!ok && lane == 0) fail_out();
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::dealloc(tmem, kTmemCols);
  cl::sync();  // the peer no longer sends into this CTA's shared memory
}

bool al(const void* p, uintptr_t x) { return (reinterpret_cast<uintptr_t>(p) & (x - 1)) == 0; }

// Clusters of the decode that run at once on the current device (0: unknown).
int tree_clusters() {
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cached[dev] > 0) return cached[dev];
  if (cudaFuncSetAttribute(tree_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::alloc) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(2);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = Smem::alloc;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, tree_decode_kernel, &lc) != cudaSuccess) return 0;
  cached[dev] = n;
  return n;
}
int tree_shares(const mla_config* cfg) {
  const int c = split_ctas(cfg) / 2;
  if (cfg->num_ctas > 0) return c > 0 ? c : 1;
  if (c <= 0) return c;
  const int most = tree_clusters();
  return most > 0 && most < c ? most : c;
}
bool tree_sizes_fit(int64_t num_q, int64_t max_blocks, int bs) {
  const int64_t tokens = max_blocks * bs;
  return num_q <= kTreeMaxRows && tokens <= ((int64_t)1 << 30) && (num_q == 0 || tokens <= ((int64_t)1 << 35) / num_q);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_tree_decode_workspace_size(const mla_config* cfg, int64_t num_q, int32_t batch) {
  if (validate_config(cfg) != MLA_OK || cfg->dtype != MLA_BF16 || num_q < 0 || num_q > kTreeMaxRows || batch < 0)
    return 0;
  const int C = tree_shares(cfg);
  if (C <= 0) return 0;
  return tree_ws(num_q, cfg->num_heads, C, batch).total;
}

mla_status mla_tree_decode(const mla_config* cfg, const void* q_abs, const void* cache, int64_t num_blocks,
                           const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                           const int32_t* query_start_loc, int32_t batch, int64_t num_q, const uint64_t* tree_mask,
                           int32_t mask_words, const void* W_uv, void* workspace, size_t ws_bytes, void* out,
                           void* stream) {
  if (validate_config(cfg) == MLA_OK && cfg->dtype != MLA_BF16) return MLA_ERR_UNSUPPORTED;
  mla_status s = decode_paged_checks(cfg, q_abs, cache, num_blocks, block_table, max_blocks_per_seq, seq_lens,
                                     query_start_loc, batch, num_q);
  if (s != MLA_OK) return s;
  if (mask_words < 1) return MLA_ERR_INVALID_ARGUMENT;
  if (mask_words > 16) return MLA_ERR_UNSUPPORTED;
  if (!workspace || !al(workspace, 256)) return MLA_ERR_INVALID_ARGUMENT;
  if (num_q == 0) return MLA_OK;
  if (!tree_mask || !W_uv || !out || !al(tree_mask, 8) || !al(W_uv, 16) || !al(out, 16)) return MLA_ERR_INVALID_ARGUMENT;
  const int H = cfg->num_heads, bs = cfg->block_size;
  if (!tree_sizes_fit(num_q, max_blocks_per_seq, bs)) return MLA_ERR_UNSUPPORTED;
  const int C = tree_shares(cfg);
  if (C <= 0) return MLA_ERR_CUDA;
  const TreeWs L = tree_ws(num_q, H, C, batch);
  if (ws_bytes < L.total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  TreeArgs a{};
  a.q_abs = (const uint16_t*)q_abs;
  a.num_blocks = num_blocks;
  a.num_q = num_q;
  a.block_table = block_table;
  a.max_blocks = max_blocks_per_seq;
  a.block_size = bs;
  a.num_heads = H;
  a.batch = batch;
  a.words = mask_words;
  a.shares = C;
  a.seq_lens = seq_lens;
  a.query_start_loc = query_start_loc;
  a.mask = tree_mask;
  a.scale_log2 = (float)(cfg->softmax_scale * 1.4426950408889634);
  a.ws = ws;
  a.status = &reinterpret_cast<WsHeader*>(ws)->status;
  a.plan = reinterpret_cast<int4*>(ws + L.plan);
  a.lse = reinterpret_cast<float*>(ws + L.lse);
  a.opart = reinterpret_cast<float*>(ws + L.opart);
  a.o_lat = reinterpret_cast<float*>(ws + L.o_lat);
  // With num_blocks == 0 every block id is rejected before any copy; the maps
  // still need an extent.
  const uint64_t rows = (uint64_t)(num_blocks > 0 ? num_blocks : 1) * bs;
  CUtensorMap slab4, rope_map, q_map, qrope_map;
  if (!encode_row_map(&q_map, q_abs, (uint64_t)num_q * H, kBlockRows) ||
      !encode_rope_half_map(&qrope_map, q_abs, (uint64_t)num_q * H, kBlockRows / 2))
    return MLA_ERR_CUDA;
  if (!encode_slab_map(&slab4, cache, rows, (uint32_t)bs, 4) ||
      !encode_rope_half_map(&rope_map, cache, rows, (uint32_t)bs))
    return MLA_ERR_CUDA;
  cudaError_t e = cudaFuncSetAttribute(tree_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::alloc);
  if (e == cudaSuccess)
    e = launch_pdl(tree_decode_kernel, dim3(2 * C), dim3(kThreads), Smem::alloc, st, slab4, rope_map, q_map, qrope_map, a);
  if (e != cudaSuccess) return MLA_ERR_CUDA;
  e = launch_tree_out(a, W_uv, out, st);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
