// mla_page8_decode and mla_page8_decode_mass: split-KV attention of absorbed
// queries over pages of e4m3 codes with one scale per page, the merge of the
// splits, the output projection, and (mass) the attention weight of every
// cached token accumulated at its slot.
//
// For query row n, head h and token t of page p with scale S_p:
//   s_t = softmax_scale * log2(e) * (S_p q_lat . code_t + q_rope . k_t)   (base 2)
//   o   = sum_t 2^(s_t - lse) S_p code_t,     lse = log2 sum_t 2^(s_t)
//
// The codes go to the 5th-generation tensor cores as they lie in the cache
// (kind::f8f6f4, fp32 accumulation in TMEM): nothing is dequantised. For that
// the 128 tokens of a tile are the rows of both products, and the few
// (row, head) columns are the other operand, split into 8-bit terms that are
// columns of their own, so a tile is read from shared memory once for all of
// them:
//   scores  S[128 tokens, 2 NH] = codes[128, 512] . (q_1 | q_2)^T,
//           R[128 tokens, NH]   = k[128, 64] . q_rope^T  (bf16)
//     q_lat 2^a = q_1 + 2^-5 q_2 in e4m3, a per head: both terms together hold
//     a bf16 exactly down to 2^-15 of the head's largest, and the rest within
//     2^-23 of that largest;
//   output  O[512, 3 NH] = codes[128, 512]^T . (p_1 | p_2 | p_3)
//     p = p_1 + p_2 + 2^-5 p_3 in e5m2, each term the nearest to what is left:
//     the f16 nearest to p, 11 significant bits (error 2^-11), in steps of
//     2^-25 of the running reference at the least, so a long tail of small
//     weights behind a large one is not lost.
// The page's scale enters a score as a factor of its token (a row), and the
// output as part of the weight: the columns hold 2^(s_t - ref) S_p, and the
// softmax sum adds the same number divided by S_p again. The running reference
// of a head follows s_t + log2 S_p, and O is rescaled in TMEM only when it is
// outgrown by more than 2^11.75.
//
// NH = 16 or 32 heads of one row make a column group; with 16 heads and several
// rows a sequence (R = 2), two rows that follow one another do, each with its
// own last token, so that a tile of tokens serves both. The work is cut as in
// the other decodes (units of one row or pair and 64 tokens in equal contiguous
// shares), and each share is taken by one CTA per group: the CTAs of a share
// read the same tokens at the same time, so a token comes from HBM once for
// all heads. Per CTA (384 or 640 threads):
//   warp 0      copies: 128 tokens a stage (4 slabs of 128 codes, one of rope
//               values), two stages, SWIZZLE_128B; block ids are checked. 64
//               tokens are copied as soon as the output products of those in
//               their place are done;
//   warp 1      issues the output products of a tile as soon as its weights are
//               stored (one lane); owns the TMEM;
//   warp 2      issues the scores of a tile as soon as it has landed and the
//               score columns are read;
//   warp 3      copies the next segment's query terms, which a kernel before
//               this one has split and laid out as the operand;
//   warps 4-    softmax, 4 warps for every 8 heads: thread r of each such group
//               owns token r. Tokens that are not there are zeroed in the
//               stage, so a weight of 0 never meets a NaN code.
// Every wait is bounded; on a timeout the roles leave their loops, the issuers
// wait for their products and the copies' warps for their copies before TMEM is
// freed.
//
// Bound and measurements (one GB300, launches alone with a cold L2):
//  - 64 sequences of 4,096 tokens, 16 heads: 41 us for 168 MB. 27 us of them are
//    the main loop, at 6.2 TB/s (0.92 of a copy's rate); the rest is the start
//    (split, block table, first pages: 5 us), the last products, the partials
//    and a tail of shares that end apart.
//  - 32 sequences of up to 32,768 tokens, 128 heads: 274 us; 4 chunks of 512 rows
//    on 2,560 tokens, 16 heads: 292 us. Neither bytes (0.18 and 0.04 of HBM) nor
//    products (tensor pipe busy 0.30 and 0.27) bound these, but the time of one
//    stage from copy to release: copy 1,700 cycles, scores 1,500, softmax 1,900,
//    output products 1,600, over two stages 3,400 cycles a tile of which the
//    products need 1,820. Three stages do not fit beside the operands of 32
//    columns (36 KB of query terms, 24 KB of weights). A tile in which a
//    reference is outgrown takes some 2,000 cycles more.
//  Tried and not kept: each slab of a stage with barriers of its own (3 to 8 %
//  slower), pairs of CTAs that copy each other's tokens by multicast (no
//  difference: the L2 is not what bounds the copies).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "async_copy.cuh"
#include "internal.h"
#include "merge.cuh"
#include "page8.cuh"
#include "pair_math.cuh"
#include "sched.cuh"
#include "tcgen05.cuh"

namespace mla {
namespace {

constexpr int kTok = 128;                     // tokens per stage
constexpr int kSlab = kTok * 128;             // 128 rows of 128 bytes
constexpr int kStageB = 5 * kSlab;            // four slabs of codes, one of rope values
constexpr int HT = 8;                         // heads (columns) of a softmax thread
constexpr int kSoftWarp0 = 4;
// named barriers: all softmax warps; each 16 columns' (2, 3); each 8 columns' (4-7)
constexpr int kSoftBar = 1, kHeadsBar = 2, kGroupBar = 4;
constexpr float kRefLog2 = 4.f;               // a weight equal to the reference is held as 2^4
constexpr float kNoRef = 1e38f;               // nref of a head without one: every score outgrows it
// the reference follows when outgrown by 2^11.75: a weight of 2^15.75 is still
// below e5m2's largest number, 1.75 * 2^15
constexpr float kGrowLog2 = 11.75f;
constexpr uint32_t kTmemCols = 512, kSCol = 0, kOCol = 128;

struct P8Args {
  const uint16_t* q_abs;
  const float* scales;
  int64_t num_blocks;
  const int32_t* block_table;
  int32_t max_blocks;
  int32_t block_size;
  int32_t num_heads;
  int32_t groups;     // column groups of a row: num_heads / NH
  int32_t shares;     // shares of the work; CTAs = shares * groups
  int64_t num_q;
  float scale_log2;
  uint8_t* ws;
  uint8_t* q8;         // [num_q, groups] query terms as shared memory holds them
  float* coef;         // [num_q, H] score factors
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  int32_t batch;
  int32_t self_plan;   // the kernel derives the split itself
  int32_t pair;        // rows go in pairs (R = 2)
  // partials of each 16 heads: [slots][16] and [slots][16][512]; the first
  // 16 heads' where ws_layout has them, the others' one after another
  float* lse_first;
  float* o_first;
  float* lse_rest;
  float* o_rest;
  int64_t slots;
  int* arrive;         // [num_q, groups] parts merged so far (fused)
  float* o_lat;        // [num_q, H, 512]
  float* lse;          // [num_q, H], base 2
  float* scores;       // [num_q, H / 16, max tokens, 16], base 2; NULL without mass
  int32_t fused;       // merge the splits in the decode kernel
};

// The partials of heads 16 t16 ... 16 t16 + 15 (of row t16 of a pair).
__device__ __forceinline__ float* lse_part(const P8Args& a, int t16) {
  return t16 == 0 ? a.lse_first : a.lse_rest + (int64_t)(t16 - 1) * a.slots * kHG;
}
__device__ __forceinline__ float* o_part(const P8Args& a, int t16) {
  return t16 == 0 ? a.o_first : a.o_rest + (int64_t)(t16 - 1) * a.slots * kHG * kDc;
}

// The decode workspace: the split plan and the first 16 heads' partials of
// ws_layout, the other heads' partials, the query terms and score factors, the
// merge's counters, the merged latents, their log-sum-exps and (with mass) the
// scores.
struct P8Ws {
  size_t lse_rest, o_rest, q8, coef, arrive, o_lat, lse, scores, total;
};
int group_heads(int H) { return H >= 32 ? 32 : 16; }
// Rows go in pairs where the 16 heads of one leave half of the columns empty
// and two of three sequences have a second row. (Rows of their own take the
// narrower kernel, which is quicker by itself.) 32 sequences of 4,096 tokens on
// one GB300, us by rows / in pairs: 32 rows 34.8 / 39.3, 48 rows 35.5 / 36.2,
// 56 rows 37.9 / 36.4, 64 rows 41.8 / 36.8; 8 chunks of 128 rows 125 / 99.
bool use_pairs(int H, int64_t num_q, int32_t batch) { return H == 16 && 3 * num_q >= 5 * (int64_t)batch; }
// Shares of the work: with one CTA per group to a share, about num_ctas CTAs.
int p8_shares(int H, int num_ctas) {
  const int s = num_ctas / (H / group_heads(H));
  return s > 0 ? s : 1;
}
// (the split counts units of 64 tokens and a row in 32 bits)
bool p8_sizes_fit(int64_t num_q, int32_t max_blocks, int bs) {
  const int64_t tokens = (int64_t)max_blocks * bs;
  return num_q <= 48 * 1024 && tokens <= (int64_t)1 << 30 && num_q * ((tokens + kTile - 1) / kTile) <= (int64_t)1 << 30;
}
P8Ws p8_ws(int64_t num_q, int H, int shares, int64_t max_tokens, bool mass) {
  const WsLayout W = ws_layout(num_q, 1, shares);
  // (16 heads: room for pairs whether they are used or not, which goes by the
  // batch, so that a workspace for many sequences does for fewer)
  const size_t rest = (size_t)((H == 16 ? 2 : H / kHG) - 1) * W.slots * kHG;
  P8Ws L;
  L.lse_rest = align_up(W.total, 256);
  L.o_rest = align_up(L.lse_rest + rest * 4, 256);
  L.q8 = align_up(L.o_rest + rest * kDc * 4, 256);
  L.coef = align_up(L.q8 + (size_t)num_q * H * (2 * kDc + 2 * kDr), 256);
  L.arrive = align_up(L.coef + (size_t)num_q * H * 4, 256);
  L.o_lat = align_up(L.arrive + (size_t)num_q * (H / kHG) * 4, 256);
  L.lse = align_up(L.o_lat + (size_t)num_q * H * kDc * 4, 256);
  L.scores = align_up(L.lse + (size_t)num_q * H * 4, 256);
  L.total = mass ? align_up(L.scores + (size_t)num_q * H * max_tokens * 4, 256) : L.scores;
  return L;
}

// Shared memory of one CTA.
template <int NH>
struct Sm {
  static constexpr int groups = NH / HT;                // of softmax warps
  static constexpr int soft = groups * 128;             // softmax threads
  static constexpr int threads = kSoftWarp0 * 32 + soft;
  static constexpr int QB = NH == 16 ? 2 : 1;           // query buffers
  static constexpr int q_slab = 2 * NH * 128;           // 128 codes of every term row
  static constexpr int q_rope = 4 * q_slab;
  static constexpr int q_bytes = q_rope + NH * 128;
  static constexpr int p_bytes = 3 * NH * kTok;         // blocks of 16 columns: [16][8 tokens][16 bytes]
  static constexpr int stage = 0;
  static constexpr int q = stage + 2 * kStageB;
  static constexpr int p = q + QB * q_bytes;
  static constexpr int coef = p + 2 * p_bytes;          // [QB][NH] score factor of a head
  static constexpr int red = coef + QB * NH * 4;        // [softmax warps][HT]
  static constexpr int merge = red + groups * 4 * HT * 4;  // merge scratch, one per 16 columns
  static constexpr int merge_bytes = (2 * kHG + kMergeChunk * kHG) * 4;
  static constexpr int info = merge + NH / 16 * merge_bytes;  // [2] tokens of a stage
  static constexpr int scale = info + 16;               // [2][8] page scales of a stage, -1: no page
  static constexpr int self_rows = NH == 16 ? kSelfMaxRows : 128;  // rows of a self-planned launch
  static constexpr int rows = scale + 64;               // [self_rows] int4
  static constexpr int bars = rows + self_rows * 16;
  static constexpr int misc = bars + 24 * 8;            // TMEM base, abort flag, merge flag
  static constexpr int bytes = misc + 16;               // ... and the plan's units
  static constexpr int alloc = bytes + 1024;
  static_assert(alloc <= 227 * 1024, "shared memory budget");
  static_assert(q % 1024 == 0 && q_rope % 1024 == 0 && q_bytes % 1024 == 0 && p % 128 == 0, "swizzle atoms");
  static_assert(bars % 8 == 0 && merge % 16 == 0 && coef % 16 == 0 && rows % 16 == 0, "alignment");
};

enum {
  kFull = 0,      // [2] stage landed
  kEmpty = 2,     // [2][2] products of a stage's first and last 64 tokens done
  kQReady = 6,    // [2] query terms landed
  kQFree = 8,     // [2] the segment's score products done, its factors read (1 + softmax warps)
  kSFull = 10,    // scores in TMEM
  kSFree = 11,    // scores read (softmax warps)
  kPFull = 12,    // [2] weights stored (softmax warps)
  kPVDone = 14,   // [2] output products done
  kODone = 16,    // the segment's output products done
  kOFree = 17,    // the output read (softmax warps)
  kFinalS = 18,   // every score product done
  kFinalO = 19,   // every output product done
  kNumBars = 20
};

// Instruction descriptor, kind::f8f6f4, fp32 accumulator: A e4m3, B e4m3 (0) or
// e5m2 (1), each K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_f8(int N, int b_type, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)b_type << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kTok >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// Lane l reads 8 consecutive 32-bit columns of TMEM lane (base + l).
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, float& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(r) : "r"(taddr));
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "f"(r) : "memory");
}

// Bounded wait that also gives up when another role has aborted.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 15u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitTimeoutNs) return false;
    }
  }
}

__device__ __forceinline__ bool bar_or(int id, int nthreads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\t"
      "barrier.red.or.pred po, %2, %3, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}

// The largest of a value over the warp (NaN does not count, unless all are).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// The log-sum-exp of merged parts (kHG apart) from the largest that is not NaN and
// 1 / the weight sum (0 where the sum is not a positive number). Where there is no
// largest, the parts have no token, or one is NaN.
__device__ __forceinline__ float merged_lse(float m, float inv, const float* lse, int parts) {
  const float nan = __int_as_float(0x7fffffff);
  if (m != -INFINITY) return inv > 0.f ? m - log2f(inv) : nan;
  for (int s = 0; s < parts; ++s)
    if (isnan(__ldcg(lse + s * kHG))) return nan;
  return m;
}

// The two e4m3 terms of 16 scaled query values (eight bf16 pairs in u):
// t1 = e4m3(x), t2 = e4m3((x - t1) 2^5); a value that is not finite is NaN.
__device__ __forceinline__ void query_terms(const uint32_t* u, float f, uint4& t1, uint4& t2) {
  uint32_t a[4], b[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    a[k] = b[k] = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = u[2 * k + i];
      // (inf - inf = NaN)
      float x0 = __uint_as_float(w << 16), x1 = __uint_as_float(w & 0xffff0000u);
      x0 = isinf(x0) ? __int_as_float(0x7fffffff) : x0 * f;
      x1 = isinf(x1) ? __int_as_float(0x7fffffff) : x1 * f;
      const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
      const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
      const __nv_fp8x2_storage_t d = __nv_cvt_float2_to_fp8x2(
          make_float2((x0 - v.x) * 32.f, (x1 - v.y) * 32.f), __NV_SATFINITE, __NV_E4M3);
      a[k] |= (uint32_t)c << (16 * i);
      b[k] |= (uint32_t)d << (16 * i);
    }
  }
  t1 = make_uint4(a[0], a[1], a[2], a[3]);
  t2 = make_uint4(b[0], b[1], b[2], b[3]);
}

// Is one of a token's codes NaN? (its row of the first slab; in any order)
__device__ __forceinline__ bool nan_code(const uint8_t* row) {
  uint32_t found = 0;
#pragma unroll 1
  for (int c = 0; c < 32; ++c) {
    const uint4 x = *reinterpret_cast<const uint4*>(row + (c >> 3) * kSlab + (c & 7) * 16);
    found |= __vcmpeq4(x.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(x.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
             __vcmpeq4(x.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(x.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
  }
  return found != 0;
}

// Untiled copy of `bytes` (a multiple of 16) to shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// The split plan: rows[n] = {sequence, position of the (pair's last) row, tiles,
// first unit}; tiles is -1 for the second row of a pair and 0 where nothing is
// to be done. fill_rows writes all but the first units, of the sequences
// first, first + step, ... and their rows (of a pair, the first) lane,
// lane + lanes, .... Sequences that are not valid own no tiles.
__device__ __forceinline__ void fill_rows(const P8Args& a, int4* rows, uint32_t* status, int first,
                                          int step, int lane, int lanes) {
  const int64_t max_len = (int64_t)a.max_blocks * a.block_size;
  const int R = a.pair ? 2 : 1;
  for (int b = first; b < a.batch; b += step) {
    const int len = a.seq_lens[b];
    const int q0 = a.query_start_loc[b], q1 = a.query_start_loc[b + 1];
    const int ql = q1 - q0;
    if (q0 < 0 || q1 > a.num_q || ql < 0) {
      set_status(status, MLA_DEV_BAD_SEQ);
      continue;
    }
    const bool bad = ql > len || len < 0 || (int64_t)len > max_len;
    if (bad && ql > 0) set_status(status, MLA_DEV_BAD_SEQ);
    for (int j = lane * R; j < ql; j += lanes * R) {
      const bool two = R == 2 && j + 1 < ql;
      const int pos = len - ql + j + (two ? 1 : 0);
      rows[q0 + j] = make_int4(b, pos, bad ? 0 : (pos + kTile) / kTile, 0);
      if (two) rows[q0 + j + 1] = make_int4(b, pos, bad ? 0 : -1, 0);
    }
  }
}
// The rows' first units, by one warp.
__device__ __forceinline__ void scan_rows(int4* rows, int num_q, int lane, int* total) {
  int run = 0;
  for (int c = 0; c < num_q; c += 32) {
    const int v = c + lane < num_q ? max(rows[c + lane].z, 0) : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (c + lane < num_q) rows[c + lane].w = run + incl - v;
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) *total = run;
}
// Where share `c` begins: a walker over the rows (each warp for itself).
__device__ __forceinline__ bool start_share(SchedWalker& sw, const int4* rows, int num_q, int total,
                                            int shares, int c, int lane) {
  sw.row_info = rows;
  sw.plan_ok = true;
  sw.G = 1;
  sw.g = 0;
  sw.share = total > 0 ? (total + shares - 1) / shares : 1;
  sw.u = c * sw.share;
  sw.u_end = min(sw.u + sw.share, total);
  if (sw.u >= sw.u_end) return false;
  for (int r = 0; r < num_q; r += 32) {
    const int4 ri = r + lane < num_q ? rows[r + lane] : make_int4(0, 0, 0, 0);
    const uint32_t hit = __ballot_sync(0xffffffffu, ri.z > 0 && ri.w <= sw.u && sw.u < ri.w + ri.z);
    if (hit) {
      const int l = __ffs(hit) - 1;
      sw.n = r + l;
      sw.k = sw.u - __shfl_sync(0xffffffffu, ri.w, l);
      return true;
    }
  }
  return false;
}

// The plan of more rows than a CTA holds: one CTA, a warp per sequence, into the
// workspace (as SchedWalker::init reads it).
template <int NT>
__device__ __forceinline__ void plan_rows(const P8Args& a, int tid) {
  __shared__ int s_warp[NT / 32];
  const int lane = tid & 31, warp = tid >> 5, Nq = (int)a.num_q;
  const WsLayout L = ws_layout(a.num_q, 1, a.shares);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(a.ws);
  int4* rows = reinterpret_cast<int4*>(a.ws + L.row_info);
  int4* cta_start = reinterpret_cast<int4*>(a.ws + L.cta_start);
  for (int n = tid; n < Nq; n += NT) rows[n] = make_int4(-1, -1, 0, 0);
  __syncthreads();
  fill_rows(a, rows, &hdr->status, warp, NT / 32, lane, 32);
  __syncthreads();
  // first units: an exclusive scan, a contiguous piece per thread
  const int per = (Nq + NT - 1) / NT;
  const int beg = min(Nq, tid * per), end = min(Nq, beg + per);
  int local = 0;
#pragma unroll 8
  for (int n = beg; n < end; ++n) local += max(rows[n].z, 0);
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int run = incl - local, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    run += w < warp ? s_warp[w] : 0;
    total += s_warp[w];
  }
  const int share = total > 0 ? (total + a.shares - 1) / a.shares : 1;
#pragma unroll 8
  for (int n = beg; n < end; ++n) {
    const int z = max(rows[n].z, 0);
    rows[n].w = run;
    // the shares that begin in this row
    for (int c = (run + share - 1) / share; c * share < run + z; ++c) cta_start[c] = make_int4(n, 0, c * share - run, 0);
    run += z;
  }
  if (tid == 0) {
    hdr->magic = kMagic;
    hdr->mode = 0;
    hdr->qblocks = 0;
    hdr->total_units = total;
    hdr->share = share;
    hdr->num_ctas = a.shares;
    hdr->groups = 1;
    hdr->num_q = Nq;
    hdr->batch = a.batch;
  }
}

// The query of one (row, column group) as the decode's operand: for each head
// its two e4m3 terms (rows h and NH + h of four 128-byte slabs) and its bf16
// rope values, swizzled as shared memory holds them, and the factor that
// undoes the head's scale. 16 threads a head, 32 latent columns each. Where the
// decode does not find its split itself, the first CTA does, beside the others.
// Latency for a decode step (4.0 us for 64 rows of 16 heads, mostly the launch,
// and hidden behind the decode's start); HBM for chunks: 15 us for 2,048 rows, 75
// MB read and written.
template <int NH>
__global__ void __launch_bounds__(NH * 16) page8_query_kernel(const __grid_constant__ P8Args a) {
  using S = Sm<NH>;
  pdl_wait();
  pdl_launch_dependents();
  if (!a.self_plan && blockIdx.x == 0) {
    plan_rows<NH * 16>(a, threadIdx.x);
    return;
  }
  const int block = blockIdx.x - (a.self_plan ? 0 : 1);
  const int h = threadIdx.x >> 4, part = threadIdx.x & 15;
  const size_t row = (size_t)block * NH + h;   // (row n, head) in order
  const uint4* src = reinterpret_cast<const uint4*>(a.q_abs + row * kRow);
  uint8_t* dst = a.q8 + (size_t)block * S::q_bytes;
  uint4 x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = src[part * 4 + k];
  uint4 rope = make_uint4(0, 0, 0, 0);
  if (part < 8) rope = src[kDc / 8 + part];
  float mx = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v0 = fabsf(__uint_as_float(u[e] << 16)), v1 = fabsf(__uint_as_float(u[e] & 0xffff0000u));
      mx = fmaxf(mx, fmaxf(isinf(v0) ? 0.f : v0, isinf(v1) ? 0.f : v1));
    }
  }
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  // 2^e with mx 2^e in [2^7, 2^8); heads below 2^-112 as 2^-112
  const int e = min(134 - (int)(__float_as_uint(mx) >> 23), 119);
  const float f = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t u[8] = {x[2 * k].x, x[2 * k].y, x[2 * k].z, x[2 * k].w,
                           x[2 * k + 1].x, x[2 * k + 1].y, x[2 * k + 1].z, x[2 * k + 1].w};
    uint4 t1, t2;
    query_terms(u, f, t1, t2);
    const int c16 = part * 2 + k;  // 16-code piece of the row
    uint8_t* slab = dst + (c16 >> 3) * S::q_slab;
    *reinterpret_cast<uint4*>(slab + sw128(h, c16 & 7)) = t1;
    *reinterpret_cast<uint4*>(slab + sw128(NH + h, c16 & 7)) = t2;
  }
  if (part < 8) *reinterpret_cast<uint4*>(dst + S::q_rope + sw128(h, part)) = rope;
  if (a.fused && threadIdx.x == 0) a.arrive[block] = 0;
  if (part == 0) a.coef[row] = a.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
}

// Zeros for the latents of rows that own no tiles.
__device__ __forceinline__ void zero_other_rows(const P8Args& a, const int4* rows, int tid, int nthreads) {
  for (int64_t n = blockIdx.x; n < a.num_q; n += gridDim.x) {
    if (rows[n].z != 0) continue;
    float4* row = reinterpret_cast<float4*>(a.o_lat + (size_t)n * a.num_heads * kDc);
    for (int i = tid; i < a.num_heads * kDc / 4; i += nthreads) row[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

template <int NH, int R>
__global__ void __launch_bounds__(Sm<NH>::threads, 1)
    page8_decode_kernel(const __grid_constant__ CUtensorMap codes_map,
                        const __grid_constant__ CUtensorMap rope_map, const __grid_constant__ P8Args a) {
  static_assert(R == 1 || NH == 32, "a pair is 2 x 16 heads");
  using S = Sm<NH>;
  constexpr int QB = S::QB, kThreads = S::threads, kSoftThreads = S::soft;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::bars);
  int* info = reinterpret_cast<int*>(sm + S::info);
  float* page_sc = reinterpret_cast<float*>(sm + S::scale);
  float* coef = reinterpret_cast<float*>(sm + S::coef);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + S::misc + 4);
  int* merge_flag = reinterpret_cast<int*>(sm + S::misc + 8);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int share = blockIdx.x / a.groups, grp = blockIdx.x % a.groups;
  uint32_t* status = &reinterpret_cast<WsHeader*>(a.ws)->status;
  const int bs = a.block_size;
  const int bs_shift = bs == 16 ? 4 : (bs == 32 ? 5 : 6);

  int4* plan = reinterpret_cast<int4*>(sm + S::rows);
  int* plan_total = reinterpret_cast<int*>(sm + S::misc + 12);
  if (a.self_plan)
    for (int n = tid; n < (int)a.num_q; n += kThreads) plan[n] = make_int4(-1, -1, 0, 0);
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const int n = (i == kSFree || i == kPFull || i == kPFull + 1 || i == kOFree) ? kSoftThreads / 32
                    : (i == kQFree || i == kQFree + 1)   ? 1 + kSoftThreads / 32
                                                         : 1;
      mbar_init(&bars[i], n);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&codes_map);
    prefetch_tensormap(&rope_map);
  }
  if (warp == 1) tc::alloc(tmem_slot, kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // The kernel before this one is page8_query_kernel, which starts when
  // everything before it has finished. So what the caller gave (lengths, pages,
  // scales) may be read now; the query terms, the workspace and the output
  // have to wait.
  SchedWalker sw;
  bool has_work;
  if (a.self_plan) {
    fill_rows(a, plan, blockIdx.x == 0 ? status : nullptr, tid, kThreads, 0, 1);
    __syncthreads();
    if (warp == 0) scan_rows(plan, (int)a.num_q, lane, plan_total);
    __syncthreads();
    has_work = start_share(sw, plan, (int)a.num_q, *plan_total, a.shares, share, lane);
  } else {
    pdl_wait();
    has_work = sw.init(a.ws, a.num_q, 1, a.shares, share);
  }
  pdl_launch_dependents();
  if (warp >= kSoftWarp0) {
    pdl_wait();
    const int st = tid - kSoftWarp0 * 32;
    if (a.self_plan && blockIdx.x == 0) {
      // the plan, for the merge kernels
      int4* row_info = reinterpret_cast<int4*>(a.ws + ws_layout(a.num_q, 1, a.shares).row_info);
      for (int n = st; n < (int)a.num_q; n += kSoftThreads) row_info[n] = sw.row_info[n];
      if (st == 0) {
        WsHeader* hdr = reinterpret_cast<WsHeader*>(a.ws);
        hdr->magic = kMagic;
        hdr->mode = 0;
        hdr->qblocks = 0;
        hdr->total_units = *plan_total;
        hdr->share = sw.share;
        hdr->num_ctas = a.shares;
        hdr->groups = 1;
        hdr->num_q = (int32_t)a.num_q;
        hdr->batch = a.batch;
      }
    }
    if (a.fused)
      zero_other_rows(a, sw.row_info, st, kSoftThreads);
  }
  Segment seg{};
  // tokens of the segment: [k0 * 64, end), in tiles of 128
  auto seg_end = [&] { return min(seg.pos + 1, seg.k1 * kTile); };
  // rows of the segment: 2 if the next row is the second of a pair
  auto seg_rows = [&] { return R == 2 && seg.n + 1 < a.num_q && sw.row_info[seg.n + 1].z == -1 ? 2 : 1; };
  auto seg_tiles = [&] { return (seg_end() - seg.k0 * kTile + kTok - 1) / kTok; };
  auto warp_wait = [&](int bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_or_abort(&bars[bar], parity, abort_flag));
  };

  if (has_work && warp == 0) {
    // -------------------------------------------------------------- copies
    // tokens that only this CTA reads leave L2 first; those that other groups
    // or rows read as well stay as they are
    uint64_t policy = l2_evict_first_policy();
    if (a.groups > 1 || a.num_q > a.batch)
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    int i = 0;
    bool ok = true;
    while (ok && sw.next(seg)) {
      const int32_t* bt = a.block_table + (size_t)seg.b * a.max_blocks;
      const int end = seg_end(), n = seg_tiles();
      // lane l holds block-table entry base + l and its page's scale
      int base = -(1 << 30), id = -1;
      float sc = -1.f;
#pragma unroll 1
      for (int t = 0; t < n; ++t, ++i) {
        const int t0 = seg.k0 * kTile + t * kTok, v = min(kTok, end - t0), slot = i & 1;
        const int b0 = t0 >> bs_shift, pages = (v + bs - 1) >> bs_shift;  // at most 8
        if (b0 < base || b0 + pages > base + 32) {
          base = b0;
          id = base + lane < a.max_blocks ? bt[base + lane] : -1;
          const bool fine = id >= 0 && id < a.num_blocks;
          sc = fine ? fmaxf(a.scales[id], __uint_as_float((uint32_t)(kP8MinExp + 127) << 23)) : -1.f;
          if (!fine) id = -1;
        }
        const int src = (b0 - base + lane) & 31;
        const int my_id = __shfl_sync(0xffffffffu, id, src);
        const float my_sc = __shfl_sync(0xffffffffu, sc, src);
        const bool mine = lane < pages && my_id >= 0;
        const uint32_t okmask = __ballot_sync(0xffffffffu, mine);
        // lanes 0-4 each copy one slab of every page
        uint8_t* dst = sm + S::stage + slot * kStageB + (lane < 5 ? lane : 0) * kSlab;
        uint32_t bytes = 0;
        // 64 tokens as soon as their place is free
        for (int half = 0; half < 2; ++half) {
          ok = i < 2 || warp_wait(kEmpty + 2 * slot + half, ((i >> 1) - 1) & 1);
          if (!ok) break;
          const int p0 = half * kTile >> bs_shift, p1 = min(pages, (half + 1) * kTile >> bs_shift);
          for (int p = p0; p < p1; ++p) {
            const int y = __shfl_sync(0xffffffffu, my_id, p) << bs_shift;
            if (!((okmask >> p) & 1)) continue;
            bytes += 5 * bs * 128;
            if (lane < 4)
              tma_load_2d_hint(dst + (p << bs_shift) * 128, &codes_map, 128 * lane, y, &bars[kFull + slot], policy);
            else if (lane == 4)
              tma_load_2d_hint(dst + (p << bs_shift) * 128, &rope_map, kDc / 2, y, &bars[kFull + slot], policy);
          }
        }
        // (read by the softmax, before whose end nothing of the stage is free;
        // the copies did not wait for the scales' loads)
        if (ok && lane < 8) page_sc[slot * 8 + lane] = mine ? my_sc : -1.f;
        __syncwarp();
        if (lane == 0) {
          if (ok && __popc(okmask) != pages) set_status(status, MLA_DEV_BAD_BLOCK);
          if (ok) info[slot] = v;
          // (the barrier's one arrival comes after the copies; of a tile that is
          // given up, too: the copies so far are waited for below)
          mbar_arrive_expect_tx(&bars[kFull + slot], bytes);
        }
        __syncwarp();
        if (!ok) {
          ++i;
          break;
        }
      }
    }
    if (lane == 0) {
      if (!ok) {
        set_status(status, MLA_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      // never leave with copies in flight
      for (int slot = 0; slot < 2; ++slot) {
        const int fills = i > slot ? (i - 1 - slot) / 2 + 1 : 0;
        if (fills > 0 && !mbar_wait(&bars[kFull + slot], (fills - 1) & 1))
          set_status(status, MLA_DEV_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (has_work && warp == 1) {
    // ----------------------------------------------------- output products
    constexpr uint32_t kIdO = idesc_f8(3 * NH, 1, true, true);
    const uint64_t vdesc = tc::smem_desc(smem_u32(sm + S::stage), kSlab, 1024, tc::kSwizzle128);
    // weights: 16-byte cores of 16 columns, 8 tokens of a core group 128 bytes
    // (leading), blocks of 16 columns 2,048 bytes apart (stride), no swizzle
    const uint64_t pdesc = tc::smem_desc(smem_u32(sm + S::p), 128, 2048, 0);
    const bool leader = tc::elect_one();
    int i = 0, seg_i = 0;
    bool ok = true;
    while (ok && sw.next(seg)) {
      const int end = seg_end(), n = seg_tiles();
#pragma unroll 1
      for (int t = 0; t < n; ++t, ++i) {
        const int nks = (min(kTok, end - (seg.k0 * kTile + t * kTok)) + 31) / 32, slot = i & 1;
        if (!warp_wait(kPFull + slot, (i >> 1) & 1) ||
            (t == 0 && seg_i > 0 && !warp_wait(kOFree, (seg_i - 1) & 1))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        if (leader) {
          const uint32_t st = (uint32_t)(slot * kStageB), pb = (uint32_t)(slot * S::p_bytes);
#pragma unroll 1
          for (int ks = 0; ks < nks; ++ks) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_f8(tmem + kOCol + (uint32_t)(j * 3 * NH), vdesc + ((st + j * kSlab + ks * 4096) >> 4),
                     pdesc + ((pb + ks * 512) >> 4), kIdO, t > 0 || ks > 0);
            if (ks == min(nks, 2) - 1) tc::commit(&bars[kEmpty + 2 * slot]);
          }
          tc::commit(&bars[kEmpty + 2 * slot + 1]);
          tc::commit(&bars[kPVDone + slot]);
          if (t == n - 1) tc::commit(&bars[kODone]);
        }
        __syncwarp();
      }
      ++seg_i;
    }
    if (!ok && leader) {
      set_status(status, MLA_DEV_TIMEOUT);
      *abort_flag = 1;
    }
    // every product issued so far must finish before TMEM is freed
    if (leader) tc::commit(&bars[kFinalO]);
    __syncwarp();
    if (!mbar_wait(&bars[kFinalO], 0) && leader) set_status(status, MLA_DEV_TIMEOUT);
    __syncwarp();
  } else if (has_work && warp == 2) {
    // -------------------------------------------------------------- scores
    constexpr uint32_t kIdS = idesc_f8(2 * NH, 0, false, false);
    constexpr uint32_t kIdR = tc::idesc_bf16(kTok, NH, false, false);
    const uint64_t kdesc = tc::smem_desc(smem_u32(sm + S::stage), 16, 1024, tc::kSwizzle128);
    const uint64_t qdesc = tc::smem_desc(smem_u32(sm + S::q), 16, 1024, tc::kSwizzle128);
    const bool leader = tc::elect_one();
    int i = 0, seg_i = 0;
    bool ok = true;
    while (ok && sw.next(seg)) {
      const int n = seg_tiles(), qb = seg_i % QB;
      if (!warp_wait(kQReady + qb, (seg_i / QB) & 1)) { ok = false; break; }
#pragma unroll 1
      for (int t = 0; t < n; ++t, ++i) {
        const int slot = i & 1;
        if (!warp_wait(kFull + slot, (i >> 1) & 1) || (i > 0 && !warp_wait(kSFree, (i - 1) & 1))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        if (leader) {
          const uint32_t st = (uint32_t)(slot * kStageB), q0 = (uint32_t)(qb * S::q_bytes);
#pragma unroll
          for (int kk = 0; kk < 16; ++kk)
            mma_f8(tmem + kSCol, kdesc + ((st + (kk >> 2) * kSlab + (kk & 3) * 32) >> 4),
                   qdesc + ((q0 + (kk >> 2) * S::q_slab + (kk & 3) * 32) >> 4), kIdS, kk > 0);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma_bf16(tmem + kSCol + 2 * NH, kdesc + ((st + 4 * kSlab + kk * 32) >> 4),
                         qdesc + ((q0 + S::q_rope + kk * 32) >> 4), kIdR, kk > 0);
          tc::commit(&bars[kSFull]);
          if (t == n - 1) tc::commit(&bars[kQFree + qb]);
        }
        __syncwarp();
      }
      ++seg_i;
    }
    if (!ok && leader) {
      set_status(status, MLA_DEV_TIMEOUT);
      *abort_flag = 1;
    }
    if (leader) tc::commit(&bars[kFinalS]);
    __syncwarp();
    if (!mbar_wait(&bars[kFinalS], 0) && leader) set_status(status, MLA_DEV_TIMEOUT);
    __syncwarp();
  } else if (has_work && warp == 3) {
    // --------------------------------------------------------- query copies
    pdl_wait();
    int seg_i = 0;
    bool ok = true;
    while (ok && sw.next(seg)) {
      const int qb = seg_i % QB;
      if (seg_i >= QB && !warp_wait(kQFree + qb, ((seg_i / QB) - 1) & 1)) { ok = false; break; }
      uint64_t* bar = &bars[kQReady + qb];
      if (lane == 0) mbar_arrive_expect_tx(bar, S::q_bytes + NH * 4);
      __syncwarp();
      uint8_t* dst = sm + S::q + qb * S::q_bytes;
      if constexpr (R == 1) {
        const int64_t tile = (int64_t)seg.n * a.groups + grp;
        if (lane == 0) bulk_load(dst, a.q8 + tile * S::q_bytes, S::q_bytes, bar);
        if (lane == 1) bulk_load(coef + qb * NH, a.coef + tile * NH, NH * 4, bar);
      } else {
        // the rows' operands, each of eight (slab, term) pieces of 16 head rows
        // and one of rope values, interleaved (a single row stands in for its
        // missing second, whose columns stay masked)
        using S1 = Sm<16>;
        const int sub = lane / 9, p = lane % 9, rows = seg_rows();
        const int64_t row = seg.n + (sub < rows ? sub : 0);
        constexpr int kPiece = kHG * 128;
        if (lane < 18)
          bulk_load(dst + (p < 8 ? (p >> 1) * S::q_slab + (p & 1) * 2 * kPiece : S::q_rope) + sub * kPiece,
                    a.q8 + row * S1::q_bytes + p * kPiece, kPiece, bar);
        else if (lane < 20)
          bulk_load(coef + (lane - 18) * kHG, a.coef + (seg.n + (lane - 18 < rows ? lane - 18 : 0)) * kHG,
                    kHG * 4, bar);
      }
      __syncwarp();
      ++seg_i;
    }
    if (lane == 0) {
      if (!ok) {
        set_status(status, MLA_DEV_TIMEOUT);
        *abort_flag = 1;
      }
      // never leave with copies in flight
      for (int qb = 0; qb < QB; ++qb) {
        const int fills = seg_i > qb ? (seg_i - 1 - qb) / QB + 1 : 0;
        if (fills > 0 && !mbar_wait(&bars[kQReady + qb], (fills - 1) & 1))
          set_status(status, MLA_DEV_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (has_work) {
    // ------------------------------------------------------------- softmax
    const int st = tid - kSoftWarp0 * 32;               // 0-255
    const int sg = st >> 7, r = st & 127, w4 = (warp & 3);  // group, token, warp of the group
    const int h0 = sg * HT, c16 = h0 / kHG;                 // first column of this thread, its 16 columns
    const uint32_t trow = tmem + ((uint32_t)(w4 * 32) << 16);
    const int bar = kGroupBar + sg;
    float* red = reinterpret_cast<float*>(sm + S::red);
    float* scratch = reinterpret_cast<float*>(sm + S::merge);
    int i = 0, seg_i = 0;
    bool aborted = false;
    while (!aborted && sw.next(seg)) {
      const int n = seg_tiles(), qb = seg_i % QB;
      const int64_t tile = (int64_t)seg.n * a.groups + grp;
      // this thread's row, its first head there, and the tokens the row sees
      const int nrows = seg_rows();
      const int64_t row = seg.n + (R == 2 ? c16 : 0);
      const int head0 = R == 2 ? h0 % kHG : grp * NH + h0;
      const int seen = R == 1 ? seg.pos + 1 : c16 < nrows ? seg.pos + 2 - nrows + c16 : 0;
      // pairs of heads go through the packed fp32 instructions. nref is what is
      // added to a score to give the exponent of its weight: kRefLog2 less the
      // head's reference, and before a head has one, enough to exceed any bound
      float2 cq[HT / 2], nref[HT / 2], l[HT / 2];
      const bool okq = warp_wait(kQReady + qb, (seg_i / QB) & 1);
#pragma unroll
      for (int k = 0; k < HT / 2; ++k) {
        cq[k] = okq ? *reinterpret_cast<const float2*>(coef + qb * NH + h0 + 2 * k) : make_float2(0.f, 0.f);
        nref[k] = make_float2(kNoRef, kNoRef);
        l[k] = make_float2(0.f, 0.f);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kQFree + qb]);
#pragma unroll 1
      for (int t = 0; t < n; ++t, ++i) {
        const int slot = i & 1;
        // the scores, the stage's info, and the weights' buffer (tile i - 2)
        bool fine = okq && wait_or_abort(&bars[kSFull], i & 1, abort_flag) &&
                    wait_or_abort(&bars[kFull + slot], (i >> 1) & 1, abort_flag) &&
                    (i < 2 || wait_or_abort(&bars[kPVDone + slot], ((i >> 1) - 1) & 1, abort_flag));
        fine = __all_sync(0xffffffffu, fine);
        float2 x[HT / 2];   // score + log2 S: the base-2 logarithm of a weight as it enters the output
        int v = 0;
        bool there = false, odd = false;
        float inv_s = 1.f;
        if (fine) {
          tc::fence_after_sync();
          float d1[HT], d2[HT], dr[HT];
          tmem_ld(trow + kSCol + h0, d1);
          tmem_ld(trow + kSCol + NH + h0, d2);
          tmem_ld(trow + kSCol + 2 * NH + h0, dr);
          v = info[slot];
          float sc = page_sc[slot * 8 + (r >> bs_shift)];
          there = r < v && sc > 0.f;
          const int tok = seg.k0 * kTile + t * kTok + r;
          const bool live = there && (R == 1 || tok < seen);
          if (!live) sc = 1.f;
          // S = m 2^e, m in [1, 2): its logarithm is exact for a power of two
          const float m = __uint_as_float((__float_as_uint(sc) & 0x7fffffu) | 0x3f800000u);
          const float lg = (float)((int)(__float_as_uint(sc) >> 23) - 127) + (m == 1.f ? 0.f : log2f(m));
          inv_s = 1.f / sc;
          const float2 c32 = make_float2(0.03125f, 0.03125f), s2 = make_float2(sc, sc);
          const float2 scale2 = make_float2(a.scale_log2, a.scale_log2), lg2 = make_float2(lg, lg);
          tc::wait_ld();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kSFree]);
          if constexpr (R == 2) {
            // a token that only the second row sees, with a NaN code: all of
            // that row is NaN by its scores, and the codes must not reach the
            // first row's columns (0 times NaN). NaN scores may also be some
            // heads' query, so the codes decide. (The row's first heads zero them
            // for all.)
            odd = sg == kHG / HT && live && nrows == 2 && tok == seen - 1;
            if (odd) {
#pragma unroll
              for (int k = 0; k < HT; ++k) odd &= isnan(d1[k]);
              if (odd) odd = nan_code(sm + S::stage + slot * kStageB + r * 128);
            }
          }
#pragma unroll
          for (int k = 0; k < HT / 2; ++k) {
            const float2 d = fma_f32x2(make_float2(d2[2 * k], d2[2 * k + 1]), c32, make_float2(d1[2 * k], d1[2 * k + 1]));
            x[k] = fma_f32x2(mul_f32x2(d, s2), cq[k],
                             fma_f32x2(make_float2(dr[2 * k], dr[2 * k + 1]), scale2, lg2));
          }
          if (a.scores && live) {
            const int64_t t16 = row * (a.num_heads / kHG) + head0 / kHG;
            float4* o = reinterpret_cast<float4*>(
                a.scores + (t16 * a.max_blocks * bs + tok) * kHG + head0 % kHG);
#pragma unroll
            for (int k = 0; k < HT / 4; ++k)
              o[k] = make_float4(x[2 * k].x - lg, x[2 * k].y - lg, x[2 * k + 1].x - lg, x[2 * k + 1].y - lg);
          }
          if (!__all_sync(0xffffffffu, live)) {
#pragma unroll
            for (int k = 0; k < HT / 2; ++k)
              if (!live) x[k] = make_float2(-INFINITY, -INFINITY);
          }
        } else {
#pragma unroll
          for (int k = 0; k < HT / 2; ++k) x[k] = make_float2(-INFINITY, -INFINITY);
        }
        // does any weight outgrow its reference? (NaN does not)
        float2 y[HT / 2];
#pragma unroll
        for (int k = 0; k < HT / 2; ++k) y[k] = add_f32x2(x[k], nref[k]);
        float top = fmaxf(y[0].x, y[0].y);
#pragma unroll
        for (int k = 1; k < HT / 2; ++k) top = fmax3(top, y[k].x, y[k].y);
        uint32_t grown = 0;
        float fl = 1.f;   // lane k: what head k's sums are multiplied by
        if (bar_or(bar, 128, !fine || top > kRefLog2 + kGrowLog2)) {
          // every head's largest weight (no branches between them), lane k
          // holding head k's
          float mx = -INFINITY;
#pragma unroll
          for (int k = 0; k < HT; ++k) {
            const float m = warp_max(k & 1 ? x[k / 2].y : x[k / 2].x);
            if (lane == k) mx = m;
          }
          if (lane < HT) red[(sg * 4 + w4) * HT + lane] = mx;
          if (bar_or(bar, 128, !fine)) {
            // (the other groups meet this at the end of the segment or here)
            bar_or(kSoftBar, kSoftThreads, true);
            aborted = true;
            break;
          }
#pragma unroll
          for (int k = 0; k < HT; ++k) {
            const float* m = red + sg * 4 * HT + k;
            const float mx = fmaxf(fmaxf(m[0], m[HT]), fmaxf(m[2 * HT], m[3 * HT]));
            float& ref = k & 1 ? nref[k / 2].y : nref[k / 2].x;
            const bool grew = mx + ref > kRefLog2 + kGrowLog2;
            const float now = grew ? kRefLog2 - mx : ref;
            const float f = grew ? fast_exp2(now - ref) : 1.f;   // (from kNoRef: 0)
            (k & 1 ? l[k / 2].y : l[k / 2].x) *= f;
            ref = now;
            grown |= (uint32_t)grew << k;
            if (lane == k) fl = f;
          }
#pragma unroll
          for (int k = 0; k < HT / 2; ++k) y[k] = add_f32x2(x[k], nref[k]);
        }
        // weights 2^(s - ref) S, and the sum of 2^(s - ref)
        uint32_t hp[HT / 2];
        const float2 inv2 = make_float2(inv_s, inv_s);
#pragma unroll
        for (int k = 0; k < HT / 2; ++k) {
          const float2 p = make_float2(fast_exp2(y[k].x), fast_exp2(y[k].y));
          l[k] = fma_f32x2(p, inv2, l[k]);
          const __half2 hh = __floats2half2_rn(p.x, p.y);
          hp[k] = *reinterpret_cast<const uint32_t*>(&hh);
        }
        // as three e5m2 terms. e5m2 is the upper byte of f16: the first two are
        // rounded to the nearest (half a step added, the lower byte dropped), so
        // each leaves at most 2^-3 of what it was given, of either sign, and the
        // third, times 2^5, holds all that is left of the f16
        uint32_t tm[3][HT / 4];
#pragma unroll
        for (int k = 0; k < HT / 2; k += 2) {
          uint32_t a0 = hp[k], a1 = hp[k + 1];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            // (0x7fff, the NaN, is 0 here and NaN in the last term)
            const uint32_t c0 = (a0 + 0x00800080u) & 0xff00ff00u, c1 = (a1 + 0x00800080u) & 0xff00ff00u;
            tm[s][k / 2] = __byte_perm(c0, c1, 0x7531);
            const __half2 r0 = __hsub2(*reinterpret_cast<const __half2*>(&a0), *reinterpret_cast<const __half2*>(&c0));
            const __half2 r1 = __hsub2(*reinterpret_cast<const __half2*>(&a1), *reinterpret_cast<const __half2*>(&c1));
            a0 = *reinterpret_cast<const uint32_t*>(&r0);
            a1 = *reinterpret_cast<const uint32_t*>(&r1);
          }
          const __half2 f = __floats2half2_rn(32.f, 32.f);
          const __half2 m0 = __hmul2(*reinterpret_cast<const __half2*>(&a0), f);
          const __half2 m1 = __hmul2(*reinterpret_cast<const __half2*>(&a1), f);
          uint16_t e0, e1;
          asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(e0) : "r"(*reinterpret_cast<const uint32_t*>(&m0)));
          asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(e1) : "r"(*reinterpret_cast<const uint32_t*>(&m1)));
          tm[2][k / 2] = (uint32_t)e0 | ((uint32_t)e1 << 16);
        }
        uint8_t* pb = sm + S::p + slot * S::p_bytes + (r >> 3) * 128 + (r & 7) * 16;
#pragma unroll
        for (int s = 0; s < 3; ++s)
          *reinterpret_cast<uint2*>(pb + (s * (NH / kHG) + c16) * 2048 + h0 % kHG) = make_uint2(tm[s][0], tm[s][1]);
        if (t > 0 && grown) {
          // the output columns of the heads that grew, two heads at a time, when
          // the products of tile i - 1 have landed (which takes as long as the
          // weights above)
          if (warp_wait(kPVDone + (slot ^ 1), ((i - 1) >> 1) & 1)) {
            tc::fence_after_sync();
            while (grown) {
              const int k0 = __ffs(grown) - 1;
              grown &= grown - 1;
              const int k1 = grown ? __ffs(grown) - 1 : k0;
              grown &= grown - 1;
              const float f0 = __shfl_sync(0xffffffffu, fl, k0), f1 = __shfl_sync(0xffffffffu, fl, k1);
              const uint32_t at0 = trow + kOCol + (uint32_t)(h0 + k0), at1 = trow + kOCol + (uint32_t)(h0 + k1);
              float o0[12], o1[12];
#pragma unroll
              for (int c = 0; c < 12; ++c) {
                tmem_ld1(at0 + c * NH, o0[c]);
                tmem_ld1(at1 + c * NH, o1[c]);
              }
              tc::wait_ld();
#pragma unroll
              for (int c = 0; c < 12; ++c) {
                tmem_st1(at0 + c * NH, o0[c] * f0);
                if (k1 != k0) tmem_st1(at1 + c * NH, o1[c] * f1);
              }
            }
            tc::wait_st();
          } else if (lane == 0) {
            // (all groups leave at their next wait or at the segment's end)
            set_status(status, MLA_DEV_TIMEOUT);
            *abort_flag = 1;
          }
        }
        if ((!there && r < ((v + 31) & ~31)) || odd) {
          // a token that is not there may hold anything: zero its codes, so that
          // a weight of 0 stays 0 (each group its part of the four slabs)
          constexpr int kSlabs = 4 / S::groups;
          uint8_t* tok_row = sm + S::stage + slot * kStageB + (odd ? 0 : kSlabs * sg) * kSlab + r * 128;
#pragma unroll 1
          for (int c = 0; c < (odd ? 32 : 8 * kSlabs); ++c)
            *reinterpret_cast<uint4*>(tok_row + (c >> 3) * kSlab + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kPFull + slot]);
      }
      if (aborted) break;

      // ---- the segment's sums, then its output rows
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
        for (int k = 0; k < HT / 2; ++k) {
          l[k].x += __shfl_xor_sync(0xffffffffu, l[k].x, o);
          l[k].y += __shfl_xor_sync(0xffffffffu, l[k].y, o);
        }
      }
      const bool okd = warp_wait(kODone, seg_i & 1);
      if (bar_or(kSoftBar, kSoftThreads, !okd)) { aborted = true; break; }
      tc::fence_after_sync();
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < HT / 2; ++k) *reinterpret_cast<float2*>(red + (sg * 4 + w4) * HT + 2 * k) = l[k];
      }
      named_bar_sync(bar, 128);
      const int c_first = seg.ustart / sw.share, c_last = (seg.ustart + seg.tiles - 1) / sw.share;
      const bool direct = a.fused && c_first == c_last;
      const int64_t slot = (int64_t)share + seg.n;
      const int t16 = R == 2 ? c16 : head0 / kHG, hr = head0 % kHG;  // which partials, head in them
      float* dst = (direct ? a.o_lat + ((size_t)row * a.num_heads + head0) * kDc
                           : o_part(a, t16) + (slot * kHG + hr) * kDc) +
                   w4 * 32 + lane;
      const bool mine_too = R == 1 || c16 < nrows;   // (a pair's missing second row)
      // (all of a row's loads before the first is used)
      float o1[2][HT], o2[2][HT], o3[2][HT];
      auto load_o = [&](int j) {
        const uint32_t at = trow + kOCol + (uint32_t)(j * 3 * NH + h0);
        tmem_ld(at, o1[j & 1]);
        tmem_ld(at + NH, o2[j & 1]);
        tmem_ld(at + 2 * NH, o3[j & 1]);
      };
      load_o(0);
      float mine = 0.f, mref = 0.f, inv[HT];
#pragma unroll
      for (int k = 0; k < HT; ++k) {
        const float sum = (red[sg * 4 * HT + k] + red[(sg * 4 + 1) * HT + k]) +
                          (red[(sg * 4 + 2) * HT + k] + red[(sg * 4 + 3) * HT + k]);
        if (r == k) mine = sum, mref = k & 1 ? nref[k / 2].y : nref[k / 2].x;
        inv[k] = sum == 0.f ? 0.f : __fdividef(1.f, sum);       // (a NaN sum stays NaN)
      }
      if (r < HT && mine_too) {
        const float lse = mine == 0.f ? -INFINITY : log2f(mine) - mref;
        if (direct)
          a.lse[(size_t)row * a.num_heads + head0 + r] = lse;
        else
          lse_part(a, t16)[slot * kHG + hr + r] = lse;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        tc::wait_ld();
        if (j < 3) load_o(j + 1);
        if (!mine_too) continue;
#pragma unroll
        for (int k = 0; k < HT; ++k)
          dst[(size_t)k * kDc + j * 128] = fmaf(o3[j & 1][k], 0.03125f, o1[j & 1][k] + o2[j & 1][k]) * inv[k];
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kOFree]);
      if (a.fused && !direct) {
        __threadfence();  // publish protocol: see count_arrival
        named_bar_sync(kSoftBar, kSoftThreads);
        if (st == 0) *merge_flag = count_arrival(&a.arrive[tile]) == c_last - c_first;
        named_bar_sync(kSoftBar, kSoftThreads);
        if (*merge_flag) {
          const int parts = c_last - c_first + 1;
          // merge_qtile leaves the maxima and the inverse weight sums in its scratch
          // (16 heads by the 256 threads that have them)
          if (mine_too) {
            float* own = scratch + c16 * (S::merge_bytes / 4);
            const int ht = st & 255, hb = head0 - h0 % kHG;
            merge_qtile<256>(lse_part(a, t16), o_part(a, t16), (int64_t)c_first + seg.n, parts, 1,
                             a.o_lat + ((size_t)row * a.num_heads + hb) * kDc, ht, own,
                             [&] { named_bar_sync(kHeadsBar + c16, 256); });
            if (ht < kHG)
              a.lse[(size_t)row * a.num_heads + hb + ht] =
                  merged_lse(own[ht], own[kHG + ht], lse_part(a, t16) + ((int64_t)c_first + seg.n) * kHG + ht, parts);
          }
        }
      }
      named_bar_sync(kSoftBar, kSoftThreads);  // red and the scratch may be written again
      ++seg_i;
    }
    if (aborted && lane == 0) {
      set_status(status, MLA_DEV_TIMEOUT);
      *abort_flag = 1;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::dealloc(tmem, kTmemCols);
}

// The parts of (row n, head h), from the row's entry of the plan: its 16
// heads' partials, one slot after another.
struct HeadParts {
  const float* lse;   // of the head, kHG apart
  const float* o;     // [512] of the head, kHG * 512 apart
  int count;
};
__device__ __forceinline__ HeadParts head_parts(const P8Args& a, const int4* rows, int share, int n, int h) {
  HeadParts r{a.lse_first, a.o_first, 0};
  int4 ri = rows[n];
  int t16 = h / kHG;
  if (ri.z == -1 && n > 0) ri = rows[--n], t16 = 1;  // the second row of a pair
  if (ri.z <= 0) return r;
  const int cf = ri.w / share, cl = (ri.w + ri.z - 1) / share;
  const int64_t slot = ((int64_t)cf + n) * kHG + h % kHG;
  r.lse = lse_part(a, t16) + slot;
  r.o = o_part(a, t16) + slot * kDc;
  r.count = cl - cf + 1;
  return r;
}
// 2^lse sums: the largest log-sum-exp m, and den = sum of 2^(lse - m), by a
// group of G neighbouring lanes. (fmaxf passes NaN over, the sum does not: den is
// NaN where a part's is, and 0 only where no part has a token.)
template <int G>
__device__ __forceinline__ void merge_weights(const HeadParts& hp, int lane_in_group, float& m, float& den) {
  m = -INFINITY;
  for (int s = lane_in_group; s < hp.count; s += G) m = fmaxf(m, hp.lse[s * kHG]);
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  den = 0.f;
  const float base = m == -INFINITY ? 0.f : m;
  for (int s = lane_in_group; s < hp.count; s += G) den += fast_exp2(hp.lse[s * kHG] - base);
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
}

// The merge of many parts of few (row, head)s: two CTAs each, of 256 columns.
// Thread (p, c) sums 4 columns over every fourth part, eight loads in flight;
// the four sums meet in shared memory. Bound by latency: 5.6 us for one row of 16
// heads, 9.6 us for two rows of 32 heads in 76 parts each (10 MB).
__global__ void __launch_bounds__(256) page8_merge_kernel(const __grid_constant__ P8Args a) {
  __shared__ float4 sAcc[3][64];
  __shared__ int4 plan[kSelfMaxRows];
  __shared__ int plan_total;
  const int n = blockIdx.x / a.num_heads, h = blockIdx.x % a.num_heads, tid = threadIdx.x;
  const int p = tid >> 6, c = blockIdx.y * 64 + (tid & 63);
  const int4* rows = reinterpret_cast<const int4*>(a.ws + ws_layout(a.num_q, 1, a.shares).row_info);
  int share;
  if (a.self_plan) {  // (as in the projection below: known before the wait)
    for (int i = tid; i < (int)a.num_q; i += 256) plan[i] = make_int4(-1, -1, 0, 0);
    __syncthreads();
    fill_rows(a, plan, nullptr, tid, 256, 0, 1);
    __syncthreads();
    if (tid < 32) scan_rows(plan, (int)a.num_q, tid, &plan_total);
    __syncthreads();
    share = plan_total > 0 ? (plan_total + a.shares - 1) / a.shares : 1;
    rows = plan;
    pdl_wait();
  } else {
    pdl_wait();
    share = reinterpret_cast<const WsHeader*>(a.ws)->share;
  }
  pdl_launch_dependents();
  const HeadParts hp = head_parts(a, rows, share, n, h);
  float4 v[8];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (s0 + 4 * u < hp.count)
        v[u] = *reinterpret_cast<const float4*>(hp.o + (size_t)(s0 + 4 * u) * kHG * kDc + 4 * c);
  };
  load(p);  // on their way while the weights are found
  float m, den;
  merge_weights<32>(hp, tid & 31, m, den);
  const float inv = den == 0.f ? 0.f : 1.f / den, b = m == -INFINITY ? 0.f : m;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int s0 = p; s0 < hp.count; s0 += 32) {
    if (s0 != p) load(s0);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (s0 + 4 * u < hp.count) {
        const float w = fast_exp2(hp.lse[(s0 + 4 * u) * kHG] - b) * inv;
        acc.x = fmaf(w, v[u].x, acc.x);
        acc.y = fmaf(w, v[u].y, acc.y);
        acc.z = fmaf(w, v[u].z, acc.z);
        acc.w = fmaf(w, v[u].w, acc.w);
      }
  }
  if (p > 0) sAcc[p - 1][tid & 63] = acc;
  __syncthreads();
  if (p == 0) {
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      const float4 x = sAcc[u][tid];
      acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
    }
    const size_t row = (size_t)n * a.num_heads + h;
    *reinterpret_cast<float4*>(a.o_lat + row * kDc + 4 * c) = acc;
    if (c == 0) a.lse[row] = den == 0.f ? -INFINITY : m + log2f(den);
  }
}

// The merge of a few parts and the output projection in one: CTA = (ROWS rows,
// head h). W_uv[h] (128 KB) comes by cp.async while 256 / ROWS threads a row
// merge its 512 latents to two bf16 terms each (one would add as much error as
// the rounding of the output); then 8 warps, each a quarter of K and half of the
// columns (m16n8k16), whose sums meet in shared memory. Every part is read once.
// MERGED: one part a row, merged before. ROWS = 8 (the second terms are the mma's
// other rows) where that still leaves at most one CTA an SM: the merge, at
// latency, is what takes the time. 64 rows of 16 heads: 9.0 us alone, 4 us behind a decode,
// which hides the weights' copy (2 MB in all); 32 rows of 128 heads: 18 us.
template <int ROWS>
struct Mp {
  static constexpr int stride = kDc * 2 + 16;     // bytes of a merged row, padded against bank conflicts
  static constexpr int w = 0;                     // two halves of 64 columns, 128-byte rows
  static constexpr int a = w + kDc * 256;
  static constexpr int red = a + 2 * ROWS * stride;  // [4][ROWS][128]
  static constexpr int rows = red + 4 * ROWS * kDv * 4;
  static constexpr int bytes = rows + kSelfMaxRows * 16 + 16;
};
template <int ROWS, bool MERGED>
__global__ void __launch_bounds__(256) page8_merge_proj_kernel(const __grid_constant__ P8Args a,
                                                               const __nv_bfloat16* W_uv,
                                                               __nv_bfloat16* out) {
  using M = Mp<ROWS>;
  constexpr int kTr = 256 / ROWS, kVec = kDc / 4 / kTr, kBatch = 16 / kVec;  // threads, float4s, parts at a time
  extern __shared__ __align__(1024) uint8_t smem_mp[];
  float* sRed = reinterpret_cast<float*>(smem_mp + M::red);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, row0 = blockIdx.x * ROWS, H = a.num_heads;
  int4* plan = reinterpret_cast<int4*>(smem_mp + M::rows);
  int* plan_total = reinterpret_cast<int*>(smem_mp + M::rows + kSelfMaxRows * 16);
  if (a.self_plan && !MERGED)
    for (int n = tid; n < (int)a.num_q; n += 256) plan[n] = make_int4(-1, -1, 0, 0);
  const __nv_bfloat16* src = W_uv + (size_t)h * kDc * kDv;
#pragma unroll 4
  for (int i = tid; i < kDc * 16; i += 256) {
    const int k = i >> 4, c = i & 15;
    cp_async16(smem_mp + M::w + (c >> 3) * (kDc * 128) + sw128(k, c & 7), src + (size_t)k * kDv + c * 8);
  }
  cp_async_commit();
  // The weights do not depend on earlier kernels, and where the parts lie is
  // known from the lengths (the split of the decode, derived again); the parts
  // themselves have to be waited for.
  const int4* rows = reinterpret_cast<const int4*>(a.ws + ws_layout(a.num_q, 1, a.shares).row_info);
  int share = 1;
  if (a.self_plan && !MERGED) {
    __syncthreads();
    fill_rows(a, plan, nullptr, tid, 256, 0, 1);
    __syncthreads();
    if (warp == 0) scan_rows(plan, (int)a.num_q, lane, plan_total);
    __syncthreads();
    share = *plan_total > 0 ? (*plan_total + a.shares - 1) / a.shares : 1;
    rows = plan;
    pdl_wait();
  } else {
    pdl_wait();
    share = reinterpret_cast<const WsHeader*>(a.ws)->share;
  }
  pdl_launch_dependents();
  {
    const int r = tid / kTr, j = tid % kTr, n = row0 + r;
    HeadParts hp{a.lse_first, a.o_first, 0};
    if (n < a.num_q)
      hp = MERGED ? HeadParts{nullptr, a.o_lat + ((size_t)n * H + h) * kDc, 1} : head_parts(a, rows, share, n, h);
    float4 v[kBatch][kVec];
    auto load = [&](int s0) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (s0 + u < hp.count) {
#pragma unroll
          for (int k = 0; k < kVec; ++k)
            v[u][k] = *reinterpret_cast<const float4*>(hp.o + (size_t)(s0 + u) * kHG * kDc + 4 * (j + kTr * k));
        }
    };
    load(0);  // on their way while the weights are found
    float m = 0.f, den = 1.f;
    if (!MERGED) merge_weights<kTr>(hp, j, m, den);
    const float inv = den == 0.f ? 0.f : 1.f / den, b = m == -INFINITY ? 0.f : m;
    if (!MERGED && j == 0 && n < a.num_q) a.lse[(size_t)n * H + h] = den == 0.f ? -INFINITY : m + log2f(den);
    float4 acc[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int s0 = 0; s0 < hp.count; s0 += kBatch) {
      if (s0 > 0) load(s0);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (s0 + u < hp.count) {
          const float w = MERGED ? 1.f : fast_exp2(hp.lse[(s0 + u) * kHG] - b) * inv;
#pragma unroll
          for (int k = 0; k < kVec; ++k) {
            acc[k].x = fmaf(w, v[u][k].x, acc[k].x);
            acc[k].y = fmaf(w, v[u][k].y, acc[k].y);
            acc[k].z = fmaf(w, v[u][k].z, acc[k].z);
            acc[k].w = fmaf(w, v[u][k].w, acc[k].w);
          }
        }
    }
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const uint32_t t0 = pack_bf16(acc[k].x, acc[k].y), t1 = pack_bf16(acc[k].z, acc[k].w);
      auto low = [](uint32_t t) { return __uint_as_float(t << 16); };
      auto high = [](uint32_t t) { return __uint_as_float(t & 0xffff0000u); };
      uint8_t* at = smem_mp + M::a + r * M::stride + (j + kTr * k) * 8;
      *reinterpret_cast<uint2*>(at) = make_uint2(t0, t1);
      *reinterpret_cast<uint2*>(at + ROWS * M::stride) =
          make_uint2(pack_bf16(acc[k].x - low(t0), acc[k].y - high(t0)),
                     pack_bf16(acc[k].z - low(t1), acc[k].w - high(t1)));
    }
  }
  cp_async_wait_all();
  __syncthreads();
  const int g = lane >> 2, q = lane & 3, kq = warp >> 1, nh = warp & 1;
  const uint8_t* sW = smem_mp + M::w + nh * (kDc * 128);
  float acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    const int k = kq * 128 + ks * 16;
    // row g + 8: of the second terms, or a row of its own
    const uint8_t* lo = smem_mp + M::a + g * M::stride + (k + 2 * q) * 2;
    auto frag = [&](int row, int at) { return *reinterpret_cast<const uint32_t*>(lo + row * M::stride + at); };
    const uint32_t a0 = frag(0, 0), a1 = frag(8, 0), a2 = frag(0, 16), a3 = frag(8, 16);
    uint32_t c0 = 0, c1 = 0, c2 = 0, c3 = 0;
    if (ROWS == 16) c0 = frag(16, 0), c1 = frag(24, 0), c2 = frag(16, 16), c3 = frag(24, 16);
    const int kr = k + (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(smem_u32(sW + sw128(kr, np * 2 + (lane >> 4))), b0, b1, b2, b3);
      mma_16816(acc[2 * np], a0, a1, a2, a3, b0, b1);
      mma_16816(acc[2 * np + 1], a0, a1, a2, a3, b2, b3);
      if (ROWS == 16) {
        mma_16816(acc[2 * np], c0, c1, c2, c3, b0, b1);
        mma_16816(acc[2 * np + 1], c0, c1, c2, c3, b2, b3);
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < 8; ++nt) {
    float* d = sRed + (kq * ROWS + g) * kDv + nh * 64 + nt * 8 + 2 * q;
    if (ROWS == 16) {
      *reinterpret_cast<float2*>(d) = make_float2(acc[nt][0], acc[nt][1]);
      *reinterpret_cast<float2*>(d + 8 * kDv) = make_float2(acc[nt][2], acc[nt][3]);
    } else {
      *reinterpret_cast<float2*>(d) = make_float2(acc[nt][0] + acc[nt][2], acc[nt][1] + acc[nt][3]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = tid; i < ROWS * kDv / 4; i += 256) {
    const int r = i / (kDv / 4), c = (i % (kDv / 4)) * 4, row = row0 + r;
    if (row >= a.num_q) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(sRed + (k * ROWS + r) * kDv + c);
      v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    *reinterpret_cast<uint2*>(out + ((size_t)row * H + h) * kDv + c) =
        make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  }
}

// mass[slot(t)] = decay * mass[slot(t)] + sum over the sequence's rows and all
// heads of 2^(score - lse), in a fixed order: P neighbouring threads per token, each
// with every P-th (row, 16 heads). Bound by latency and the scores' bytes: 8.7 us
// for 64 sequences of 4,096 tokens and 16 heads (16.8 MB, most of it still in L2).
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
template <int P>
__global__ void __launch_bounds__(256) page8_mass_kernel(MassArgs a) {
  // (what the caller gave and the old mass are there, see page8_decode_kernel;
  // the scores and sums have to be waited for)
  const int b = blockIdx.y, t = blockIdx.x * (256 / P) + threadIdx.x / P, part = threadIdx.x % P;
  const int len = a.seq_lens[b], q0 = a.query_start_loc[b], q1 = a.query_start_loc[b + 1];
  const int ql = q1 - q0;
  const int64_t max_tokens = (int64_t)a.max_blocks * a.block_size;
  bool mine = q0 >= 0 && q1 <= a.num_q && ql > 0 && ql <= len && (int64_t)len <= max_tokens && t < len;
  float* m = a.mass;
  float old = 0.f;
  if (mine) {
    const int32_t p = a.block_table[(size_t)b * a.max_blocks + t / a.block_size];
    mine = p >= 0 && p < a.num_blocks;
    if (mine) {
      m += (size_t)p * a.block_size + t % a.block_size;
      if (a.decay > 0.f) old = a.decay * *m;
    }
  }
  pdl_wait();
  pdl_launch_dependents();
  float sum = 0.f;
  if (mine) {
    // rows at or behind token t (of at most 48 * 1,024, of 8 groups each)
    const int end = q1 * a.groups;
#pragma unroll 2
    for (int tile = max(q0, q0 + t - (len - ql)) * a.groups + part; tile < end; tile += P) {
      const float4* s = reinterpret_cast<const float4*>(a.scores + (tile * max_tokens + t) * kHG);
      const float4* e = reinterpret_cast<const float4*>(a.lse + (size_t)tile * kHG);
#pragma unroll
      for (int k = 0; k < kHG / 4; ++k) {
        const float4 x = s[k], y = e[k];
        sum += (fast_exp2(x.x - y.x) + fast_exp2(x.y - y.y)) + (fast_exp2(x.z - y.z) + fast_exp2(x.w - y.w));
      }
    }
  }
#pragma unroll
  for (int o = 1; o < P; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (mine && part == 0) *m = old + sum;
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
  const int H = cfg->num_heads, bs = cfg->block_size, C = split_ctas(cfg);
  if (!p8_sizes_fit(num_q, max_blocks, bs) || C <= 0) return MLA_ERR_UNSUPPORTED;
  const bool pair = use_pairs(H, num_q, batch);
  const int NH = pair ? 32 : group_heads(H);
  const int shares = p8_shares(H, C);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const P8Ws L = p8_ws(num_q, H, shares, (int64_t)max_blocks * bs, with_mass);
  if (ws_bytes < L.total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  const WsLayout W = ws_layout(num_q, 1, shares);
  // With num_blocks == 0 every block id is rejected before any copy; the maps
  // still need an extent.
  CUtensorMap codes_map, rope_map;
  if (!encode_fp8_maps(&codes_map, &rope_map, cache8,
                       (uint64_t)(num_blocks > 0 ? num_blocks : 1) * bs, (uint32_t)bs))
    return MLA_ERR_CUDA;
  P8Args a{};
  a.q_abs = (const uint16_t*)q_abs;
  a.scales = page_scales;
  a.num_blocks = num_blocks;
  a.block_table = block_table;
  a.max_blocks = max_blocks;
  a.block_size = bs;
  a.num_heads = H;
  a.groups = pair ? 1 : H / NH;
  a.pair = pair;
  a.shares = shares;
  a.num_q = num_q;
  a.scale_log2 = (float)(cfg->softmax_scale * 1.4426950408889634);
  a.ws = ws;
  a.q8 = ws + L.q8;
  a.coef = reinterpret_cast<float*>(ws + L.coef);
  a.seq_lens = seq_lens;
  a.query_start_loc = query_start_loc;
  a.batch = batch;
  // (64 rows of 16 heads: 21.9 us, 25.3 with the plan in the kernel before; 256
  // rows: 49.0 and 57.7; 128 rows of 32 heads: 39.4 and 42.0)
  a.self_plan = num_q <= (NH == 16 ? Sm<16>::self_rows : Sm<32>::self_rows);
  a.lse_first = reinterpret_cast<float*>(ws + W.lse);
  a.o_first = reinterpret_cast<float*>(ws + W.opart);
  a.lse_rest = reinterpret_cast<float*>(ws + L.lse_rest);
  a.o_rest = reinterpret_cast<float*>(ws + L.o_rest);
  a.slots = W.slots;
  a.arrive = reinterpret_cast<int*>(ws + L.arrive);
  a.o_lat = reinterpret_cast<float*>(ws + L.o_lat);
  a.lse = reinterpret_cast<float*>(ws + L.lse);
  a.scores = with_mass ? reinterpret_cast<float*>(ws + L.scores) : nullptr;
  // Who merges the splits. With many outputs (rows x heads) most tiles are
  // whole and the rest is merged in the decode kernel; the tensor-core
  // projection follows. Below, the merge goes into the projection, unless there
  // are so few outputs, each cut into more than a few parts (one per 64 tokens at
  // the most), that the merge has to spread over the device first. Measured on
  // one GB300, us:
  //   rows x heads       320 x 16  448 x 16  56 x 128  256 x 32  256 x 128  (1,024 tokens)
  //   in the projection    72.3      93.3      61.1      75.1      223.5
  //   in the decode        73.8      88.4      54.7      73.1      178.1
  //   rows x heads (65,536 tokens)  1 x 16  8 x 16  16 x 16  32 x 16  1 x 128  4 x 128
  //   in the projection              61.1    27.4    24.9     23.2      52.5     45.7
  //   spread                         26.6    23.6    25.2     28.5      46.8     51.2
  //   tokens of 2 x 32       512   1,024  2,048
  //   in the projection      14.6   16.3   20.3  (one launch less: 2.7 us of the host's time)
  //   spread                 15.6   15.7   15.4
  const bool many_parts = num_q * H < 256 && (int64_t)max_blocks * bs > 512;
  a.fused = num_q * H >= 7168;
  const bool merge_proj = !a.fused && !many_parts;
  cudaError_t e;
  // (a row of a pair has its operand as 16 heads by themselves do)
  const dim3 query_ctas((unsigned)(num_q * a.groups + !a.self_plan));
  e = H == 16 ? launch_pdl(page8_query_kernel<16>, query_ctas, dim3(256), 0, st, a)
              : launch_pdl(page8_query_kernel<32>, query_ctas, dim3(512), 0, st, a);
  if (e != cudaSuccess) return MLA_ERR_CUDA;
  auto launch = [&](auto kernel, int threads, int smem) {
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return r != cudaSuccess
               ? r
               : launch_pdl(kernel, dim3(shares * a.groups), dim3(threads), smem, st, codes_map, rope_map, a);
  };
  e = pair       ? launch(page8_decode_kernel<32, 2>, Sm<32>::threads, Sm<32>::alloc)
      : NH == 16 ? launch(page8_decode_kernel<16, 1>, Sm<16>::threads, Sm<16>::alloc)
                 : launch(page8_decode_kernel<32, 1>, Sm<32>::threads, Sm<32>::alloc);
  if (e == cudaSuccess && many_parts)
    e = launch_pdl(page8_merge_kernel, dim3((unsigned)(num_q * H), 2), dim3(256), 0, st, a);
  auto project = [&](auto kernel, int rows, int smem) {
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return r != cudaSuccess ? r
                            : launch_pdl(kernel, dim3((unsigned)((num_q + rows - 1) / rows), H), dim3(256), smem,
                                         st, a, (const __nv_bfloat16*)W_uv, (__nv_bfloat16*)out);
  };
  if (e == cudaSuccess && merge_proj) {
    // (40 rows of 16 heads: 24.3 us by 8, 25.9 by 16; 96 rows: 40.3 and 36.4)
    e = (num_q + 7) / 8 * H <= (int64_t)shares * a.groups
            ? project(page8_merge_proj_kernel<8, false>, 8, Mp<8>::bytes)
            : project(page8_merge_proj_kernel<16, false>, 16, Mp<16>::bytes);
  }
  if (e != cudaSuccess) return MLA_ERR_CUDA;
  if (with_mass) {
    const MassArgs ma{a.scores, a.lse, seq_lens, query_start_loc, block_table, max_blocks, bs,
                      H / kHG, num_q, num_blocks, decay, mass};
    const int64_t tokens = (int64_t)max_blocks * bs;
    if (tokens > 0) {
      auto launch_mass = [&](auto kernel, int per_token) {
        return launch_pdl(kernel, dim3((unsigned)((tokens * per_token + 255) / 256), (unsigned)batch), dim3(256), 0,
                          st, ma);
      };
      // A warp a token from 8 (row, 16 heads) of a sequence on. By thread / by warp,
      // us of the whole call: 64 x 4,096, 16 heads, 1 row 47.1 / 108; 16 x 4,096, 64
      // heads, 1 row 42.9 / 54.3; 8 x 2,048, 128 heads, 1 row 36.0 / 33.6; 8 x 1,000, 16
      // heads, 16 rows 41.9 / 34.5; 4 x 2,560, 16 heads, 512 rows 3,157 / 659.
      e = num_q * (H / kHG) >= 8 * (int64_t)batch ? launch_mass(page8_mass_kernel<32>, 32)
                                                  : launch_mass(page8_mass_kernel<1>, 1);
      if (e != cudaSuccess) return MLA_ERR_CUDA;
    }
  }
  if (merge_proj) return MLA_OK;
  if (many_parts)
    return project(page8_merge_proj_kernel<8, true>, 8, Mp<8>::bytes) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
  // Two terms a latent, as in the projection above: the output is rounded once
  // whichever form a call takes. (Few rows too: 100 rows of 128 heads 60.0 us, 70.9
  // by the projection above, of merged latents; 224 of 32 heads 51.7 and 51.8.)
  CUtensorMap w_map;
  if (!encode_map_2d(&w_map, W_uv, kDv, (uint64_t)H * kDc, 64, 64)) return MLA_ERR_CUDA;
  return launch_out_proj_tc(w_map, a.o_lat, out, num_q, H, true, st) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_page8_decode_workspace_size(const mla_config* cfg, int64_t num_q, int32_t batch,
                                       int32_t max_blocks_per_seq, int32_t with_mass) {
  if (validate_config(cfg) != MLA_OK || cfg->dtype != MLA_BF16 || num_q < 0 || batch < 0 ||
      max_blocks_per_seq < 0 || !p8_sizes_fit(num_q, max_blocks_per_seq, cfg->block_size))
    return 0;
  const int C = split_ctas(cfg), H = cfg->num_heads;
  if (C <= 0) return 0;
  return p8_ws(num_q, H, p8_shares(H, C), (int64_t)max_blocks_per_seq * cfg->block_size, with_mass != 0).total;
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
