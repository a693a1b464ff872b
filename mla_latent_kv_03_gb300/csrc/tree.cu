// A speculative step's small operators over a tree of drafted tokens:
//   mla_tree_plan     parents -> positions, ancestor masks, cache slots
//   mla_tree_verify   which path the target accepts, and the token behind it
//   mla_tree_commit   the accepted rows moved behind the past in every layer
// (mla_tree_decode, the attention between them, is in tree_decode.cu.)
#include "async_copy.cuh"
#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kTreeRows = 1024;   // rows of one tree at the most
constexpr int kMaxWords = kTreeRows / 64;

bool t_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ------------------------------------------------------------------------ plan
// One CTA a sequence, a thread a row. The mask of a row is found by doubling:
// after k rounds it holds 2^k rows on the way up and `jump` is the row above
// them, so a chain of 1,024 takes 10 rounds. The words lie word by word, so that a
// warp's rows are in different banks, and a row has none behind its own. Bound by
// latency: 8 us for 256 trees of 333 rows (11.4 with the words row by row), and for
// masks of one word, in a kernel of their own, 3 us for 64 of 8 (5.2 in the wide one).
struct PlanTreeArgs {
  const int32_t* parents;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  const int32_t* block_table;
  int32_t max_blocks, block_size, words;
  int64_t num_blocks, num_q;
  uint64_t* mask;
  int32_t* positions;
  int64_t* slots;
  uint32_t* status;
};

template <int MAXW>
__global__ void __launch_bounds__(64 * MAXW) tree_plan_kernel(const __grid_constant__ PlanTreeArgs a) {
  extern __shared__ uint64_t sAnc[];                                  // [words][64 * words + 1]
  const int W = MAXW == 1 ? 1 : a.words, i = threadIdx.x, b = blockIdx.x, pitch = 64 * W + 1;
  int* sJump = reinterpret_cast<int*>(sAnc + (size_t)W * pitch);      // [64 * words]
  int* sDepth = sJump + 64 * W;
  pdl_wait();
  pdl_launch_dependents();
  const int q0 = a.query_start_loc[b], q1 = a.query_start_loc[b + 1], len = a.seq_lens[b];
  if (q0 < 0 || q1 > a.num_q || q1 < q0) {
    if (i == 0) set_status(a.status, MLA_DEV_BAD_SEQ);
    return;
  }
  const int ql = q1 - q0;
  if (ql == 0) return;
  bool bad = ql > len || ql > 64 * W || (int64_t)len > (int64_t)a.max_blocks * a.block_size;
  int up = -1;
  if (!bad && i < ql) {
    up = a.parents[q0 + i];
    bad = up < -1 || up >= i;
  }
  if (__syncthreads_or(bad)) {
    if (i == 0) set_status(a.status, MLA_DEV_BAD_SEQ);
    for (int j = i; j < ql; j += blockDim.x) {
      for (int w = 0; w < W; ++w) a.mask[(size_t)(q0 + j) * W + w] = 0;
      a.positions[q0 + j] = 0;
      a.slots[q0 + j] = -1;
    }
    return;
  }
  const bool live = i < ql;
  if (live) {
    for (int w = 0; w < W; ++w) sAnc[w * pitch + i] = w == i >> 6 ? 1ull << (i & 63) : 0ull;
    sJump[i] = up;
    sDepth[i] = up >= 0;
  }
  int more = __syncthreads_or(live && up >= 0);
  while (more) {
    uint64_t t[MAXW];
    int nj = -1, nd = 0;
    if (live && up >= 0) {
#pragma unroll
      for (int w = 0; w < MAXW; ++w)
        if (w <= up >> 6) t[w] = sAnc[w * pitch + up];     // (none behind its own)
      nj = sJump[up];
      nd = sDepth[up];
    }
    __syncthreads();
    if (live && up >= 0) {
#pragma unroll
      for (int w = 0; w < MAXW; ++w)
        if (w <= up >> 6) sAnc[w * pitch + i] |= t[w];
      sJump[i] = up = nj;
      sDepth[i] += nd;
    }
    more = __syncthreads_or(live && up >= 0);
  }
  if (MAXW > 1)     // word by word as they lie
    for (int k = i; k < ql * W; k += blockDim.x) a.mask[(size_t)q0 * W + k] = sAnc[(k % W) * pitch + k / W];
  if (!live) return;
  if (MAXW == 1) a.mask[q0 + i] = sAnc[i];
  const int past = len - ql, at = past + i;
  a.positions[q0 + i] = past + sDepth[i];
  const int32_t page = a.block_table[(size_t)b * a.max_blocks + at / a.block_size];
  const bool there = page >= 0 && page < a.num_blocks;
  if (!there) set_status(a.status, MLA_DEV_BAD_BLOCK);
  a.slots[q0 + i] = there ? (int64_t)page * a.block_size + at % a.block_size : -1;
}

// ---------------------------------------------------------------------- verify
// A cluster of 1 to 16 CTAs takes a sequence, each CTA a piece of the
// vocabulary, each warp a contiguous piece of that. What the walk asks of
// single tokens is gathered first, for all rows of the tree at once; every CTA
// then takes the same walk (warp 0) and meets the others only where a sum over
// the vocabulary is wanted: behind a rejection when there are draft
// probabilities, and for the last draw. Weights enter the sums as whole numbers
// of 2^-40, so a sum does not depend on how the vocabulary is cut, and neither
// does the drawn token. 64 chains over 102,400 tokens take 16 us, of which the 49 MB
// that the rejections' sums read from HBM are 7.4; 32 trees over 50,001 tokens 16:
// up to four passes one behind another, each of some 5,000 cycles (its loads and sums
// 2,400, meeting the other CTAs 1,500, the next step of the walk 1,000 to 2,000).
constexpr int kVerWarps = 16, kVerThreads = 32 * kVerWarps, kVerMaxCl = 16;
constexpr int kVerUnroll = 4;   // 128 tokens each, in flight in a warp

struct VerifyArgs {
  const float* p;
  const float* q;        // NULL: the drafted tokens were not drawn
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* query_start_loc;
  const float* u;
  const float* u_last;
  int32_t* path;
  int32_t* path_lens;
  int32_t* next;
  uint32_t* status;
  int64_t num_q;
  int32_t vocab, max_path;
  int32_t warp_tokens;   // of a warp's piece, a multiple of 128
};

__device__ __forceinline__ float clamp01(float x) { return fminf(fmaxf(x, 0.f), 1.f); }  // (NaN: 0)

// floor(w 2^40) of w in [0, 1] as hi 2^20 + lo, hi = floor(w 2^20): adding 8 with
// the sum rounded down leaves steps of 2^-20, whose number is in the sum's low bits.
__device__ __forceinline__ void fixed40(float w, uint32_t& hi, uint32_t& lo) {
  const float s = __fadd_rd(w, 8.f);
  const float rest = w - (s - 8.f);                       // exact, below 2^-20
  hi = __float_as_uint(s) - __float_as_uint(8.f);
  lo = __float_as_uint(__fmaf_rd(rest, 1048576.f, 8.f)) - __float_as_uint(8.f);
}
__device__ __forceinline__ uint64_t fixed40(float w) {
  uint32_t hi, lo;
  fixed40(w, hi, lo);
  return ((uint64_t)hi << 20) + lo;
}

// What is left of p after the rejections so far: w <- max(w - Z q, 0) for each.
template <int N>
__device__ __forceinline__ void rest_of(float4 (&w)[N], const float4 (&q)[N], const float* z, int r) {
#pragma unroll
  for (int u = 0; u < N; ++u) w[u] = make_float4(clamp01(w[u].x), clamp01(w[u].y), clamp01(w[u].z), clamp01(w[u].w));
#pragma unroll 1
  for (int k = 0; k < r; ++k) {
    const float m = -z[k];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      w[u].x = fmaxf(fmaf(m, q[u].x, w[u].x), 0.f);
      w[u].y = fmaxf(fmaf(m, q[u].y, w[u].y), 0.f);
      w[u].z = fmaxf(fmaf(m, q[u].z, w[u].z), 0.f);
      w[u].w = fmaxf(fmaf(m, q[u].w, w[u].w), 0.f);
    }
  }
  if (r > 0) {
#pragma unroll
    for (int u = 0; u < N; ++u)
      w[u] = make_float4(fminf(w[u].x, 1.f), fminf(w[u].y, 1.f), fminf(w[u].z, 1.f), fminf(w[u].w, 1.f));
  }
}
__device__ __forceinline__ float rest_of(float p, float q, const float* z, int r) {
  float w = clamp01(p);
  for (int k = 0; k < r; ++k) w = fmaxf(fmaf(-z[k], q, w), 0.f);
  return fminf(w, 1.f);
}

template <bool DRAFT>
__global__ void __launch_bounds__(kVerThreads) tree_verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ int sUp[kTreeRows], sTok[kTreeRows], sOut[DRAFT ? 1 : kTreeRows];
  __shared__ float sU[kTreeRows], sP[kTreeRows], sQ[DRAFT ? kTreeRows : 1], sZ[DRAFT ? kTreeRows : 1];
  __shared__ uint64_t sWarp[kVerWarps], sCta[2][kVerMaxCl];
  __shared__ uint64_t sDraw[2][kVerWarps], sGoal;
  __shared__ bool sYes[kTreeRows];      // the row is accepted if none of its siblings was rejected
  __shared__ int sCur, sRej, sDone;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int CL = (int)gridDim.y, rank = (int)cl::rank(), b = blockIdx.x;
  const int V = a.vocab;
  cl::started();       // (waited for behind the gathering of the rows)
  pdl_wait();
  pdl_launch_dependents();
  const int q0 = a.query_start_loc[b], q1 = a.query_start_loc[b + 1];
  const float last_u = tid == 0 ? a.u_last[b] : 0.f;
  const int ql = q1 - q0;
  const bool bad = q0 < 0 || q1 > a.num_q || ql < 0 || ql > kTreeRows;
  if (bad || ql == 0) {   // (the whole cluster)
    if (rank == 0) {
      for (int i = tid; i < a.max_path; i += kVerThreads) a.path[(size_t)b * a.max_path + i] = -1;
      if (tid == 0) {
        a.path_lens[b] = 0;
        a.next[b] = -1;
        if (bad) set_status(a.status, MLA_DEV_BAD_SEQ);
      }
    }
    __syncwarp();
    cl::wait_started();
    return;
  }
  for (int i = tid; i < ql; i += kVerThreads) {
    int up = i > 0 ? a.parents[q0 + i] : -1;
    const int x = i > 0 ? a.tokens[q0 + i] : 0;
    if (up < -1 || up >= i) {
      up = -1;
      if (rank == 0) set_status(a.status, MLA_DEV_BAD_SEQ);
    }
    if (up >= 0 && (x < 0 || x >= V)) {
      up = -1;
      if (rank == 0) set_status(a.status, MLA_DEV_BAD_TOKEN);
    }
    sUp[i] = up;
    sTok[i] = x;
    sU[i] = a.u[q0 + i];
    if (up >= 0) {
      const size_t at = (size_t)(q0 + up) * V + x;
      const float w = clamp01(a.p[at]);
      double bar = (double)sU[i];
      if constexpr (DRAFT) {
        sQ[i] = a.q[at];
        bar *= (double)sQ[i];
      }
      sP[i] = w;
      sYes[i] = bar < (double)w;
    }
  }
  __syncwarp();
  cl::wait_started();  // (sums go to the others' shared memory from here on)
  __syncthreads();

  // the walk's state, of warp 0
  int i = 0, cur = 0, depth = 1, rej = 0;
  double z = 1.0;
  const bool writer = rank == 0 && tid == 0;
  int32_t* path = a.path + (size_t)b * a.max_path;
  if (writer) path[0] = 0;
  // goes on until a sum over the vocabulary is wanted: true if for the last draw
  auto walk = [&]() -> bool {
    while (depth < a.max_path) {
      int nxt = ql;   // the next row whose parent is `cur`
      for (int j0 = i + 1; j0 < ql; j0 += 32) {
        const int j = j0 + lane;
        const uint32_t hit = __ballot_sync(0xffffffffu, j < ql && sUp[j] == cur);
        if (hit) { nxt = j0 + __ffs(hit) - 1; break; }
      }
      if (nxt == ql) return true;
      i = nxt;
      float w = sP[i];
      bool yes;
      if (rej == 0) {
        yes = sYes[i];
      } else if constexpr (DRAFT) {
        w = rest_of(sP[i], sQ[i], sZ, rej);
        yes = (double)sU[i] * (double)sQ[i] * z < (double)w;
      } else {
        bool gone = false;   // the token was rejected before
        for (int k = lane; k < rej; k += 32) gone |= sOut[k] == sTok[i];
        if (__any_sync(0xffffffffu, gone)) w = 0.f;
        yes = (double)sU[i] * z < (double)w;
      }
      if (yes) {
        cur = i;
        if (writer) path[depth] = i;
        ++depth;
        rej = 0;
        z = 1.0;
      } else if constexpr (DRAFT) {
        if (lane == 0) sZ[rej] = (float)z;
        ++rej;
        __syncwarp();
        return false;
      } else if (w > 0.f) {
        if (lane == 0) sOut[rej] = sTok[i];
        ++rej;
        __syncwarp();
        z = fmax(z - (double)w, 0.0);
      }
    }
    return true;
  };

  const int base = (rank * kVerWarps + warp) * a.warp_tokens;   // of this warp's piece
  // 4 weights from place v of row `cur`'s pieces (place = token + off, off the
  // row's offset to 16 bytes), without the tokens rejected so far
  auto load4 = [&](const float* row, int v, int off) -> float4 {
    if (v >= off && v + 4 <= V + off) return __ldg(reinterpret_cast<const float4*>(row + (v - off)));
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = v + k >= off && v + k < V + off ? __ldg(row + (v + k - off)) : 0.f;
    return make_float4(x[0], x[1], x[2], x[3]);
  };
  int passes = 0;
  uint64_t total = 0;
  // the sums of every warp and CTA, and of all, for (row, rejections)
  auto sum_all = [&](int row, int r) {
    const size_t first = (size_t)(q0 + row) * V;
    const int off = (int)(first & 3), end = min(base + a.warp_tokens, V + off);
    const float *pr = a.p + first, *qr = DRAFT ? a.q + first : nullptr;
    uint32_t hi = 0, lo = 0;
    for (int v0 = base + 4 * lane; v0 < end; v0 += 128 * kVerUnroll) {
      float4 w[kVerUnroll], qv[kVerUnroll];
#pragma unroll
      for (int u = 0; u < kVerUnroll; ++u) {
        const int v = v0 + 128 * u;
        w[u] = v < end ? load4(pr, v, off) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (DRAFT) qv[u] = v < end && r > 0 ? load4(qr, v, off) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      rest_of(w, qv, sZ, DRAFT ? r : 0);
#pragma unroll
      for (int u = 0; u < kVerUnroll; ++u) {
        const float x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t h1, l1;
          fixed40(x[k], h1, l1);
          hi += h1;
          lo += l1;
        }
      }
    }
    uint64_t s = ((uint64_t)hi << 20) + lo;
    if constexpr (!DRAFT) {   // the rejected tokens of this piece weigh nothing
      for (int k = lane; k < r; k += 32) {
        const int v = sOut[k] + off;
        if (v >= base && v < end) s -= fixed40(clamp01(pr[sOut[k]]));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sWarp[warp] = s;
    __syncthreads();
    const int par = passes++ & 1;
    if (tid < CL) {
      uint64_t c = 0;
#pragma unroll
      for (int w = 0; w < kVerWarps; ++w) c += sWarp[w];
      const uint32_t dst = cl::map(smem_u32(&sCta[par][rank]), (uint32_t)tid);
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dst), "l"(c) : "memory");
    }
    cl::sync();
    total = 0;
    for (int c = 0; c < CL; ++c) total += sCta[par][c];
  };

  bool done = false;
  while (!done) {
    if (warp == 0) {
      const bool last = walk();
      if (lane == 0) {
        sCur = cur;
        sRej = rej;
        sDone = last;
      }
    }
    __syncthreads();
    done = sDone;
    // (a rejection's sums are the last draw's too, where no row follows it)
    if (!done || !DRAFT || sRej == 0) sum_all(sCur, sRej);
    if (DRAFT && !done && warp == 0) z = (double)(__ull2float_rn(total) * 0x1p-40f);
  }
  int row = sCur, r = sRej;
  if (total == 0 && r > 0) {   // nothing is left: the target's own distribution
    r = 0;
    sum_all(row, 0);
  }
  if (rank == 0) {
    const int n = __shfl_sync(0xffffffffu, depth, 0);   // (warp 0's)
    if (warp == 0)
      for (int k = n + lane; k < a.max_path; k += 32) path[k] = -1;
    if (tid == 0) {
      a.path_lens[b] = n;
      if (total == 0) {
        a.next[b] = -1;
        set_status(a.status, MLA_DEV_BAD_TOKEN);
      }
    }
  }
  if (total == 0) return;
  // the first token whose running sum passes u * total: its CTA, its warp, it
  // (64-bit products by one thread: of all 512 they take 1,000 cycles)
  if (tid == 0) sGoal = min((uint64_t)__double2ull_rd(fmax((double)last_u, 0.0) * (double)total), total - 1);
  __syncthreads();
  uint64_t goal = sGoal;
  const int par = (passes - 1) & 1;
  for (int c = 0; c < rank; ++c) {
    if (goal < sCta[par][c]) return;
    goal -= sCta[par][c];
  }
  if (goal >= sCta[par][rank]) return;
  int piece = 0;
  for (; goal >= sWarp[piece]; ++piece) goal -= sWarp[piece];
  // all of the CTA looks through that warp's piece
  const size_t first = (size_t)(q0 + row) * V;
  const int off = (int)(first & 3), from = (rank * kVerWarps + piece) * a.warp_tokens;
  const int end = min(from + a.warp_tokens, V + off);
  const float *pr = a.p + first, *qr = DRAFT ? a.q + first : nullptr;
  for (int v0 = from, flip = 0; v0 < end; v0 += 4 * kVerThreads, flip ^= 1) {
    const int v = v0 + 4 * tid;
    float4 w[1], qv[1];
    w[0] = qv[0] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (v < end) {
      w[0] = load4(pr, v, off);
      if (DRAFT && r > 0) qv[0] = load4(qr, v, off);
    }
    rest_of(w, qv, sZ, DRAFT ? r : 0);
    const float x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
    uint64_t f[4], own = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = fixed40(x[k]);
    if constexpr (!DRAFT) {
      for (int m = 0; m < r; ++m) {
        const int k = sOut[m] + off - v;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (k == u) f[u] = 0;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) own += f[k];
    uint64_t upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) sDraw[flip][warp] = upto;
    __syncthreads();
    uint64_t all = 0;
#pragma unroll
    for (int k = 0; k < kVerWarps; ++k) {
      if (k == warp) upto += all;
      all += sDraw[flip][k];
    }
    if (goal < all) {
      if (goal < upto && goal >= upto - own) {
        uint64_t run = upto - own;
        int k = 0;
        while (k < 3 && (run += f[k]) <= goal) ++k;
        a.next[b] = v + k - off;
      }
      return;
    }
    goal -= all;
  }
}

// CTAs of a cluster: as many as keep a CTA's piece at 2,048 tokens at the least
// and all clusters on the device at once (two CTAs an SM).
int verify_cluster(int64_t vocab, int64_t batch) {
  int c = 1;
  while (c < kVerMaxCl && vocab / (2 * c) >= 2048 && batch * 2 * c <= 304) c *= 2;
  return c;
}

// ---------------------------------------------------------------------- commit
// A thread moves one 16-byte column of one sequence's rows in one layer. A row
// goes to a place before its own or stays, and the path ascends, so no place
// that is written holds a row that is still to be read by the same column.
constexpr int kComThreads = 288, kComBatch = 8;

struct CommitArgs {
  uint8_t* cache;
  int64_t layer_bytes, num_blocks;
  int32_t row_bytes, layers;
  const int32_t* block_table;
  int32_t max_blocks, block_size;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  const int32_t* path;
  const int32_t* path_lens;
  int32_t max_path;
  int32_t* new_lens;
  uint32_t* status;
};

__global__ void __launch_bounds__(kComThreads) tree_commit_kernel(const __grid_constant__ CommitArgs a) {
  __shared__ int64_t sSrc[kTreeRows], sDst[kTreeRows];
  const int b = blockIdx.x, tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int q0 = a.query_start_loc[b], q1 = a.query_start_loc[b + 1], len = a.seq_lens[b];
  const int ql = q1 - q0, n = a.path_lens[b];
  const bool first = tid == 0 && blockIdx.y == 0;
  if (q0 < 0 || q1 < q0 || ql > len || (int64_t)len > (int64_t)a.max_blocks * a.block_size) {
    if (first) {
      a.new_lens[b] = 0;
      set_status(a.status, MLA_DEV_BAD_SEQ);
    }
    return;
  }
  const int past = len - ql;
  bool bad = n < 0 || n > a.max_path || n > ql || n > kTreeRows;
  if (!bad)
    for (int i = tid; i < n; i += kComThreads) {
      const int p = a.path[(size_t)b * a.max_path + i];
      const int before = i > 0 ? a.path[(size_t)b * a.max_path + i - 1] : -1;
      if (p <= before || p >= ql || before < -1) bad = true;
      int64_t src = -1, dst = -1;
      if (p != i && p >= 0 && p < ql) {
        const int s = past + p, d = past + i;
        const int32_t sp = a.block_table[(size_t)b * a.max_blocks + s / a.block_size];
        const int32_t dp = a.block_table[(size_t)b * a.max_blocks + d / a.block_size];
        if (sp < 0 || sp >= a.num_blocks || dp < 0 || dp >= a.num_blocks) {
          set_status(a.status, MLA_DEV_BAD_BLOCK);
        } else {
          src = (int64_t)sp * a.block_size + s % a.block_size;
          dst = (int64_t)dp * a.block_size + d % a.block_size;
        }
      }
      sSrc[i] = src;
      sDst[i] = dst;
    }
  bad = __syncthreads_or(bad);
  if (first) {
    a.new_lens[b] = past + (bad ? 0 : n);
    if (bad) set_status(a.status, MLA_DEV_BAD_SLOT);
  }
  const int cols = a.row_bytes / 16, layer = blockIdx.y * (kComThreads / cols) + tid / cols;
  if (bad || tid >= kComThreads / cols * cols || layer >= a.layers) return;
  uint8_t* at = a.cache + (size_t)layer * a.layer_bytes + (tid % cols) * 16;
  for (int i0 = 0; i0 < n; i0 += kComBatch) {
    uint4 v[kComBatch];
#pragma unroll
    for (int u = 0; u < kComBatch; ++u)
      if (i0 + u < n && sSrc[i0 + u] >= 0) v[u] = *reinterpret_cast<const uint4*>(at + sSrc[i0 + u] * a.row_bytes);
#pragma unroll
    for (int u = 0; u < kComBatch; ++u)
      if (i0 + u < n && sSrc[i0 + u] >= 0) *reinterpret_cast<uint4*>(at + sDst[i0 + u] * a.row_bytes) = v[u];
  }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

mla_status mla_tree_plan(const mla_config* cfg, const int32_t* parents, const int32_t* seq_lens,
                         const int32_t* query_start_loc, const int32_t* block_table,
                         int32_t max_blocks_per_seq, int64_t num_blocks, int32_t batch,
                         int64_t num_q, int32_t mask_words, uint64_t* tree_mask,
                         int32_t* positions, int64_t* slots, uint32_t* dev_status, void* stream) {
  mla_status s = validate_config(cfg);
  if (s != MLA_OK) return s;
  if (num_q < 0 || batch < 0 || num_blocks < 0 || max_blocks_per_seq < 0 || mask_words < 1)
    return MLA_ERR_INVALID_ARGUMENT;
  if (mask_words > kMaxWords || num_q > ((int64_t)1 << 30) ||
      num_blocks > ((int64_t)1 << 31) / cfg->block_size ||
      max_blocks_per_seq > ((int64_t)1 << 30) / cfg->block_size)
    return MLA_ERR_UNSUPPORTED;
  if (num_q == 0) return MLA_OK;
  if (!parents || !seq_lens || !query_start_loc || !block_table || !tree_mask || !positions ||
      !slots || batch == 0)
    return MLA_ERR_INVALID_ARGUMENT;
  if (!t_aligned(parents, 4) || !t_aligned(seq_lens, 4) || !t_aligned(query_start_loc, 4) ||
      !t_aligned(block_table, 4) || !t_aligned(tree_mask, 8) || !t_aligned(positions, 4) ||
      !t_aligned(slots, 8) || !t_aligned(dev_status, 4))
    return MLA_ERR_INVALID_ARGUMENT;
  const PlanTreeArgs a{parents, seq_lens, query_start_loc, block_table, max_blocks_per_seq,
                       cfg->block_size, mask_words, num_blocks, num_q, tree_mask, positions, slots,
                       dev_status};
  const int rows = 64 * mask_words, smem = (rows + 1) * mask_words * 8 + rows * 8;
  auto kernel = mask_words == 1 ? tree_plan_kernel<1> : tree_plan_kernel<kMaxWords>;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = launch_pdl(kernel, dim3((unsigned)batch), dim3(rows), smem,
                   reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

mla_status mla_tree_verify(const float* target_probs, const float* draft_probs, int32_t vocab_size,
                           const int32_t* tokens, const int32_t* parents,
                           const int32_t* query_start_loc, int32_t batch, int64_t num_q,
                           const float* uniforms, const float* final_uniforms, int32_t* path,
                           int32_t* path_lens, int32_t max_path, int32_t* next_tokens,
                           uint32_t* dev_status, void* stream) {
  if (vocab_size < 1 || batch < 0 || num_q < 0 || max_path < 1) return MLA_ERR_INVALID_ARGUMENT;
  if (vocab_size > (1 << 20) || num_q > ((int64_t)1 << 30)) return MLA_ERR_UNSUPPORTED;
  if (batch == 0) return MLA_OK;
  if (!query_start_loc || !final_uniforms || !path || !path_lens || !next_tokens)
    return MLA_ERR_INVALID_ARGUMENT;
  if (num_q > 0 && (!target_probs || !tokens || !parents || !uniforms)) return MLA_ERR_INVALID_ARGUMENT;
  if (!t_aligned(target_probs, 16) || !t_aligned(draft_probs, 16) || !t_aligned(tokens, 4) ||
      !t_aligned(parents, 4) || !t_aligned(query_start_loc, 4) || !t_aligned(uniforms, 4) ||
      !t_aligned(final_uniforms, 4) || !t_aligned(path, 4) || !t_aligned(path_lens, 4) ||
      !t_aligned(next_tokens, 4) || !t_aligned(dev_status, 4))
    return MLA_ERR_INVALID_ARGUMENT;
  const int CL = verify_cluster(vocab_size, batch);
  const int warps = CL * kVerWarps;
  // (a row begins up to 3 tokens behind its first 16 bytes)
  const int piece = ((vocab_size + 3 + warps - 1) / warps + 127) / 128 * 128;
  const VerifyArgs a{target_probs, draft_probs, tokens, parents, query_start_loc, uniforms,
                     final_uniforms, path, path_lens, next_tokens, dev_status, num_q, vocab_size,
                     max_path, piece};
  auto kernel = draft_probs ? tree_verify_kernel<true> : tree_verify_kernel<false>;
  cudaError_t e = cudaSuccess;
  if (CL > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return MLA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)batch, (unsigned)CL);
  cfg.blockDim = dim3(kVerThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = (unsigned)CL;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

mla_status mla_tree_commit(const mla_config* cfg, void* cache, int32_t num_layers,
                           int64_t num_blocks, int32_t row_bytes, const int32_t* block_table,
                           int32_t max_blocks_per_seq, const int32_t* seq_lens,
                           const int32_t* query_start_loc, int32_t batch, const int32_t* path,
                           const int32_t* path_lens, int32_t max_path, int32_t* new_lens,
                           uint32_t* dev_status, void* stream) {
  mla_status s = validate_config(cfg);
  if (s != MLA_OK) return s;
  if (num_layers < 0 || num_blocks < 0 || max_blocks_per_seq < 0 || batch < 0 ||
      max_path < 1)
    return MLA_ERR_INVALID_ARGUMENT;
  if (row_bytes != kRow * (cfg->dtype == MLA_BF16 ? 2 : 4) && !(cfg->dtype == MLA_BF16 && row_bytes == kRow8))
    return MLA_ERR_UNSUPPORTED;
  if (num_blocks > ((int64_t)1 << 31) / cfg->block_size ||
      max_blocks_per_seq > ((int64_t)1 << 30) / cfg->block_size || num_layers > 65535)
    return MLA_ERR_UNSUPPORTED;
  if (batch == 0) return MLA_OK;
  if (!block_table || !seq_lens || !query_start_loc || !path || !path_lens || !new_lens ||
      (!cache && num_layers > 0))
    return MLA_ERR_INVALID_ARGUMENT;
  if (!t_aligned(cache, 16) || !t_aligned(block_table, 4) || !t_aligned(seq_lens, 4) ||
      !t_aligned(query_start_loc, 4) || !t_aligned(path, 4) || !t_aligned(path_lens, 4) ||
      !t_aligned(new_lens, 4) || !t_aligned(dev_status, 4))
    return MLA_ERR_INVALID_ARGUMENT;
  const CommitArgs a{(uint8_t*)cache, num_blocks * cfg->block_size * row_bytes, num_blocks,
                     row_bytes, num_layers, block_table, max_blocks_per_seq, cfg->block_size,
                     seq_lens, query_start_loc, path, path_lens, max_path, new_lens, dev_status};
  const int per = kComThreads / (row_bytes / 16);
  const dim3 grid((unsigned)batch, (unsigned)(num_layers > 0 ? (num_layers + per - 1) / per : 1));
  const cudaError_t e = launch_pdl(tree_commit_kernel, grid, dim3(kComThreads), 0,
                                   reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
