// What the kernels of mla_tree_decode share: their arguments, their workspace, and
// where the parts of a (row, head) lie in it.
#pragma once
#include "common.cuh"
#include "internal.h"

namespace mla {

constexpr int kTreeBlockRows = 128;    // (row, head) pairs of a q-block
constexpr int kTreeTok = 64;           // tokens of a tile

struct TreeArgs {
  const uint16_t* q_abs;
  int64_t num_blocks, num_q;
  const int32_t* block_table;
  int32_t max_blocks, block_size, num_heads, batch, words, shares;
  const int32_t* seq_lens;
  const int32_t* query_start_loc;
  const uint64_t* mask;
  float scale_log2;
  uint8_t* ws;
  uint32_t* status;
  int4* plan;      // [batch] {first unit, first item, tiles, q-blocks}
  float* lse;      // [slots][2][128]
  float* opart;    // [slots][128][512]
  float* o_lat;    // [num_q, H, 512]
};

// Workspace: header (status word, share), plan, partials. An item is what one
// q-block has in one strip; its part in cluster c has slot c + item, which is
// unique because items and shares are both contiguous and in order.
struct TreeWs {
  size_t plan, lse, opart, o_lat, total;
};
__host__ __device__ inline TreeWs tree_ws(int64_t num_q, int heads, int shares, int64_t batch) {
  TreeWs L;
  // items: a q-block has one, and one more for every share's worth of its units
  const int64_t slots = 2 * (int64_t)shares + num_q * heads / kTreeBlockRows + batch + 1;
  size_t off = kLayoutStart;
  L.plan = off;   off = align_up(off + (size_t)batch * 16, 256);
  L.lse = off;    off = align_up(off + (size_t)slots * 2 * kTreeBlockRows * 4, 256);
  L.o_lat = off;  off = align_up(off + (size_t)num_q * heads * kDc * 4, 256);
  L.opart = off;  off = align_up(off + (size_t)slots * kTreeBlockRows * kDc * 4, 256);
  L.total = off;
  return L;
}

__host__ __device__ __forceinline__ int tree_strips(int n, int m, int share) {
  return m <= 1 ? m : (n + share - 1) / share;
}

// Unit `off` of a sequence of n tiles and m > 1 q-blocks: tile k of q-block j in the
// strip of `tiles` tiles from strip * share on. (share * m passes 32 bits where few
// clusters have long sequences of many q-blocks; n * m does not.)
struct TreeUnit {
  int strip, tiles, j, k;
};
__host__ __device__ __forceinline__ TreeUnit tree_unit(int off, int n, int m, int share) {
  TreeUnit x;
  x.strip = off / m / share;
  const int first = x.strip * share, rem = off - first * m;
  x.tiles = share < n - first ? share : n - first;
  x.j = rem / x.tiles;
  x.k = rem - x.j * x.tiles;
  return x;
}

// Which slots of the decode's ring (four) hold half of a segment's query, and the barrier
// and the phase that say that it is read. A slot is taken again four stages on, while a
// segment may have only three (its query's two and a tile): by then the same half of the
// next segment's query may be read too, and a barrier for both would be a phase ahead of
// the wait. That of the segment after it (six stages on) is not on its way yet, so there
// is a barrier for each half and each parity of the segment.
struct QuerySlots {
  static constexpr int kBars = 4;
  uint32_t bits = 0;   // per slot: held [0, 4), barrier [8, 16), parity [16, 20)

  __host__ __device__ __forceinline__ static int bar_of(int seg, int part) { return 2 * (seg & 1) + part; }
  __host__ __device__ __forceinline__ void put(int slot, int seg, int part) {
    bits = (bits & ~(0x10001u << slot | 3u << (8 + 2 * slot))) | 1u << slot |
           (uint32_t)bar_of(seg, part) << (8 + 2 * slot) | (uint32_t)((seg >> 1) & 1) << (16 + slot);
  }
  __host__ __device__ __forceinline__ void clear(int slot) { bits &= ~(1u << slot); }
  __host__ __device__ __forceinline__ bool held(int slot) const { return (bits >> slot) & 1; }
  __host__ __device__ __forceinline__ int bar(int slot) const { return (bits >> (8 + 2 * slot)) & 3; }
  __host__ __device__ __forceinline__ uint32_t parity(int slot) const { return (bits >> (16 + slot)) & 1; }
};

// The merge of a call's parts and the projection, after the attention on `st`.
cudaError_t launch_tree_out(const TreeArgs& a, const void* W_uv, void* out, cudaStream_t st);

}  // namespace mla
