// attn_core_walk.cuh — which tiles of which sequences a persistent CTA of the
// attention kernels works on (attn_core.cu, attn_core_tc.cu).
#pragma once

#include "attn_core.h"
#include "device.cuh"

namespace tpmlp {

constexpr uint32_t kAll = 0xffffffffu;

// What a CTA works on: `rows` tokens (a tile or a run of tiles) of a head of a sequence.
struct Item {
  int64_t row0;
  int tile, head, len, seq;  // len 0: no more items
};

// Debug build: whether an item lies in its sequence and that in the T rows, so that everything read and written for it does.
// A CTA whose item does not ends as after its last one.
__device__ __forceinline__ bool in_bounds(const CoreShape& s, const Item& it, int heads, int rows, int* status) {
  return TPMLP_DCHECK(it.seq >= 0 && it.seq < s.batch && it.head >= 0 && it.head < heads && it.tile >= 0 &&
                          int64_t(it.tile) * rows < it.len && it.row0 >= 0 && it.row0 + it.len <= s.T,
                      status, kChkAttnTile);
}

// The place of a CTA's item number `round` among all: a CTA takes one of every gridDim.x, from the front and from the back in
// turn, so that all get about the same where the items are in order of their work, the most first.
__device__ __forceinline__ uint64_t walk_place(uint64_t round) {
  const uint32_t g = gridDim.x;
  return round * g + (round & 1 ? g - 1 - blockIdx.x : blockIdx.x);
}

// The items of sequences of any lengths: 64 sequences at a time, the ones with at least d tiles, d from the longest's down
// (their d-th tile from the front, or from the back). With a causal mask that is the order of their work. Without one every
// tile of a sequence costs the whole length, and the longest sequences' last items come among those of short ones: of 13
// sequences of 1 to 1500 tokens, 12 heads, the fullest CTA of 152 has 58 tiles of 128 keys where the average is 40.6 (in
// order of the lengths it would have 42); 12 heads of 128: forward, dQ, dK and dV 71, 111 and 119 us, 13 equal sequences of
// as many tokens, with 0.64 of the scores, 59, 80 and 84. With a causal mask: all tiles of one index, of which
// those past a sequence's end are skipped, was worse: of 13 sequences of 1 to 1500 tokens, 12 heads, causal, the fullest
// CTA of dQ (bf16) had 66 key tiles in the place of 36 (33.6 on average), and of 1000 sequences in 65536 tokens, 32 heads of
// 128 on 8, it took dQ 888 us in the place of 756, and 16600 where max_seq was left at 65536.
struct SequenceWalk {
  const CoreShape& s;
  int* status;
  int heads, rows;
  bool last_first;  // the last tiles of a sequence have the most work
  int lane;
  int base = -64;                 // the first of the 64 sequences
  int c0, c1, d = 1;              // tiles of sequences base + `lane` and + 32; those with at least d are next, 0: no more
  uint32_t m0, m1;                // which these are
  uint64_t first = 0, count = 0;  // place of their first item, and how many there are

  __device__ __forceinline__ SequenceWalk(const CoreShape& s_, int* status_, int heads_, int rows_, bool last_first_, int lane_)
      : s(s_), status(status_), heads(heads_), rows(rows_), last_first(last_first_), lane(lane_) {}
  // The tiles of the next 64 sequences that have any.
  __device__ __forceinline__ void take() {
    for (base += 64, d = 0; base < s.batch; base += 64) {
      c0 = tiles_of(base + lane);
      c1 = tiles_of(base + lane + 32);
      d = __reduce_max_sync(kAll, max(c0, c1));
      if (d > 0) return choose();
    }
  }
  __device__ __forceinline__ int tiles_of(int b) const {
    int64_t row0;
    return b < s.batch ? (core_sequence(s, b, row0, status) + rows - 1) / rows : 0;
  }
  __device__ __forceinline__ void choose() {
    m0 = __ballot_sync(kAll, c0 >= d);
    m1 = __ballot_sync(kAll, c1 >= d);
    count = static_cast<uint64_t>(__popc(m0) + __popc(m1)) * heads;
  }
  // The k-th of a mask's set bits.
  __device__ __forceinline__ static int bit_of(uint32_t mask, int k) {
    for (; k > 0; --k) mask &= mask - 1;
    return __ffs(mask) - 1;
  }
  // Tile, head and sequence of the item at place `at`, which is no less than the last one asked for; all lanes of a warp.
  __device__ __forceinline__ bool find(uint64_t at, Item& it) {
    while (d > 0 && at >= first + count) {
      first += count;
      if (--d > 0)
        choose();
      else
        take();
    }
    if (d <= 0) return false;
    const uint32_t in = static_cast<uint32_t>(at - first);
    const int k = in / heads, n0 = __popc(m0);
    const int b = k < n0 ? bit_of(m0, k) : 32 + bit_of(m1, k - n0);
    const int c = __shfl_sync(kAll, b < 32 ? c0 : c1, b & 31);
    it.head = in % heads;
    it.tile = last_first ? d - 1 : c - d;
    it.seq = base + b;
    return true;
  }
};

}  // namespace tpmlp
