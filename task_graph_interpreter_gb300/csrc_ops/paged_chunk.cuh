// Shared by the chunk kernels over bf16 and e4m3 pages: the descriptor of a
// part of an item, and its masks.
#pragma once

#include "paged_attention.cuh"

namespace mk {

constexpr int kSegRing = 4;  // descriptors

struct Segment {
  int row0;       // first query row of the item (token index in q)
  int b, g;       // request, key/value head
  int ctx, t0;    // cached tokens; the item's first token in its request
  int n;          // new tokens of the request
  int k0, k1;     // key blocks of this part
  int end[2];     // end of each tile's key blocks, >= k0
  int slot;       // partial record, or -1: the part is the whole item
  int valid;      // 0: no more parts
  int split;      // the item has one tile, and the two take its key blocks in turn (over e4m3 pages)
};

// The first key that the item's first row does not see, and the first that no row of it does.
__device__ __forceinline__ int masked_from(const Segment& s) { return s.ctx + s.t0 + 1; }
__device__ __forceinline__ int masked_to(const Segment& s, const AttnParams& p) {
  return s.ctx + min(s.n, s.t0 + 2 * p.tq);
}

// Of 32 keys of a block, from `key` on, those of missing pages.
__device__ __forceinline__ uint32_t missing_keys(uint32_t miss, int key, int page_shift) {
  uint32_t bits = 0;
#pragma unroll 1
  for (int c = 0; c < 32; ++c) bits |= ((miss >> ((key + c) >> page_shift)) & 1) << c;
  return bits;
}

}  // namespace mk
