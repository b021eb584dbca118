// Attention over a paged cache: what its two kernels and their join share --
// parameters, and the even division of the work over workers.
//
// An item is what one worker could do alone: a key/value head of a request,
// with all of its query rows (few rows) or with one tile of them (chunks).
// Items lie one after the other on a line, each as long as the keys it reads
// plus a constant for its fixed cost, in order of request, head and tile.
// Worker w of W takes the part [U w / W, U (w + 1) / W) of the line's length
// U, rounded to whole blocks of keys.  Lengths are read on the GPU, so
// every worker finds its part for itself: one pass over the requests for U,
// one to its first item.  An item cut by a worker's border leaves partial
// (m, l, o) records, at most two per worker (its first and its last item).
// Each worker leaves a note of them, and the join kernel merges an item's
// records, in order of keys, where the item ends.
#pragma once

#include <cuda_bf16.h>

#include "paged.h"
#include "ptx_ops.cuh"

namespace mk {

struct AttnParams {
  const __nv_bfloat16 *q, *v;  // v: the value pool
  __nv_bfloat16* out;
  int64_t ld_q, ld_out;
  const int32_t *table, *cu, *ctx;
  float* part;      // partial records: [slots][rows][D], then (m, l) [slots][rows][2]
  int32_t* status;
  float scale;      // softmax scale times log2(e)
  int B, N, Hq, Hkv, G, max_new, max_pages, num_pages, page_shift;
  int workers;
  int rows;         // rows of a partial record
  int tq;           // tokens per query tile (chunks): 128 / G
  int wait_limit;   // seconds that a wait may take: a part of the longest request
};

constexpr int kRowBlockBytes = 16384;  // keys and values of a few-rows block

// Keys that a part's results are summed over by the products alone.  The tensor cores cut each sum off towards zero
// (measured: 2^-22 of it per 16 keys), which over a long part is a shrinkage: values of 1.0 came out as 0.996 behind
// 2^20 keys and as 0.976 behind 2^22.  So every 2^16 keys a worker adds its results to the place of its partial
// record, in f32 and rounded to nearest, and goes on from zero; what is lost stays under 2^-11.  The sums of
// probabilities likewise: added block by block to a sum of 2^25, equal blocks may all be rounded the same way, by 1 %.
constexpr int kFoldKeys = 65536;

// The same over e4m3 pages (paged_rows8.cu, paged_chunk8.cu): codes, and a scale per page and head.
struct Attn8Params : AttnParams {
  const uint8_t* v8;
  const float *kscale, *vscale;
};
constexpr int kRowBlockBytes8 = 8192;  // keys and values of a few-rows block
constexpr int kRowWarps8 = 8;          // warps (workers) per CTA of its kernel, a multiple of kRowWarps

// Geometry of an item: few query rows (all of a request's), or a pair of
// 128-row query tiles; E8: of e4m3 pages.
template <int D, bool CHUNK, bool E8 = false>
struct Geometry {
  static constexpr int kKeys = CHUNK ? 128 : E8 ? kRowBlockBytes8 / D / 2 : kRowBlockBytes / D / 4;  // keys per block
  // an item's fixed cost, in keys: measured for few rows (paged_rows.cu); for chunks what surrounds a part's
  // blocks, some 2 us at 1.1 us for 128 keys of both tiles (256, 288 and 384 took the same time within noise, on
  // seven ragged chunks)
  static constexpr int kFixed = CHUNK ? 320 : E8 ? 128 : 96;
};

struct Seq {
  int n, ctx, nq;      // new tokens, cached tokens, items per head
  int row0;            // first query row
  int64_t base, step;  // cost of item i: base + i step
  int64_t per_head;
  bool bad;
};

template <int D, bool CHUNK, bool E8 = false>
__device__ __forceinline__ Seq load_seq(const AttnParams& p, int b) {
  Seq s;
  const int c0 = p.cu[b], c1 = p.cu[b + 1];
  s.ctx = p.ctx[b];
  s.row0 = c0;
  s.n = c1 - c0;
  s.bad = c0 < 0 || c1 < c0 || c1 > p.N || s.n > p.max_new || s.ctx < 0 ||
          (int64_t)s.ctx + s.n > ((int64_t)p.max_pages << p.page_shift);
  if (s.bad || s.n == 0) {
    s.n = 0;
    s.nq = 0;
    s.base = s.step = s.per_head = 0;
    return s;
  }
  constexpr int F = Geometry<D, CHUNK, E8>::kFixed;
  if (CHUNK) {
    const int tp = 2 * p.tq;
    s.nq = (s.n + tp - 1) / tp;
    s.base = (int64_t)s.ctx + tp + F;
    s.step = tp;
  } else {
    s.nq = 1;
    s.base = (int64_t)s.ctx + s.n + F;
    s.step = 0;
  }
  s.per_head = s.nq * s.base + s.step * ((int64_t)s.nq * (s.nq - 1) / 2);
  return s;
}

__device__ __forceinline__ int64_t warp_incl_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// r / d for 0 <= r, 0 < d and a quotient under 2^20: a float quotient put right (64-bit division is a long
// routine, and the workers' start is on the critical path of a small call)
__device__ __forceinline__ int small_quotient(int64_t r, int64_t d) {
  int q = (int)((float)r / (float)d);
#pragma unroll 1
  while ((int64_t)q * d > r) --q;
#pragma unroll 1
  while ((int64_t)(q + 1) * d <= r) ++q;
  return q;
}

// The line: its length, the length of a worker's part, and this lane's first request.
struct Line {
  int64_t u, part;
  int64_t own;  // requests' lengths on the line, lane = request, of the first 32
  bool bad;     // lengths that do not fit
  __device__ __forceinline__ int64_t border(int w) const { return min(part * w, u); }
};

// A whole warp; lanes agree but for `own`.
template <int D, bool CHUNK, bool E8 = false>
__device__ __forceinline__ Line measure_line(const AttnParams& p, int lane) {
  Line l;
  l.own = 0;
  int64_t u = 0;
  bool wrong = false;
#pragma unroll 1
  for (int b = lane; b < p.B; b += 32) {
    const Seq s = load_seq<D, CHUNK, E8>(p, b);
    const int64_t v = s.per_head * p.Hkv;
    if (b == lane) l.own = v;
    u += v;
    wrong |= s.bad;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
  l.bad = __any_sync(0xffffffffu, wrong);
  l.u = u;
  // whole blocks, a few at least: fewer records to join where there is little to do, and a worker behind an
  // item's first block always has a part of it
  constexpr int K = Geometry<D, CHUNK, E8>::kKeys, kLeast = (CHUNK ? 1 : 2) * K;
  const int64_t even = (u + p.workers - 1) / p.workers;
  l.part = even <= kLeast ? kLeast : (even + K - 1) / K * K;
  return l;
}

// A place on the line: the item holding it.  Uniform over the warp.
template <int D, bool CHUNK, bool E8 = false>
struct Cursor {
  int b, g, i;      // request, key/value head, tile
  Seq s;
  int64_t start;    // where the item begins
  __device__ __forceinline__ int64_t cost() const { return s.base + i * s.step; }
  // blocks of keys the item has
  __device__ __forceinline__ int blocks(const AttnParams& p) const {
    int keys = s.ctx + s.n;
    if (CHUNK) keys = (int)min((int64_t)keys, s.ctx + (i + 1) * s.step);
    constexpr int K = Geometry<D, CHUNK, E8>::kKeys;
    return (keys + K - 1) / K;
  }
  // the block that a place on the line falls to
  __device__ __forceinline__ int block_at(int64_t x, int nk) const {
    constexpr int K = Geometry<D, CHUNK, E8>::kKeys;
    if (x >= start + cost()) return nk;
    const int64_t k = x - start - Geometry<D, CHUNK, E8>::kFixed + K / 2;
    return k <= 0 ? 0 : (int)min((int64_t)nk, k / K);
  }
  // the worker that has the item's first block: the last whose part begins before the place from which
  // block_at() is 1
  __device__ __forceinline__ int first_worker(const Line& line) const {
    constexpr int K = Geometry<D, CHUNK, E8>::kKeys;
    return small_quotient(start + Geometry<D, CHUNK, E8>::kFixed + K / 2 - 1, line.part);
  }
  // the item holding place x of the line (0 <= x < U)
  __device__ __forceinline__ void find(const AttnParams& p, const Line& line, int64_t x, int lane) {
    int64_t before = 0;
#pragma unroll 1
    for (int b0 = 0;; b0 += 32) {
      int64_t own = line.own;
      if (b0 > 0) own = b0 + lane < p.B ? load_seq<D, CHUNK, E8>(p, b0 + lane).per_head * p.Hkv : 0;
      const int64_t end = warp_incl_scan(own, lane) + before;
      const unsigned hit = __ballot_sync(0xffffffffu, own > 0 && end > x);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b = b0 + src;
        start = __shfl_sync(0xffffffffu, end - own, src);
        break;
      }
      before = __shfl_sync(0xffffffffu, end, 31);
      if (b0 + 32 >= p.B) {  // not reached for x < U
        b = p.B;
        start = before;
        return;
      }
    }
    s = load_seq<D, CHUNK, E8>(p, b);
    const int64_t r = x - start;
    g = small_quotient(r, s.per_head);
    start += g * s.per_head;
    i = 0;
    if (CHUNK) {
      const int64_t rr = x - start;
      int lo = 0, hi = s.nq - 1;  // the last tile that begins at or before rr
#pragma unroll 1
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (mid * s.base + s.step * ((int64_t)mid * (mid - 1) / 2) <= rr) lo = mid;
        else hi = mid - 1;
      }
      i = lo;
      start += i * s.base + s.step * ((int64_t)i * (i - 1) / 2);
    }
  }
  // the next item; b == p.B behind the last
  __device__ __forceinline__ void next(const AttnParams& p) {
    start += cost();
    if (++i < s.nq) return;
    i = 0;
    if (++g < p.Hkv) return;
    g = 0;
#pragma unroll 1
    while (++b < p.B) {
      s = load_seq<D, CHUNK, E8>(p, b);
      if (s.n > 0) return;
    }
  }
};

// The workspace: outputs [2 * workers slots][rows][D] (chunks: [D / 4][rows][4], a row per lane), (m, l)
// [2 * workers][rows][2], notes [workers].
// Slot 2 w is worker w's part of an item that began before it, slot 2 w + 1
// its part of an item that goes on behind it.
__device__ __forceinline__ float* part_o(const AttnParams& p, int D, int slot, int row) {
  return p.part + ((size_t)slot * p.rows + row) * D;
}
// the same of a chunk: four columns of the row, the next four kTileRows pieces on
constexpr int kTileRows = 256;
__device__ __forceinline__ float4* part_cols(const AttnParams& p, int D, int slot, int row, int col) {
  return reinterpret_cast<float4*>(p.part + (size_t)slot * kTileRows * D) + (col / 4) * kTileRows + row;
}
__device__ __forceinline__ float* part_ml(const AttnParams& p, int D, int slot, int row) {
  return p.part + (size_t)2 * p.workers * p.rows * D + ((size_t)slot * p.rows + row) * 2;
}
// A worker's note of the item that began before it and ends with it (tokens 0: there is none): the
// worker it began with, whose second slot has its first part, the first query row, the key/value head,
// the tokens.
struct Note {
  int first, row0, g, tokens;
};
__device__ __forceinline__ Note* note_of(const AttnParams& p, int D, int w) {
  return reinterpret_cast<Note*>(p.part + (size_t)2 * p.workers * p.rows * (D + 2)) + w;
}

// What results folded at the maximum `at` are worth at the maximum `m` (both -inf: nothing was seen, and they are 0).
__device__ __forceinline__ float fold_weight(float at, float m) { return at == m ? 1.f : ptx::ex2(at - m); }

// Wait for a phase of an mbarrier, at most `limit` seconds or so, or until another thread has given up.
struct Patience {
  int gave_up;  // a wait has run out
  int limit;
};
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile Patience* state) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  uint32_t t0 = (uint32_t)clock();
  int left = state->limit;
#pragma unroll 1
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (state->gave_up) return false;
    if ((uint32_t)clock() - t0 > 2000000000u) {
      if (--left <= 0) state->gave_up = 1;
      t0 = (uint32_t)clock();
    }
  }
  return true;
}

cudaError_t launch_rows(const AttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int D,
                        cudaStream_t stream);
cudaError_t launch_chunk(const AttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, int D, cudaStream_t stream);
cudaError_t launch_rows8(const Attn8Params& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int D,
                         cudaStream_t stream);
cudaError_t launch_chunk8(const Attn8Params& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, int D, cudaStream_t stream);
constexpr int kRowWarps = 4;    // warps (workers) per CTA of the few-rows kernel
constexpr int kMaxFewRows = 8;  // query rows of a request and head that it takes
constexpr int kMaxFewRows8 = 16;  // and over e4m3 pages

}  // namespace mk
