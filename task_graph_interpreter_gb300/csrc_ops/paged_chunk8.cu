// Paged attention of chunks over e4m3 pages, on the tcgen05 tensor cores: items,
// tiles, tensor memory and the turns of the two tiles are those of bf16 pages
// (paged_chunk.cu).  What differs is how 8-bit keys and values meet 16-bit
// queries and probabilities without losing what those hold:
//
//   S = Q K^T   kind::f8f6f4, keys as TMA brings them.  A query row, times a
//               power of two that brings its largest element to [2^7, 2^8), is
//               the sum of two e4m3 numbers (four significant bits each make
//               bf16's eight; elements 2^-10 below the largest keep 2^-18 of
//               it), so S is two products of twice the rate of one bf16 product
//   O += P V    kind::f16, P rounded to f16 (2^-11), values widened to f16 in
//               shared memory: three parts of P in e4m3 would cost the softmax
//               more than its powers do
//
// The scale of a page's keys is a factor of its columns of S, in f32: one factor
// per 16 columns in the softmax, which multiplies each score by the softmax
// scale anyway.  The scale of its values goes onto the values as they are
// widened, relative to the power of two of the largest scale of the part so far;
// O carries that unit and is rescaled where it rises, as where the running
// maximum does.  (Widened values are exact where scales are powers of two within
// 2^15 of each other; others are rounded to f16.)  That is the largest scale that
// all rows of the item see.  In a block of which some rows see a part only, one
// page may hold values so large that others, which more rows see, would be lost
// in the common unit: such a block's values stay codes, and its scales go onto
// each row's P, relative to the largest scale that the row sees.
//
// An item with one tile of tokens (drafts, the end of a prompt) would leave the
// other tile's products and softmax idle: its key blocks are dealt to both in
// turn, and the two results meet at the end of the part, the second's maxima and
// sums through shared memory, its O read from tensor memory.
//
// Bound by the chain of one tile (products of S, softmax, products of O: the
// other tile's overlap it) and by shared memory: a pair of blocks takes 3050 to
// 3450 cycles where bf16 pages take 2300.  Of a prompt of 8192 tokens, 8/32 heads
// of 128, 422 us (1.30 PFLOP/s; bf16 pages 315): without the widening, which
// moves 48 KB of shared memory per block, 383; the second parts of the queries
// are 82 of a form at 433; without powers, scales, or the packing of P no less.
// Four requests of 32768 keys and 20 rows 65 us (4.1 TB/s; bf16 pages 90), and 76
// before items of one tile were dealt to both; seven ragged chunks, 4/32 heads of
// 64, 51 us.  Scores are read in halves of 64: a whole row's 128 left 140 to 312
// bytes of spilled registers at every split of them.
//
//   warps 0-3, 4-7   softmax of tile 0 and tile 1, one row per thread
//   warp 8     copies: query tiles, key and value blocks, pages' scales
//   warps 9, 11   products of tile 0 and of tile 1
//   warp 10    division of the work
//   warps 12-15   queries into their two parts in place, a row per thread;
//              values to f16, a key per thread: those that were not loaded become
//              zero, and those that are NaN are set aside where a row does not
//              see the key
#include <cuda_fp16.h>

#include "paged_chunk.cuh"

namespace mk {
namespace {

using namespace ptx;

constexpr int kThreads = 512;
// registers: the launch's 4 x 128 threads x 128, moved to the softmax warpgroups
constexpr int kLaunchRegs = 128, kConsumerRegs = 176, kOtherRegs = 80, kWidenRegs = 80;
static_assert(2 * kConsumerRegs + kOtherRegs + kWidenRegs <= 4 * kLaunchRegs, "register shares within the launch's");
constexpr float kBias = 6.f;  // probabilities are kept times 2^kBias; a row's maximum may lag by 2^8
constexpr int kFar = 15;      // widened values are exact down to scales 2^kFar below the unit

template <int D>
struct Smem {
  static constexpr int kQuery = 128 * D * 2;     // a query tile
  static constexpr int kCodes = 128 * D;         // a block's keys, or values, as they come
  static constexpr int kHalf = 128 * 128;        // 128 rows of 128 bytes
  static constexpr int kValues = kHalf * (D / 64);
  static constexpr int kKeyStages = D == 128 ? 3 : 4, kRawStages = D == 128 ? 3 : 4, kValueStages = D == 128 ? 2 : 3;
  static constexpr int kControl = 3 * 1024;      // barriers, descriptors (struct Control)
  static constexpr int kBytes =
      kControl + 2 * kQuery + kKeyStages * kCodes + kRawStages * kCodes + kValueStages * kValues;
};
static_assert(Smem<128>::kBytes <= 232448, "227 KB of shared memory per CTA");

struct Block {  // what is known of a block of keys
  float ks[8], vs[8];  // scales of its pages
  uint32_t missing;    // pages that are not in the pool, one bit each
  int ve;              // exponent of the largest scale of values of the part so far
  int apart;           // its values are codes, and P carries their scales
};
struct Control {
  uint64_t k_full[4], k_empty[4], raw_full[4], raw_empty[4], v_full[4], v_empty[4], q_full[2], q_ready[2], q_empty[2],
      s_full[2], p_full[2][2], o_done[2], s_free[2], turn[2], seg_full[kSegRing], seg_empty[kSegRing], drained[2],
      known[8], half_done[2], second_done, second_read;
  Segment segs[kSegRing];
  int odd[kSegRing];      // a value set aside in this part
  Block blocks[8];        // ring
  uint32_t tmem;
  Patience patience;
  float2 ml[128];            // maximum and sum of a row's second half of key blocks (a split part),
  uint8_t second_ve[128];    // and the unit of its results
  uint8_t q_exp[2][2][128];  // exponents of the query rows' largest elements, by part's parity and tile
};
static_assert(sizeof(Control) <= Smem<128>::kControl, "control block");

template <int R>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// D[tmem] (+)= A B, e4m3 inputs, f32 sums; descriptors as in tc_mma_bf16_lo
__device__ __forceinline__ void tc_mma_f8_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of f32 sums and types coded 0: f16 (kind::f16), e4m3 (kind::f8f6f4).
__host__ __device__ constexpr uint32_t idesc_type0(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// Descriptor of a K-major operand of 64-byte rows, 64-byte swizzle
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) |
         ((uint64_t)1u << 46) | ((uint64_t)4u << 61);
}

__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }
__device__ __forceinline__ float unit_of(int ve) { return __uint_as_float((uint32_t)ve << 23); }

// Four bf16 elements times `up`, as e4m3 and what that leaves in e4m3.
__device__ __forceinline__ void split4(uint32_t w0, uint32_t w1, float up, uint32_t& hi, uint32_t& lo) {
  const float f[4] = {bf_lo(w0) * up, bf_hi(w0) * up, bf_lo(w1) * up, bf_hi(w1) * up};
  uint16_t h[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    uint32_t back;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(h[i]));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&back));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(l[i]) : "f"(f[2 * i + 1] - b.y), "f"(f[2 * i] - b.x));
  }
  hi = (uint32_t)h[0] | (uint32_t)h[1] << 16;
  lo = (uint32_t)l[0] | (uint32_t)l[1] << 16;
}

// A query row's bf16 elements into its two parts, in place: at D = 128 the first 128-byte row becomes the one, the
// second the other; at D = 64 the halves of the row.  Returns the exponent of the largest element.
template <int D>
__device__ __forceinline__ int split_query(uint32_t tile, int row) {
  constexpr int NC = D / 16;  // pieces of 16 elements
  const uint32_t at = tile + row * 128;
  const auto piece = [&](int c) {  // 8 elements
    return at + (c >> 3) * Smem<D>::kHalf + (((c & 7) ^ (row & 7)) << 4);
  };
  uint32_t big = 0;
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 v = lds128(piece(c));
    big = __vmaxu2(big, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                 __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
  }
  const int e = max((int)(max(big & 0xFFFFu, big >> 16) >> 7), 8);
  // 2^(7 - (e - 127)); a row with an element that is not finite is NaN
  const float up = __uint_as_float(e == 255 ? 0x7FC00000u : (uint32_t)(134 + 127 - e) << 23);
  uint4 low[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    // (pieces 2 c and 2 c + 1 are read before piece c is written)
    const uint4 a = lds128(piece(2 * c)), b = lds128(piece(2 * c + 1));
    uint4 hi;
    split4(a.x, a.y, up, hi.x, low[c].x);
    split4(a.z, a.w, up, hi.y, low[c].y);
    split4(b.x, b.y, up, hi.z, low[c].z);
    split4(b.z, b.w, up, hi.w, low[c].w);
    sts128(piece(c), hi);
    // (the second parts follow where pieces have been read)
    if (c >= NC / 2) {
      sts128(piece(2 * c), low[2 * c - NC]);
      sts128(piece(2 * c + 1), low[2 * c - NC + 1]);
    }
  }
  return e;
}

// For 32 columns of a row's result, the values that are NaN, of the keys it sees that other rows of the item do not
// (they were set aside).
__device__ __noinline__ void add_odd_values(const Attn8Params& p, const Segment& s, int lim, int D, int c, float* add) {
  const int pmask = (1 << p.page_shift) - 1;
  for (int key = max(s.k0 * 128, masked_from(s)); key <= min(lim, s.k1 * 128 - 1); ++key) {
    const int id = p.table[(size_t)s.b * p.max_pages + (key >> p.page_shift)];
    if ((unsigned)id >= (unsigned)p.num_pages) continue;
    const uint8_t* v = p.v8 + ((((int64_t)id * p.Hkv + s.g) << p.page_shift) + (key & pmask)) * D + c;
    for (int e = 0; e < 32; ++e)
      if ((v[e] & 0x7F) == 0x7F) add[e] = __uint_as_float(0x7FC00000u);
  }
}

// Every kFold blocks of a part a row's results, in units of `unit`, go from tensor memory to the place of the part's
// record (where the part is a whole item, to the worker's second, which is still free), and at the part's end what lies
// there is added to the rest (`last`); so does its sum of probabilities, l, whose new value is returned.  `m` is the
// row's maximum now, `some` whether results lie there already.  A whole warp, out of line: few parts are so long.
constexpr int kFold = kFoldKeys / 128;
__device__ __noinline__ float fold_results(const Attn8Params& p, int D, int slot, int row, uint32_t to, float m, float l,
                                           float unit, bool mine, bool some, bool last) {
  float2* at = reinterpret_cast<float2*>(part_ml(p, D, slot, row));  // the maximum of what lies there, and its sum
  const float2 there = mine && some ? *at : make_float2(m, 0.f);
  const float f = fold_weight(there.x, m), sum = l + there.y * f;
  if (mine) *at = make_float2(m, sum);
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tmem_ld32(to + c, o);
    tmem_wait_ld();
    float4* rec = part_cols(p, D, slot, row, c);
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (mine) {
        if (some) x = rec[e / 4 * kTileRows];
        x = make_float4(o[e] * unit + x.x * f, o[e + 1] * unit + x.y * f, o[e + 2] * unit + x.z * f,
                        o[e + 3] * unit + x.w * f);
        if (!last) rec[e / 4 * kTileRows] = x;
      }
      o[e] = last ? x.x : 0.f;
      o[e + 1] = last ? x.y : 0.f;
      o[e + 2] = last ? x.z : 0.f;
      o[e + 3] = last ? x.w : 0.f;
    }
    tmem_st32(to + c, o);
  }
  tmem_wait_st();
  return last ? sum : 0.f;
}

// The largest of 64 scores, in the exponent of two: 16 columns have one factor.
__device__ __forceinline__ float most_of(const float (&x)[64], const float* kf) {
  float top = -INFINITY;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float a = fmaxf(fmaxf(x[c * 16], x[c * 16 + 1]), x[c * 16 + 2]);
    float d = fmaxf(fmaxf(x[c * 16 + 3], x[c * 16 + 4]), x[c * 16 + 5]);
#pragma unroll
    for (int e = 6; e < 16; e += 4) {
      a = fmaxf(fmaxf(a, x[c * 16 + e]), x[c * 16 + e + 1]);
      if (e + 3 < 16) d = fmaxf(fmaxf(d, x[c * 16 + e + 2]), x[c * 16 + e + 3]);
    }
    top = fmaxf(top, fmaxf(a, d) * kf[c]);
  }
  return top;
}

// A row's results in tensor memory times f.
template <int D>
__device__ __forceinline__ void rescale(uint32_t to, float f) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tmem_ld32(to + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] *= f;
    tmem_st32(to + c, o);
  }
}

// The softmax of a block whose values are codes: what chunk8_kernel does with others, but for the row's unit, which is
// that of the largest scale of the pages that it sees (to its `last` key of the block), and the scales on P.  Out of
// line and of the loop over blocks: few are such, and a branch to it inside took a prompt of 8192 tokens from 419 to 488 us.
struct RowState {
  float m, l;  // maximum, sum of probabilities
  int ve;      // unit of the results
};
template <int D>
__device__ __noinline__ RowState scores_apart(const Attn8Params& p, Control& ctl, int w, int block, uint32_t ts, uint32_t to,
                                              uint32_t tp, int last, float rowf, RowState row, bool first) {
  const Block& b = ctl.blocks[block];
  float x[32], top = -INFINITY;
  int ve = row.ve;
  // 32 scores; those of keys that the row does not see are -inf
  const auto load = [&](int c) {
    const int n = last + 1 - c;
    uint32_t see = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1;
    if (b.missing) see &= ~missing_keys(b.missing, c, p.page_shift);
    tmem_ld32(ts + c, x);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = see >> e & 1 ? x[e] : -INFINITY;
  };
  const auto factor = [&](int c, int e) { return fmaxf(b.ks[(c + e) >> p.page_shift] * rowf, 0x1p-126f); };
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    load(c);
#pragma unroll
    for (int e = 0; e < 32; ++e) top = fmaxf(top, x[e] * factor(c, e / 16 * 16));
    if (c <= last) ve = max(ve, min((int)(__float_as_uint(b.vs[c >> p.page_shift]) >> 23 & 0xFF), 253));
    if (c + 16 <= last) ve = max(ve, min((int)(__float_as_uint(b.vs[(c + 16) >> p.page_shift]) >> 23 & 0xFF), 253));
  }
  const bool far = first || top > row.m + 8.f;
  if (!first && __any_sync(0xffffffffu, far || ve != row.ve)) {
    const float f = far ? ex2(row.m - top) : 1.f;
    row.l *= f;
    rescale<D>(to, ve - row.ve > 126 ? 0.f : f * unit_of(127 + row.ve - ve));
  }
  if (far) row.m = top;
  row.ve = ve;
  const float mu = row.m == -INFINITY ? 0.f : kBias - row.m;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    uint32_t r[16];
    load(c);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float f = factor(c, e / 8 * 16);
      // (a page that the row does not see may have any scale: its P is zero)
      const float v = fminf(b.vs[(c + e / 8 * 16) >> p.page_shift] * unit_of(254 - ve), 2.f);
      const float a = ex2(fmaf(x[2 * e], f, mu)), d = ex2(fmaf(x[2 * e + 1], f, mu));
      row.l += a + d;
      r[e] = pack_f16(a * v, d * v);
    }
    tmem_st16(tp + c / 2, r);  // (over scores that have been read, where P lies there)
    if (c & 32) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (threadIdx.x % 32 == 0) {
        mbar_arrive(&ctl.p_full[w][c >> 6]);
        if (D == 64 && c == 96) mbar_arrive(&ctl.s_free[w]);
      }
    }
  }
  return row;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk8_kernel(const __grid_constant__ Attn8Params p, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<D>;
  constexpr int NH = D / 64, KS = S::kKeyStages, RS = S::kRawStages, VS = S::kValueStages;
  // tensor memory columns of S_0, S_1, of O_0, O_1, and of P_0, P_1: over the scores at D = 128, apart at D = 64
  constexpr bool kApart = D == 64;
  constexpr uint32_t kSCol = 0, kOCol = 256, kPCol = kApart ? 384 : 0, kPStep = kApart ? 64 : 128;
  // no static shared memory: the dynamic part starts 1024-byte aligned, as the swizzled tiles need
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Control& ctl = *reinterpret_cast<Control*>(smem_raw);
  auto& segs = ctl.segs;
  auto& patience = ctl.patience;
  uint8_t* qt = smem_raw + S::kControl;          // [2] query tiles
  uint8_t* kring = qt + 2 * S::kQuery;           // [KS][128 keys][D]
  uint8_t* rawring = kring + KS * S::kCodes;     // [RS][128 keys][D]
  uint8_t* vring = rawring + RS * S::kCodes;     // [VS][NH][128 keys][128 B]
  // (broadcast, so that the compiler knows a warp's role and what follows from it uniform)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (smem_addr(smem_raw) & 1023u) {
    if (threadIdx.x == 0) set_status(p.status, MK_DEV_RING_TIMEOUT);
    return;
  }
  if (threadIdx.x == 0) {
    patience.gave_up = 0;
    patience.limit = p.wait_limit;
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ctl.k_full[i], 1);
      mbar_init(&ctl.k_empty[i], 2);
      mbar_init(&ctl.raw_full[i], 1);
      mbar_init(&ctl.raw_empty[i], 4);
      mbar_init(&ctl.v_full[i], 4);
      mbar_init(&ctl.v_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.q_full[i], 1);
      mbar_init(&ctl.q_ready[i], 4);
      mbar_init(&ctl.q_empty[i], 1);
      mbar_init(&ctl.drained[i], 1);
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_full[i][0], 4);
      mbar_init(&ctl.p_full[i][1], 4);
      mbar_init(&ctl.turn[i], 1);
      mbar_init(&ctl.s_free[i], 4);
      mbar_init(&ctl.o_done[i], 1);
      mbar_init(&ctl.half_done[i], 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&ctl.known[i], 1);
    mbar_init(&ctl.second_done, 4);
    mbar_init(&ctl.second_read, 4);
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(&ctl.seg_full[i], 1);
      mbar_init(&ctl.seg_empty[i], kThreads / 32 - 1);  // every warp but the one that makes them
    }
    fence_mbar_init();
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  if (warp == 9) {
    tmem_alloc(&ctl.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();
  wait_dependency();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0);
  const int pmask = (1 << p.page_shift) - 1;

  if (warp >= 12) {
    // -------------------------------------------------- queries into parts, values to f16
    reg_dec<kWidenRegs>();
    const int row = threadIdx.x & 127;
    const uint32_t q0 = smem_addr(qt), raw0 = smem_addr(rawring), v0 = smem_addr(vring);
    uint32_t blk = 0;
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      const int sst = i % kSegRing;
      if (!wait_phase(&ctl.seg_full[sst], (i / kSegRing) & 1, &patience)) break;
      const Segment& s = segs[sst];
      if (!s.valid) break;
      const int k0 = s.k0, k1 = s.k1, from = masked_from(s), to = masked_to(s, p);
      const bool second = s.split || s.t0 + p.tq < s.n;
#pragma unroll 1
      for (int w = 0; w < 2; ++w) {
        if (!(ok = wait_phase(&ctl.q_full[w], i & 1, &patience))) break;
        if (w == 0 || second) {
          ctl.q_exp[i & 1][w][row] = (uint8_t)split_query<D>(q0 + w * S::kQuery, row);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.q_ready[w]);
      }
      for (int k = k0; k < k1 && ok; ++k, ++blk) {
        const int rst = blk % RS, vst = blk % VS;
        if (!(ok = wait_phase(&ctl.raw_full[rst], (blk / RS) & 1, &patience))) break;
        if (!(ok = wait_phase(&ctl.v_empty[vst], ((blk / VS) & 1) ^ 1, &patience))) break;
        const Block& b = ctl.blocks[blk & 7];
        const int key = k * 128 + row;
        const float rel = b.apart ? 1.f : b.vs[min(row >> p.page_shift, 7)] * unit_of(254 - b.ve);
        const __half2 rel2 = __float2half2_rn(rel);
        // 16 codes of the row, from and to where the swizzles put them
        const uint32_t src = raw0 + rst * S::kCodes + row * D, dst = v0 + vst * S::kValues + row * 128;
        const auto codes = [&](int c) { return lds128(src + ((c ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4)); };
        const auto put = [&](int c, const uint4& v) {
          uint32_t out[8];
          widen_e4m3(v.x, out[0], out[1]);
          widen_e4m3(v.y, out[2], out[3]);
          widen_e4m3(v.z, out[4], out[5]);
          widen_e4m3(v.w, out[6], out[7]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&out[e]), rel2);
            out[e] = *reinterpret_cast<const uint32_t*>(&x);
          }
          const uint32_t d = dst + (c >> 2) * S::kHalf;
          sts128(d + ((((c & 3) * 2) ^ (row & 7)) << 4), make_uint4(out[0], out[1], out[2], out[3]));
          sts128(d + ((((c & 3) * 2 + 1) ^ (row & 7)) << 4), make_uint4(out[4], out[5], out[6], out[7]));
        };
        bool odd = false;
        if (k * 128 + 128 <= from && b.missing == 0) {
#pragma unroll 4
          for (int c = 0; c < D / 16; ++c) put(c, codes(c));
        } else {
          // keys that were not loaded are zero; a NaN of a key that some row of the item does not see is set aside
          const bool there = key < to && !((b.missing >> (row >> p.page_shift)) & 1);
          const auto clean = [&](uint32_t w) {
            const uint32_t nan = nan_codes(w);
            odd |= there && nan != 0 && key >= from;
            return !there ? 0u : key >= from ? w & ~nan : w;
          };
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            const uint4 v = codes(c);
            // (a page that is not there has no scale: 0 times 0)
            put(c, make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w)));
          }
        }
        if (odd) ctl.odd[sst] = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl.raw_empty[rst]);
          mbar_arrive(&ctl.v_full[vst]);
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.seg_empty[sst]);
    }
  } else if (warp >= 8) {
    reg_dec<kOtherRegs>();
    if (warp == 10) {
      // ------------------------------------------------ division of the work
      const Line line = measure_line<D, true>(p, lane);
      if (line.bad && blockIdx.x == 0 && lane == 0) set_status(p.status, MK_DEV_BAD_INDEX);
      const int64_t x0 = line.border(blockIdx.x), x1 = line.border(blockIdx.x + 1);
      if (lane == 0) *note_of(p, D, blockIdx.x) = Note{0, 0, 0, 0};
      Cursor<D, true> c;
      bool more = !line.bad && x0 < x1, begun = false;
      if (more) c.find(p, line, x0, lane);
      for (uint32_t made = 0;; ++made) {
        // the next part of this CTA, or the note that there is none
        int k0 = 0, k1 = 0, nk = 0;
        while (more) {
          if (begun) c.next(p);
          begun = true;
          more = c.b < p.B && c.start < x1;
          if (!more) break;
          nk = c.blocks(p);
          k0 = c.block_at(x0, nk);
          k1 = c.block_at(x1, nk);
          if (k0 < k1) break;
        }
        const int st = made % kSegRing;
        if (!wait_phase(&ctl.seg_empty[st], ((made / kSegRing) & 1) ^ 1, &patience)) break;
        if (lane == 0) {
          Segment& s = segs[st];
          s.valid = more ? 1 : 0;
          if (more) {
            const int t0 = c.i * 2 * p.tq;
            s.b = c.b;
            s.g = c.g;
            s.ctx = c.s.ctx;
            s.n = c.s.n;
            s.t0 = t0;
            s.row0 = c.s.row0 + t0;
            s.k0 = k0;
            s.k1 = k1;
            s.split = c.s.n - t0 <= p.tq && k1 - k0 > 1;
            s.slot = k0 == 0 && k1 == nk ? -1 : 2 * (int)blockIdx.x + (k0 == 0 ? 1 : 0);
            if (k0 != 0 && k1 == nk)
              *note_of(p, D, blockIdx.x) = Note{c.first_worker(line), s.row0, c.g, min(2 * p.tq, c.s.n - t0)};
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int first = t0 + (s.split ? 0 : w * p.tq), last = min(first + p.tq, c.s.n) - 1;
              s.end[w] = first < c.s.n ? max(k0, min(k1, (c.s.ctx + last) / 128 + 1)) : k0;
            }
          }
          ctl.odd[st] = 0;
          mbar_arrive(&ctl.seg_full[st]);
        }
        __syncwarp();
        if (!more) break;
      }
    } else if (warp == 8) {
      // ------------------------------------------------ copies
      const int box = min(128, pmask + 1), npg = 128 / box;
      uint32_t blk = 0, nk = 0, nv = 0, nq = 0;  // blocks; keys and values asked for; query tile pairs
      const auto load_q = [&](const Segment& s) {
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          if (!wait_phase(&ctl.q_empty[w], (nq & 1) ^ 1, &patience)) return false;
          if (lane == 0) {
            // (a second tile without tokens is not read; one that shares the first's has them too)
            const bool some = w == 0 || s.split || s.t0 + p.tq < s.n;
            mbar_arrive_expect_tx(&ctl.q_full[w], some ? NH * p.tq * p.G * 128 : 0);
            for (int h = 0; h < NH && some; ++h)
              tma_load_3d(qt + w * S::kQuery + h * S::kHalf, &qmap, h * 64, s.g * p.G, s.row0 + (s.split ? 0 : w * p.tq),
                          &ctl.q_full[w]);
          }
          __syncwarp();
        }
        ++nq;
        return true;
      };
      for (uint32_t i = 0;; ++i) {
        const int sst = i % kSegRing;
        if (!wait_phase(&ctl.seg_full[sst], (i / kSegRing) & 1, &patience)) break;
        const Segment s = segs[sst];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.seg_empty[sst]);
        if (!s.valid) break;
        const int L = masked_to(s, p);
        // the query tiles, behind the first keys and values where the last item's products still read theirs
        const bool early = __all_sync(0xffffffffu, mbar_test_wait(&ctl.q_empty[0], (nq & 1) ^ 1) &&
                                                       mbar_test_wait(&ctl.q_empty[1], (nq & 1) ^ 1));
        bool ok = !early || load_q(s);
        // lane = page; table entries are read two blocks ahead, scales one
        const int32_t* table = p.table + (size_t)s.b * p.max_pages;
        const auto entry = [&](int k) {  // (no key past the last block: it could pass 2^31)
          if (k >= s.k1 || lane >= npg) return -1;
          const int key = k * 128 + lane * box;
          return key < L ? table[key >> p.page_shift] : -1;
        };
        const auto scale_of = [&](const float* scales, int id, float none) {
          return (unsigned)id < (unsigned)p.num_pages ? __ldg(scales + (int64_t)id * p.Hkv + s.g) : none;
        };
        int id = entry(s.k0), id1 = entry(s.k0 + 1), ve = 1;
        float ks = scale_of(p.kscale, id, 1.f), vs = scale_of(p.vscale, id, 0.f);
        for (int k = s.k0; k < s.k1 && ok; ++k, ++blk) {
          const int id2 = entry(k + 2);
          const float ks1 = scale_of(p.kscale, id1, 1.f), vs1 = scale_of(p.vscale, id1, 0.f);
          const bool in = lane < npg && k * 128 + lane * box < L;
          const bool good = in && (unsigned)id < (unsigned)p.num_pages;
          if (in && !good) set_status(p.status, MK_DEV_BAD_INDEX);
          const uint32_t lanes = __ballot_sync(0xffffffffu, good), miss = __ballot_sync(0xffffffffu, in && !good);
          const int row = ((id * p.Hkv + s.g) << p.page_shift) + (k * 128 & pmask);
          const uint32_t bytes = __popc(lanes) * box * D;
          // (the copies start before the scales are known; the phase ends with the arrival behind them)
          const int kst = blk % KS, rst = blk % RS;
          if (!(ok = wait_phase(&ctl.k_empty[kst], ((blk / KS) & 1) ^ 1, &patience))) break;
          if (good) tma_load_2d(kring + kst * S::kCodes + lane * box * D, &kmap, 0, row, &ctl.k_full[kst]);
          Block& b = ctl.blocks[blk & 7];
          if (lane < 8) {
            b.ks[lane] = ks;
            b.vs[lane] = vs;
          }
          const int e = (int)(__float_as_uint(vs) >> 23 & 0xFF);
          ve = max(ve, __reduce_max_sync(0xffffffffu, e));
          ve = min(ve, 253);
          const bool far = __any_sync(0xffffffffu, good && e != 0 && e + kFar < ve);
          if (lane == 0) {
            b.missing = miss;
            b.ve = ve;
            b.apart = far && k * 128 + 128 > masked_from(s);
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_expect_tx(&ctl.k_full[kst], bytes);
            mbar_arrive(&ctl.known[blk & 7]);
          }
          ++nk;
          if (!(ok = wait_phase(&ctl.raw_empty[rst], ((blk / RS) & 1) ^ 1, &patience))) break;
          if (lane == 0) mbar_arrive_expect_tx(&ctl.raw_full[rst], bytes);
          __syncwarp();
          if (good) tma_load_2d(rawring + rst * S::kCodes + lane * box * D, &vmap, 0, row, &ctl.raw_full[rst]);
          ++nv;
          __syncwarp();
          id = id1;
          id1 = id2;
          ks = ks1;
          vs = vs1;
          if (k == s.k0 && !early) ok = load_q(s);
        }
        if (!ok) break;
      }
      if (*(volatile int*)&patience.gave_up) {
        if (lane == 0) set_status(p.status, MK_DEV_RING_TIMEOUT);
        // copies in flight land before the shared memory goes
        for (uint32_t d = nk > KS ? nk - KS : 0; d < nk; ++d)
          for (int j = 0; j < 100000 && !mbar_try_wait(&ctl.k_full[d % KS], (d / KS) & 1); ++j) {
          }
        for (uint32_t d = nv > RS ? nv - RS : 0; d < nv; ++d)
          for (int j = 0; j < 100000 && !mbar_try_wait(&ctl.raw_full[d % RS], (d / RS) & 1); ++j) {
          }
        for (int w = 0; w < 2 && nq; ++w)
          for (int j = 0; j < 100000 && !mbar_try_wait(&ctl.q_full[w], (nq - 1) & 1); ++j) {
          }
      }
    } else {
      // ------------------------------------------------ products of tile w
      // (what steers this loop or makes up a descriptor is a vote's or a broadcast's result, so that the compiler
      // knows it uniform and keeps the descriptors in uniform registers)
      const int w = warp == 9 ? 0 : 1;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_phase(bar, parity, &patience)) != 0;
      };
      const uint32_t idesc_s = idesc_type0(128, 128);
      const uint32_t idesc_o = idesc_type0(128, D) | kIdescBMnMajor;
      // low words of the operands' descriptors; a step of 32 bytes along a row adds 2, 16 value rows 128
      const uint64_t qd = smem_desc_sw128(smem_addr(qt) + w * S::kQuery, 1024u);
      const uint64_t kd = D == 128 ? smem_desc_sw128(smem_addr(kring), 1024u) : smem_desc_sw64(smem_addr(kring), 512u);
      const uint64_t vd = smem_desc_sw128_mn(smem_addr(vring), S::kHalf, 1024u);
      const uint32_t qhi = (uint32_t)(qd >> 32), khi = (uint32_t)(kd >> 32), vhi = (uint32_t)(vd >> 32);
      const uint32_t ts = tmem + kSCol + w * 128, to = tmem + kOCol + w * D, tp = tmem + kPCol + w * kPStep;
      uint32_t blk = 0, np = 0, nturn = 0;  // blocks; P handed over; turns taken (scores made, at D = 64)
      bool ok = true;
      for (uint32_t i = 0; ok; ++i) {
        const int sst = i % kSegRing;
        if (!(ok = wait(&ctl.seg_full[sst], (i / kSegRing) & 1))) break;
        const int valid = __shfl_sync(0xffffffffu, segs[sst].valid, 0), k0 = segs[sst].k0;
        const int nt = __shfl_sync(0xffffffffu, segs[sst].k1 - k0, 0);
        const int split = __shfl_sync(0xffffffffu, segs[sst].split, 0);
        // this tile's blocks: the first ones, or every other one from the w-th on (a split part)
        const int ntw = split ? (nt + 1 - w) / 2 : __shfl_sync(0xffffffffu, segs[sst].end[w] - k0, 0);
        const int steps = split ? (nt + 1) / 2 : nt, stride = split ? 2 : 1, first = split ? w : 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.seg_empty[sst]);
        if (!valid) break;
        if (!(ok = wait(&ctl.q_ready[w], i & 1))) break;
        tc_fence_after();
        if (ntw == 0 && lane == 0) mbar_arrive(&ctl.q_empty[w]);
        // P V of block j out of ring place vst; as soon as half of P is there
        const auto values = [&](int j, uint32_t vst) {
          const uint32_t b_lo = (uint32_t)vd + vst * (S::kValues >> 4);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (c == 1) {
              if (!wait(&ctl.p_full[w][1], np & 1)) return false;
              tc_fence_after();
            }
            if (elect_one()) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int kk = c * 4 + e;  // 16 keys
                tc_mma_bf16_ts_lo(to, tp + kk * 8, b_lo + kk * 128, vhi, idesc_o, kk != 0 ? 1u : j != 0 ? 1u : 0u);
              }
              if (c == 0) tc_commit(&ctl.half_done[w]);
              if (c == 1) {
                tc_commit(&ctl.v_empty[vst]);
                if (split) tc_commit(&ctl.v_empty[vst]);  // (for the other tile, which does not see the block)
                if (kApart || j + 1 == ntw) tc_commit(&ctl.o_done[w]);
              }
            }
            __syncwarp();
          }
          ++np;
          return true;
        };
        // S of block j out of ring place kst: the queries' first parts, then their second
        const auto scores = [&](int j, uint32_t kst) {
          const uint32_t b_lo = (uint32_t)kd + kst * (S::kCodes >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const int part = kk / (D / 32), e = kk % (D / 32);
              tc_mma_f8_lo(ts, (uint32_t)qd + part * (D == 128 ? S::kHalf >> 4 : 4) + e * 2, qhi, b_lo + e * 2, khi, idesc_s,
                           kk != 0 ? 1u : 0u);
              // the other tile's warp takes a while to see its turn
              if (!kApart && kk == D / 32 - 1) mbar_arrive(&ctl.turn[w ^ 1]);
            }
            tc_commit(&ctl.s_full[w]);
            tc_commit(&ctl.k_empty[kst]);
            if (split) tc_commit(&ctl.k_empty[kst]);
            if (j + 1 == ntw) tc_commit(&ctl.q_empty[w]);
          }
          __syncwarp();
        };
        for (int j = -1; j < steps; ++j) {
          // j-th block's values, next block's keys
          const int jv = j * stride + first, jk = jv + stride;
          const uint32_t kb = blk + jk, vb = blk + jv, kst = kb % KS, vst = vb % VS;
          const bool there_v = j >= 0 && jv < nt, there_k = jk < nt, pv = there_v && j < ntw, qk = there_k && j + 1 < ntw;
          if constexpr (kApart) {
            // S (block j + 1) as soon as the softmax has S (block j) in registers, P V (block j) as P comes
            if (there_k) {
              if (!(ok = wait(&ctl.k_full[kst], (kb / KS) & 1))) break;
              if (qk) {
                if (!(ok = wait(&ctl.s_free[w], (nturn & 1) ^ 1))) break;
                ++nturn;
                tc_fence_after();
                scores(j + 1, kst);
              } else if (lane == 0) {
                mbar_arrive(&ctl.k_empty[kst]);
              }
            }
            if (there_v) {
              if (!(ok = wait(&ctl.v_full[vst], (vb / VS) & 1))) break;
              if (pv) {
                if (!(ok = wait(&ctl.p_full[w][0], np & 1))) break;
                tc_fence_after();
                if (!(ok = values(j, vst))) break;
              } else if (lane == 0) {
                mbar_arrive(&ctl.v_empty[vst]);
              }
            }
            __syncwarp();
          } else {
            // P V (block j) before S (block j + 1).  A block that this tile does not need is handed back as it comes
            if (there_v && !(ok = wait(&ctl.v_full[vst], (vb / VS) & 1))) break;
            if (there_k && !(ok = wait(&ctl.k_full[kst], (kb / KS) & 1))) break;
            // tile 0 starts; then each block's products of one tile, then of the other
            if (!(ok = wait(&ctl.turn[w], (nturn & 1) ^ (w ^ 1)))) break;
            ++nturn;
            if (pv && !(ok = wait(&ctl.p_full[w][0], np & 1))) break;
            tc_fence_after();
            if (pv) {
              if (!(ok = values(j, vst))) break;
            } else if (there_v && lane == 0) {
              mbar_arrive(&ctl.v_empty[vst]);
            }
            if (qk) {
              scores(j + 1, kst);
            } else {
              if (lane == 0) {
                mbar_arrive(&ctl.turn[w ^ 1]);
                if (there_k) mbar_arrive(&ctl.k_empty[kst]);
              }
              __syncwarp();
            }
          }
        }
        blk += nt;
      }
      if (*(volatile int*)&patience.gave_up) {
        // products in flight end before the tensor memory is freed
        if (elect_one()) tc_commit(&ctl.drained[w]);
        __syncwarp();
        for (int j = 0; j < 100000 && !mbar_try_wait(&ctl.drained[w], 0); ++j) {
        }
      }
    }
  } else {
    // -------------------------------------------------- softmax: one row per thread
    reg_inc<kConsumerRegs>();
    const int w = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's tensor-memory lanes (lane field, bits 16 up)
    const uint32_t ts = tmem + lanes + kSCol + w * 128, to = tmem + lanes + kOCol + w * D,
                   tp = tmem + lanes + kPCol + w * kPStep;
    const int tok_in = row / p.G, head = row % p.G;
    const int per16 = p.page_shift - 4;  // a page has 2^per16 sixteens of keys
    uint32_t ns = 0, no = 0, np = 0, blk = 0, nsplit = 0;  // scores, results seen; P handed over; blocks; split parts
    for (uint32_t i = 0;; ++i) {
      const int sst = i % kSegRing;
      if (!wait_phase(&ctl.seg_full[sst], (i / kSegRing) & 1, &patience)) break;
      const Segment& s = segs[sst];
      if (!s.valid) break;
      const int k0 = s.k0, nb = s.end[w] - k0;
      // this tile's blocks: the first nb, or every other one from the w-th on (a split part, whose tokens are the first
      // tile's)
      const bool split = s.split != 0;
      const int nt = split ? (nb + 1 - w) / 2 : nb, stride = split ? 2 : 1, first = split ? w : 0;
      const int t1 = s.t0 + (split ? 0 : w * p.tq), tok = t1 + tok_in;  // in the request
      const bool mine = tok_in < p.tq && tok < s.n;
      const int lim = min(s.ctx + tok, s.ctx + s.n - 1);  // the last key this row sees
      const int jm = ((s.ctx + t1 + 1) >> 7) - k0;          // the first block that the tile does not wholly see
      float m = -INFINITY, l = 0.f, rowf = 0.f;
      int ve = 1;
      bool ok = true;
      // what is known of the next block, read while its scores are on their way
      float kf[8];
      uint32_t miss = 0;
      int now = 1, apart = 0;
      const auto look = [&](uint32_t n) {
        if (!wait_phase(&ctl.known[n & 7], (n >> 3) & 1, &patience)) return false;
        const Block& b = ctl.blocks[n & 7];
        miss = b.missing;
        now = b.ve;
        apart = b.apart;
#pragma unroll
        for (int e = 0; e < 8; ++e) kf[e] = b.ks[e >> per16];
        return true;
      };
      if (nt > 0) ok = look(blk + first);
      const int fold_slot = s.slot >= 0 ? s.slot : 2 * (int)blockIdx.x + 1;
#pragma unroll 1
      for (int j = 0, stop = kFold; ok;) {
        for (; j < min(nt, stop) && !apart; ++j) {
          if (!(ok = wait_phase(&ctl.s_full[w], ns & 1, &patience))) break;
          ++ns;
          tc_fence_after();
          const int jb = j * stride + first;  // the block
          if (jb >= jm || miss) {
            // scores of keys that the row does not see become -inf where they lie, 32 columns at a time (a loop,
            // for the sake of the code's size)
            const int last = lim - (k0 + jb) * 128;
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
              const int n = last + 1 - c;
              uint32_t see = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1;
              if (miss) see &= ~missing_keys(miss, c, p.page_shift);
              if (__all_sync(0xffffffffu, see == ~0u)) continue;
              float y[32];
              tmem_ld32(ts + c, y);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((see >> e) & 1)) y[e] = -INFINITY;
              tmem_st32(ts + c, y);
            }
            tmem_wait_st();
          }
          // softmax scale 2^(e - 134): what a row's scores are worth before the keys' scales
          if (j == 0) rowf = p.scale * unit_of(max((int)ctl.q_exp[i & 1][w][row] - 7, 1));
#pragma unroll
          for (int e = 0; e < 8; ++e) kf[e] = fmaxf(kf[e] * rowf, 0x1p-126f);  // (a masked score times 0 is NaN)
          float x[64];
          tmem_ld32(ts, x);
          tmem_ld32(ts + 32, x + 32);
          tmem_wait_ld();
          float top = most_of(x, kf);
          if (j == 0) {
            m = top;
            ve = now;
          } else {
            if constexpr (kApart) {  // the last block's product has read P, and O is whole
              if (!(ok = wait_phase(&ctl.o_done[w], no & 1, &patience))) break;
              ++no;
              tc_fence_after();
            }
            const bool far = top > m + 8.f;
            if (__any_sync(0xffffffffu, far || now != ve)) {
              // (at D = 128 the barrier of this block's S covers every product into O)
              const float f = far ? ex2(m - top) : 1.f;
              if (far) m = top;
              l *= f;
              rescale<D>(to, now - ve > 126 ? 0.f : f * unit_of(127 + ve - now));
              ve = now;
            }
          }
          float mu = m == -INFINITY ? 0.f : kBias - m;
          uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float* xc = x + (c & 1) * 32;
            if (c == 2) {
              // the second half of the scores: its maximum moves the row's only where it is far above the first half's,
              // whose product is waited for then
              tmem_wait_ld();
              if constexpr (kApart) {  // the next scores may come
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.s_free[w]);
              }
              top = most_of(x, kf + 4);
              const bool far = top > m + 8.f;
              if (__any_sync(0xffffffffu, far)) {
                if (!(ok = wait_phase(&ctl.half_done[w], np & 1, &patience))) break;
                tc_fence_after();
                const float f = far ? ex2(m - top) : 1.f;
                if (far) m = top;
                l *= f;
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] = mul2(sum[e], pair_f32(f, f));
                rescale<D>(to, f);
                mu = m == -INFINITY ? 0.f : kBias - m;
              }
            }
            const uint64_t mu2 = pair_f32(mu, mu);
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float f = kf[c * 2 + e / 8];
              const float2 y = unpair_f32(fma2(pair_f32(xc[2 * e], xc[2 * e + 1]), pair_f32(f, f), mu2));
              const float a = ex2(y.x), d = ex2(y.y);
              sum[e & 3] = add2(sum[e & 3], pair_f32(a, d));
              r[e] = pack_f16(a, d);
            }
            if (c < 2) tmem_ld32(ts + 64 + c * 32, xc);
            tmem_st16(tp + c * 16, r);
            if (c & 1) {  // half of the keys: the product starts on them
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&ctl.p_full[w][c >> 1]);
            }
          }
          if (!ok) break;
          ++np;
          const float2 t = unpair_f32(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
          l += t.x + t.y;
          if (j + 1 < nt && !(ok = look(blk + jb + stride))) break;
        }
        if (!ok || j >= nt) break;
        if (j < stop) {  // a block of codes
          if (!(ok = wait_phase(&ctl.s_full[w], ns & 1, &patience))) break;
          ++ns;
          if (kApart && j > 0) {
            if (!(ok = wait_phase(&ctl.o_done[w], no & 1, &patience))) break;
            ++no;
          }
          tc_fence_after();
          if (j == 0) rowf = p.scale * unit_of(max((int)ctl.q_exp[i & 1][w][row] - 7, 1));
          const int jb = j * stride + first;
          const RowState r = scores_apart<D>(p, ctl, w, (blk + jb) & 7, ts, to, tp, lim - (k0 + jb) * 128, rowf, {m, l, ve},
                                             j == 0);
          m = r.m;
          l = r.l;
          ve = r.ve;
          ++np;
          apart = 0;
          if (++j < nt) ok = look(blk + jb + stride);
          continue;
        }
        // O is whole once the next scores are there (at D = 64, once its last product is done)
        if (!(ok = wait_phase(kApart ? &ctl.o_done[w] : &ctl.s_full[w], (kApart ? no : ns) & 1, &patience))) break;
        tc_fence_after();
        l = fold_results(p, D, fold_slot, w * 128 + row, to, m, l, unit_of(ve), mine, stop > kFold, false);
        stop += kFold;
      }
      if (!ok) break;
      blk += s.k1 - k0;
      if (nt > 0) {
        if (!wait_phase(&ctl.o_done[w], no & 1, &patience)) break;
        ++no;
        tc_fence_after();
      }
      if (nt > kFold) {
        l = fold_results(p, D, fold_slot, w * 128 + row, to, m, l, unit_of(ve), mine, true, true);
        ve = 127;
      }
      // the two tiles of a split part: the second's maxima and sums go by shared memory, its results are read where they
      // are
      float fa = unit_of(ve), fb = 0.f;
      if (split && w == 1) {
        ctl.ml[row] = make_float2(m, l);
        ctl.second_ve[row] = (uint8_t)ve;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.second_done);
      } else if (split) {
        if (!wait_phase(&ctl.second_done, nsplit & 1, &patience)) break;
        tc_fence_after();
        const float2 other = ctl.ml[row];
        const float mn = fmaxf(m, other.x), mu = mn == -INFINITY ? 0.f : mn;
        const float f0 = ex2(m - mu), f1 = ex2(other.x - mu);
        m = mn;
        l = l * f0 + other.y * f1;
        fa *= f0;
        fb = unit_of(ctl.second_ve[row]) * f1;
      }
      const bool stores = mine && !(split && w == 1);
      const bool set_aside = nt > 0 && ctl.odd[sst];
      const float f = s.slot >= 0 ? 1.f : nt == 0 || l == 0.f ? 0.f : 1.0f / l;
      const bool none = nt == 0 || (s.slot < 0 && l == 0.f);  // a row without keys is zero
      __nv_bfloat16* dst = p.out + ((int64_t)s.row0 + (split ? 0 : w * p.tq) + tok_in) * p.ld_out + (int64_t)(s.g * p.G + head) * D;
      float4* rec = nullptr;
      if (s.slot >= 0) {
        rec = part_cols(p, D, s.slot, w * 128 + row, 0);
        if (stores) *reinterpret_cast<float2*>(part_ml(p, D, s.slot, w * 128 + row)) = make_float2(m, nt > 0 ? l : 0.f);
      }
      // (32-byte stores where a row allows it: lanes hold different rows, and each store takes a cycle per lane)
      const bool wide = (p.ld_out & 15) == 0 && (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
#pragma unroll 1
      for (int c = 0; c < (split && w == 1 ? 0 : D); c += 32) {
        float o[32];
        if (nt > 0) {
          tmem_ld32(to + c, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= fa;
        if (split) {
          float o1[32];
          tmem_ld32(to + D + c, o1);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = fmaf(o1[e], fb, o[e]);
        }
        if (set_aside && stores) {
          float add[32] = {};
          add_odd_values(p, s, lim, D, c, add);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] += add[e];
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : o[e] * f;
        if (stores && !rec) {
#pragma unroll
          for (int e = 0; e < 32; e += 16) {
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = pack_bf16(o[e + 2 * k], o[e + 2 * k + 1]);
            if (wide) {
              st_v8(dst + c + e, v);
            } else {
              *reinterpret_cast<uint4*>(dst + c + e) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(dst + c + e + 8) = make_uint4(v[4], v[5], v[6], v[7]);
            }
          }
        } else if (stores && nt > 0) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            rec[(c + e) / 4 * kTileRows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (split) {  // the second tile's results are read before it goes on
        if (w == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.second_read);
        } else if (!wait_phase(&ctl.second_read, nsplit & 1, &patience)) {
          break;
        }
        ++nsplit;
      }
      tc_fence_before();  // O is read before the next part's first P is handed over
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.seg_empty[sst]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_chunk8_t(const Attn8Params& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  static std::atomic<int> regs{0};
  cudaError_t e = allow_smem(chunk8_kernel<D>, Smem<D>::kBytes, &allowed);
  if (e != cudaSuccess) return e;
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes a;
    if ((e = cudaFuncGetAttributes(&a, chunk8_kernel<D>)) != cudaSuccess) return e;
    regs.store(a.numRegs, std::memory_order_relaxed);
  }
  // the register shares add up to this allocation: with fewer a warpgroup would wait for registers for ever (build.py
  // checks the compiler's count, so that this is met by builds of another kind only)
  if (regs.load(std::memory_order_relaxed) != kLaunchRegs) return cudaErrorInvalidKernelImage;
  return launch_early(chunk8_kernel<D>, dim3((unsigned)p.workers), dim3(kThreads), Smem<D>::kBytes, stream, p, qmap, kmap,
                      vmap);
}

}  // namespace

cudaError_t launch_chunk8(const Attn8Params& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, int D, cudaStream_t stream) {
  return D == 128 ? launch_chunk8_t<128>(p, qmap, kmap, vmap, stream) : launch_chunk8_t<64>(p, qmap, kmap, vmap, stream);
}

}  // namespace mk
