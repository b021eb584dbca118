// Norms of queries and keys for each head, the rotary embedding, and the
// stores of keys and values into pages of e4m3 with a scale for each page and
// head.
//
//   s = the smallest power of two, at least 2^-126, with max |x| <= 448 s
//
// over the page's new tokens and, where the page is begun (its first token is not
// among them), s at least its old scale; if that grows, what the page holds is
// rounded to the new one, e4m3(code s_old / s).  A power of two makes that exact but
// for codes that become subnormal, which are rounded twice then: others do not depend
// on the steps in which the page was filled.  A scale does not go down again before
// the page's first token is stored anew: one that a rejected draft raised stays, and
// what it rounded.
//
// Bound by bytes, as the bf16 form is (paged.cu): activations are read once,
// queries written in 16 bits, keys and values in 8.  A page's maximum has to
// be known before its first value is stored, so the unit of work is a run: the
// neighbouring rows that go to one page, of one key or value head.  A block
// takes the runs that begin in its window of rows, a few rows per pass, and
// follows the last of them behind the window.  Values stay in registers between
// the maximum and the store (those of runs that reach far behind the window are
// read again), each lane turns its pairs itself, and one warp finds the runs
// while the rows are on their way, so the block meets three times.
//
// A prompt of 8192 tokens, 8/32 heads of 128, bf16: 49 us, of which queries
// are 24.5 (5.5 TB/s) and keys and values the rest, where bytes alone would take 8
// (f32: 60.5 of 43):
// a third of the warps' time is the three meetings, a third the rows' first
// arrival.  Measured on the way: angles shared by a row's heads in shared memory
// 38 us for keys and values (more meetings), a warp alone per window and head,
// without any, 14 us for each of its runs of 64 rows.  One token 4.0 us, 64
// tokens of as many requests 4.3 us: the chain positions, runs, rows, store.
#include <cuda_fp16.h>

#include "paged_norm.cuh"

namespace mk {
namespace {

constexpr int kGap = 15;  // rows that are not stored which a run may have between two that are

struct Store8Params : NormParams {
  uint8_t *kcodes, *vcodes;
  float *kscale, *vscale;
  unsigned checks, kv_blocks;  // blocks that look for pages of two runs; of keys and values
};

template <typename T>
constexpr int kElems = sizeof(T) == 4 ? 4 : 8;  // of each half of a head, per lane
// A block of THREADS takes the runs that begin among WINDOW rows, ROWS at a time; the values of KEPT such passes stay in
// registers.
template <typename T_, int D_, int THREADS_, int WINDOW_, int KEPT_>
struct Shape {
  using T = T_;
  static constexpr int D = D_, THREADS = THREADS_, WINDOW = WINDOW_, KEPT = KEPT_;
  static constexpr int E = kElems<T>, LPH = D / 2 / E, ROWS = THREADS / LPH, PASSES = WINDOW / ROWS;
  static_assert(PASSES >= 1 && WINDOW % ROWS == 0 && KEPT >= PASSES && WINDOW <= 64, "the window's own rows are kept");
};

// Four coefficients of a pair, gains folded in: y_a = r (a ca + b sb), y_b = r (b cb + a sa).
template <int D>
struct Turn {
  float ca[D / 2], sb[D / 2], cb[D / 2], sa[D / 2];
};
template <int D>
__device__ __forceinline__ void make_turn(Turn<D>& t, int j, const Store8Params& p, int pos) {
  const __nv_bfloat16* gamma = p.q_gamma;
  const float ga = gamma ? __bfloat162float(gamma[j]) : 1.f, gb = gamma ? __bfloat162float(gamma[j + D / 2]) : 1.f;
  const uint64_t turn = (uint64_t)(uint32_t)pos * p.freq[j];
  float s, c;
  sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
  t.ca[j] = c * ga;
  t.sb[j] = -s * gb;
  t.cb[j] = c * gb;
  t.sa[j] = s * ga;
}

// Sines and cosines of two angles, in 2^-32 turns: the nearest quarter turn is taken off, the series of what is left (at
// most an eighth of a turn) are summed up to the terms under 2^-25, and the quarter turns swap and sign the two.
__device__ __forceinline__ void sincos2(const uint32_t (&turn)[2], uint64_t& sine, uint64_t& cosine) {
  float x[2];
  uint32_t quarter[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    quarter[e] = (turn[e] + 0x20000000u) >> 30;
    x[e] = (float)(int32_t)(turn[e] - (quarter[e] << 30)) * (0x1p-31f * 3.14159265f);
  }
  const auto both = [](float c) { return ptx::pair_f32(c, c); };
  const uint64_t a = ptx::pair_f32(x[0], x[1]), a2 = ptx::mul2(a, a);
  uint64_t s = ptx::fma2(a2, both(1.f / 362880.f), both(-1.f / 5040.f));
  uint64_t c = ptx::fma2(a2, both(1.f / 40320.f), both(-1.f / 720.f));
  s = ptx::fma2(a2, s, both(1.f / 120.f));
  c = ptx::fma2(a2, c, both(1.f / 24.f));
  s = ptx::fma2(a2, s, both(-1.f / 6.f));
  c = ptx::fma2(a2, c, both(-0.5f));
  s = ptx::fma2(ptx::mul2(a2, a), s, a);
  c = ptx::fma2(a2, c, both(1.f));
  const float2 s1 = ptx::unpair_f32(s), c1 = ptx::unpair_f32(c);
  float sv[2] = {s1.x, s1.y}, cv[2] = {c1.x, c1.y};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float u = quarter[e] & 1 ? cv[e] : sv[e], v = quarter[e] & 1 ? sv[e] : cv[e];
    sv[e] = __uint_as_float(__float_as_uint(u) ^ (quarter[e] & 2) << 30);
    cv[e] = __uint_as_float(__float_as_uint(v) ^ ((quarter[e] + 1) & 2) << 30);
  }
  sine = ptx::pair_f32(sv[0], sv[1]);
  cosine = ptx::pair_f32(cv[0], cv[1]);
}

// A lane's elements of a head, normed (`norm`) and turned.  The lanes of `mask` hold the head.
template <int E, int D>
__device__ __forceinline__ void norm_turn(float (&a)[E], float (&b)[E], const Turn<D>& t, int gl, bool norm, float eps,
                                          unsigned mask) {
  constexpr int LPH = D / 2 / E;
  float r = 1.f;
  if (norm) {
    uint64_t ss = 0;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const uint64_t u = ptx::pair_f32(a[i], a[i + 1]), v = ptx::pair_f32(b[i], b[i + 1]);
      ss = ptx::fma2(u, u, ptx::fma2(v, v, ss));
    }
    const float2 two = ptx::unpair_f32(ss);
    float sum = two.x + two.y;
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
    r = rsqrtf(sum * (1.0f / D) + eps);
  }
  const uint64_t r2 = ptx::pair_f32(r, r);
#pragma unroll
  for (int i = 0; i < E; i += 4) {
    const float4 ca = *reinterpret_cast<const float4*>(t.ca + gl * E + i);
    const float4 sb = *reinterpret_cast<const float4*>(t.sb + gl * E + i);
    const float4 cb = *reinterpret_cast<const float4*>(t.cb + gl * E + i);
    const float4 sa = *reinterpret_cast<const float4*>(t.sa + gl * E + i);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = i + 2 * e;
      const uint64_t u = ptx::mul2(r2, ptx::pair_f32(a[k], a[k + 1])), v = ptx::mul2(r2, ptx::pair_f32(b[k], b[k + 1]));
      const uint64_t c1 = e ? ptx::pair_f32(ca.z, ca.w) : ptx::pair_f32(ca.x, ca.y);
      const uint64_t s1 = e ? ptx::pair_f32(sb.z, sb.w) : ptx::pair_f32(sb.x, sb.y);
      const uint64_t c2 = e ? ptx::pair_f32(cb.z, cb.w) : ptx::pair_f32(cb.x, cb.y);
      const uint64_t s2 = e ? ptx::pair_f32(sa.z, sa.w) : ptx::pair_f32(sa.x, sa.y);
      const float2 ya = ptx::unpair_f32(ptx::fma2(v, s1, ptx::mul2(u, c1)));
      const float2 yb = ptx::unpair_f32(ptx::fma2(u, s2, ptx::mul2(v, c2)));
      a[k] = ya.x;
      a[k + 1] = ya.y;
      b[k] = yb.x;
      b[k + 1] = yb.y;
    }
  }
}

// The smallest power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 * 2^8), for a finite amax >= 0.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// Two values to e4m3, the first in the low byte; what is not finite becomes NaN (it was made NaN before).
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int E>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* v, float inv) {
  uint32_t w[E / 4];
#pragma unroll
  for (int i = 0; i < E; i += 4)
    w[i / 4] = pack_e4m3(v[i] * inv, v[i + 1] * inv) | pack_e4m3(v[i + 2] * inv, v[i + 3] * inv) << 16;
  if constexpr (E == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(p) = w[0];
}
__device__ __forceinline__ uint32_t rescale2(uint32_t two, float by) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_e4m3(f.x * by, f.y * by);
}
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float by) {
  return rescale2(w & 0xFFFFu, by) | rescale2(w >> 16, by) << 16;
}

// What a block keeps in shared memory.
template <int WINDOW, int D>
struct Runs {
  static constexpr int BACK = kGap + 1, SPAN = BACK + WINDOW + 64;  // rows around the window that are looked at at once
  uint64_t freq[D / 2];
  float2 gain[D / 2];               // of both elements of a pair
  int slot[SPAN], pos[SPAN];
  int run[WINDOW];                  // the first row of a row's run; -1: of another window's, or none
  uint64_t leads;                   // rows that begin a run
  int more;                         // rows behind the window up to the end of the last run
  unsigned top[WINDOW];             // maxima of the runs, by first row
  float inv[WINDOW], again[WINDOW]; // 1 / scale; what held codes are multiplied with (1: they stay)
  unsigned written[WINDOW][8];      // offsets that a run writes, where what a page holds is looked at again
  int upto[WINDOW];                 // the last one
  int grown;
};

// The slot of a row; -1: it is not stored, kNoPage: it should be, outside of the pool.
constexpr int kNoPage = -2;
__device__ __forceinline__ int stored_slot(const Store8Params& p, int slot, int pos) {
  return (slot | pos) < 0 ? -1 : (slot >> p.page_shift) < p.num_pages ? slot : kNoPage;
}
// The same of row r, and its position
__device__ __forceinline__ int stored_row(const Store8Params& p, int64_t r, int& pos) {
  if (r < 0 || r >= p.N) return pos = -1;
  const int slot = p.slots[r];
  pos = p.positions[r];
  return stored_slot(p, slot, pos);
}

// Two runs of a page would set its scale both, each for its own rows.  None of the blocks that store them sees the other,
// so blocks of their own, before those, look at all rows and mark the page of each that begins a run in a bitmap; a page
// that is marked already is reported.  A block per kSeen pages of the pool.  These blocks are short while a thread has few
// rows; a call of more has them in a launch of their own with more threads, and the stores beside it.
constexpr int kSeen = 65536;
struct Seen {
  unsigned bits[kSeen / 32];
};
// Row r goes to `slot`; `before`: the slot of the row before, where that is stored.
__device__ __forceinline__ void mark_run(const Store8Params& p, Seen& sm, int first, int64_t r, int slot, int before) {
  if (slot < 0) return;
  if (before < 0) {
    int pos;
#pragma unroll 1
    for (int i = 2; i <= kGap + 1 && before < 0; ++i) before = stored_row(p, r - i, pos);
  }
  if (before >= 0 && (before ^ slot) >> p.page_shift == 0) return;  // goes on
  const unsigned at = (unsigned)((slot >> p.page_shift) - first);
  if (at < kSeen && (atomicOr(&sm.bits[at / 32], 1u << (at % 32)) >> (at % 32) & 1)) set_status(p.status, MK_DEV_BAD_INDEX);
}
// (Out of line: inlined, 777 mixed rows took 7.4 us for 7.2.)
template <int THREADS>
__device__ __noinline__ void check_runs(const Store8Params& p, Seen& sm, unsigned part) {
  constexpr unsigned AHEAD = 4;  // rows of a thread on their way
  const int first = (int)part * kSeen;
  const unsigned lane = threadIdx.x % 32, n = p.N;
  for (int i = threadIdx.x; i < kSeen / 32; i += THREADS) sm.bits[i] = 0;
  __syncthreads();
#pragma unroll 1
  for (unsigned base = threadIdx.x - lane; base < n; base += AHEAD * THREADS) {
    int slot[AHEAD][2], pos[AHEAD][2];  // of a row, and of the one before
#pragma unroll
    for (unsigned k = 0; k < AHEAD; ++k) {
      const unsigned r = min(base + k * THREADS + lane, n - 1), before = r > 0 ? r - 1 : 0;
      slot[k][0] = p.slots[r];
      pos[k][0] = p.positions[r];
      slot[k][1] = p.slots[before];
      pos[k][1] = p.positions[before];
    }
#pragma unroll
    for (unsigned k = 0; k < AHEAD; ++k) {
      const unsigned r = base + k * THREADS + lane;
      if (r < n)
        mark_run(p, sm, first, r, stored_slot(p, slot[k][0], pos[k][0]), r > 0 ? stored_slot(p, slot[k][1], pos[k][1]) : -1);
    }
  }
}

// The runs of a key or value head that begin in a window; the rows of a run go to one page, each at a higher offset than
// the one before.
template <typename S>
__device__ __forceinline__ void store_runs(const Store8Params& p, Runs<S::WINDOW, S::D>& sm, unsigned block) {
  using T = typename S::T;
  constexpr int D = S::D, E = S::E, LPH = S::LPH, ROWS = S::ROWS, WINDOW = S::WINDOW, PASSES = S::PASSES, KEPT = S::KEPT;
  constexpr int THREADS = S::THREADS, BACK = Runs<WINDOW, D>::BACK, SPAN = Runs<WINDOW, D>::SPAN;
  const int tid = threadIdx.x, lane = tid % 32, gl = tid % LPH, group = tid / LPH;
  const int hh = block % (2 * p.Hkv);
  const int64_t r0 = (int64_t)(block / (2 * p.Hkv)) * WINDOW;
  const bool is_v = hh >= p.Hkv;
  const int head = is_v ? hh - p.Hkv : hh, page = 1 << p.page_shift;
  const unsigned mask = (LPH == 32 ? 0xffffffffu : ((1u << LPH) - 1u)) << (lane / LPH * LPH);
  const T* base = static_cast<const T*>(p.x) + (int64_t)(p.Hq + hh) * D + gl * E;
  const auto slot_at = [&](int64_t r, int& pos) { return stored_row(p, r, pos); };
  // the slot of row r0 + i
  const auto slot_of = [&](int i) {
    int pos;
    return i < SPAN - BACK ? sm.slot[BACK + i] : slot_at(r0 + i, pos);
  };
  // the window's rows are on their way while their runs are found (where a page may be larger than the window, many
  // windows have no run of their own)
  const bool early = page <= WINDOW;
  Raw<T, E> ra[KEPT], rb[KEPT];
  const auto load = [&](int w, Raw<T, E>& a, Raw<T, E>& b) {
    const T* x = base + (r0 + w * ROWS + group) * p.ld_x;
    a.load(x);
    b.load(x + D / 2);
  };
  if (tid < 32) {
    // the first warp finds the runs
    // (all loads, then what is made of them: with both in one loop a prompt of 8192 tokens took 53 us for 49)
    constexpr int LOADS = (SPAN + 31) / 32;
    int slots[LOADS], at[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      const int64_t r = r0 - BACK + k * 32 + lane;
      const bool there = r >= 0 && r < p.N;
      slots[k] = there ? p.slots[r] : -1;
      at[k] = there ? p.positions[r] : -1;
    }
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      const int i = k * 32 + lane;
      if (i >= SPAN) break;
      sm.slot[i] = stored_slot(p, slots[k], at[k]);
      sm.pos[i] = at[k];
    }
    __syncwarp();
    const auto same_page = [&](int a, int b) { return b >= 0 && (a >> p.page_shift) == (b >> p.page_shift); };
    // the slot of the nearest stored row before row r0 + i
    const auto before_of = [&](int i) {
      int b = slot_of(i - 1);
#pragma unroll 1
      for (int k = 2; k <= BACK && b < 0; ++k) b = slot_of(i - k);
      return b;
    };
    uint64_t leads = 0, ends = 0;  // rows that begin a run, and all that end one
#pragma unroll
    for (int i0 = 0; i0 < WINDOW; i0 += 32) {
      const int i = i0 + lane, slot = i < WINDOW ? sm.slot[BACK + i] : -1, before = slot >= 0 ? before_of(i) : -1;
      const bool again_page = slot >= 0 && same_page(slot, before);
      // a page that comes again in another order: two runs would both set its scale
      const bool twice = again_page && slot <= before;
      if (hh == 0 && (slot == kNoPage || twice)) set_status(p.status, MK_DEV_BAD_INDEX);
      const unsigned l = __ballot_sync(0xffffffffu, slot >= 0 && !again_page);
      const unsigned t = __ballot_sync(0xffffffffu, twice);
      leads |= (uint64_t)l << i0;
      ends |= (uint64_t)(l | t) << i0;
    }
    const auto run_of = [&](int row) {
      const uint64_t e = ends & ((2ull << row) - 1ull);
      const int at = e ? 63 - __clzll((long long)e) : -1;
      return at >= 0 && (leads >> at & 1) ? at : -1;
    };
    for (int i = lane; i < WINDOW; i += 32) sm.run[i] = sm.slot[BACK + i] >= 0 ? run_of(i) : -1;
    // the last run's rows behind the window
    int more = 0;
    const bool goes_on = run_of(WINDOW - 1) >= 0;
#pragma unroll 1
    for (int i0 = WINDOW; goes_on; i0 += 32) {
      const int i = i0 + lane, slot = slot_of(i), before = slot >= 0 ? before_of(i) : -1;
      const bool on = slot >= 0 && same_page(slot, before) && slot > before;
      const unsigned stop = __ballot_sync(0xffffffffu, slot >= 0 && !on);
      const unsigned all = __ballot_sync(0xffffffffu, on), mine = stop ? all & ((stop & -stop) - 1) : all;
      if (mine) more = i0 - WINDOW + 32 - __clz((int)mine);
      if (stop || !all) break;  // (a run goes on within BACK rows)
    }
    if (lane == 0) {
      sm.leads = leads;
      sm.more = more;
      sm.grown = 0;
    }
  } else if (!is_v) {
    for (int j = tid - 32; j < D / 2; j += THREADS - 32) {
      sm.freq[j] = p.freq[j];
      sm.gain[j] = p.k_gamma ? make_float2(__bfloat162float(p.k_gamma[j]), __bfloat162float(p.k_gamma[j + D / 2]))
                             : make_float2(1.f, 1.f);
    }
  }
  if (early) {
#pragma unroll
    for (int w = 0; w < PASSES; ++w)
      if (r0 + w * ROWS + group < p.N) load(w, ra[w], rb[w]);
  }
  for (int i = tid; i < WINDOW; i += THREADS) sm.top[i] = 0;
  __syncthreads();
  const uint64_t lead_bits = sm.leads;
  if (lead_bits == 0) return;
  const int more = sm.more, passes = PASSES + (more + ROWS - 1) / ROWS;
  const int last = passes > PASSES ? sm.run[63 - __clzll((long long)lead_bits)] : 0;  // the run that goes on
  // this group's row of a pass: its run, and its slot (-1: none of this window's)
  const auto run_in = [&](int w) { return w < PASSES ? sm.run[w * ROWS + group] : last; };
  const auto slot_in = [&](int w) {
    const int i = w * ROWS + group;
    if (w < PASSES) return sm.run[i] >= 0 ? sm.slot[BACK + i] : -1;
    return i - WINDOW < more ? slot_of(i) : -1;
  };
  // the values to be stored
  const auto values = [&](int w, const Raw<T, E>& ra, const Raw<T, E>& rb, float (&a)[E], float (&b)[E]) {
    ra.get(a);
    rb.get(b);
    if (!is_v) {
      float r = 1.f;
      if (p.k_gamma) {
        uint64_t ss = 0;
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          const uint64_t u = ptx::pair_f32(a[i], a[i + 1]), v = ptx::pair_f32(b[i], b[i + 1]);
          ss = ptx::fma2(u, u, ptx::fma2(v, v, ss));
        }
        const float2 two = ptx::unpair_f32(ss);
        float sum = two.x + two.y;
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
        r = rsqrtf(sum * (1.0f / D) + p.eps);
      }
      const int k = w * ROWS + group;
      int pos;
      if (k < SPAN - BACK) pos = sm.pos[BACK + k];
      else slot_at(r0 + k, pos);
      const uint64_t r2 = ptx::pair_f32(r, r);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        uint32_t turn[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) turn[e] = (uint32_t)((uint64_t)(uint32_t)pos * sm.freq[gl * E + i + e] >> 32);
        uint64_t s2, c2;
        sincos2(turn, s2, c2);
        const float2 g0 = sm.gain[gl * E + i], g1 = sm.gain[gl * E + i + 1];
        const uint64_t u = ptx::mul2(ptx::mul2(r2, ptx::pair_f32(g0.x, g1.x)), ptx::pair_f32(a[i], a[i + 1]));
        const uint64_t v = ptx::mul2(ptx::mul2(r2, ptx::pair_f32(g0.y, g1.y)), ptx::pair_f32(b[i], b[i + 1]));
        const uint64_t n2 = s2 ^ 0x8000000080000000ull;
        const float2 ya = ptx::unpair_f32(ptx::fma2(v, n2, ptx::mul2(u, c2)));
        const float2 yb = ptx::unpair_f32(ptx::fma2(u, s2, ptx::mul2(v, c2)));
        a[i] = ya.x;
        a[i + 1] = ya.y;
        b[i] = yb.x;
        b[i + 1] = yb.y;
      }
    }
#pragma unroll
    for (int i = 0; i < E; i += 2) {  // an infinity becomes NaN
      const uint64_t u = ptx::pair_f32(a[i], a[i + 1]), v = ptx::pair_f32(b[i], b[i + 1]);
      const float2 x = ptx::unpair_f32(ptx::fma2(u, 0, u)), y = ptx::unpair_f32(ptx::fma2(v, 0, v));
      a[i] = x.x;
      a[i + 1] = x.y;
      b[i] = y.x;
      b[i + 1] = y.y;
    }
  };
  const auto raise = [&](int run, const float (&a)[E], const float (&b)[E]) {
    float m = 0.f;  // (a maximum leaves NaN out)
#pragma unroll
    for (int i = 0; i < E; ++i) m = fmaxf(m, fmaxf(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
    if (gl == 0) atomicMax(&sm.top[run], __float_as_uint(m));
  };
  int slot_k[KEPT], run_k[KEPT];
#pragma unroll
  for (int w = 0; w < KEPT; ++w) {
    slot_k[w] = w < passes ? slot_in(w) : -1;
    run_k[w] = max(run_in(w), 0);
    if ((w >= PASSES || !early) && slot_k[w] >= 0) load(w, ra[w], rb[w]);
  }
  float ka[KEPT][E], kb[KEPT][E];
#pragma unroll
  for (int w = 0; w < KEPT; ++w) {
    if (slot_k[w] < 0) continue;  // (whole lane groups; the shuffles name their lanes only)
    values(w, ra[w], rb[w], ka[w], kb[w]);
    raise(run_k[w], ka[w], kb[w]);
  }
#pragma unroll 1
  for (int w = KEPT; w < passes; ++w) {
    if (slot_in(w) < 0) continue;
    Raw<T, E> xa, xb;
    float a[E], b[E];
    load(w, xa, xb);
    values(w, xa, xb, a, b);
    raise(last, a, b);
  }
  __syncthreads();
  float* scales = is_v ? p.vscale : p.kscale;
  uint8_t* codes = is_v ? p.vcodes : p.kcodes;
  if (tid < WINDOW && (lead_bits >> tid & 1)) {
    const int slot = sm.slot[BACK + tid];
    float* at = scales + (int64_t)(slot >> p.page_shift) * p.Hkv + head;
    float s = scale_for(__uint_as_float(sm.top[tid])), by = 1.f;
    if ((slot & (page - 1)) != 0) {  // a page that is begun
      const float old = *at;
      if (old >= s) s = old;
      else by = old / s;
      if (by != 1.f) sm.grown = 1;
    }
    *at = s;
    sm.inv[tid] = 1.f / s;
    sm.again[tid] = by;
  }
  __syncthreads();
  if (sm.grown) {
    // pages whose scale grew: what they hold below the last new row, but for what is new
    for (int i = tid; i < WINDOW; i += THREADS) sm.upto[i] = 0;
    for (int i = tid; i < WINDOW * 8; i += THREADS) sm.written[i / 8][i % 8] = 0;
    __syncthreads();
    for (int w = 0; w < passes; ++w) {
      const int slot = slot_in(w), off = slot & (page - 1);
      if (gl != 0 || slot < 0) continue;
      atomicOr(&sm.written[run_in(w)][off / 32], 1u << (off % 32));
      atomicMax(&sm.upto[run_in(w)], off);
    }
    __syncthreads();
    for (uint64_t rest = lead_bits; rest; rest &= rest - 1) {
      const int i = __ffsll((long long)rest) - 1;
      const float by = sm.again[i];
      if (by == 1.f) continue;
      uint4* at = reinterpret_cast<uint4*>(
          codes + (((int64_t)(sm.slot[BACK + i] >> p.page_shift) * p.Hkv + head) << p.page_shift) * D);
      for (int j = tid; j < sm.upto[i] * (D / 16); j += THREADS) {
        const int off = j / (D / 16);
        if (sm.written[i][off / 32] >> (off % 32) & 1) continue;
        uint4 v = at[j];
        v.x = rescale4(v.x, by); v.y = rescale4(v.y, by); v.z = rescale4(v.z, by); v.w = rescale4(v.w, by);
        at[j] = v;
      }
    }
  }
  const auto put = [&](int slot, int run, const float (&a)[E], const float (&b)[E]) {
    uint8_t* dst = codes + ((((int64_t)(slot >> p.page_shift) * p.Hkv + head) << p.page_shift) + (slot & (page - 1))) * D +
                   gl * E;
    const float inv = sm.inv[run];
    store_codes<E>(dst, a, inv);
    store_codes<E>(dst + D / 2, b, inv);
  };
#pragma unroll
  for (int w = 0; w < KEPT; ++w)
    if (slot_k[w] >= 0) put(slot_k[w], run_k[w], ka[w], kb[w]);
#pragma unroll 1
  for (int w = KEPT; w < passes; ++w) {
    const int slot = slot_in(w);
    if (slot < 0) continue;
    Raw<T, E> xa, xb;
    float a[E], b[E];
    load(w, xa, xb);
    values(w, xa, xb, a, b);
    put(slot, last, a, b);
  }
}

// Windows of 16 rows in one launch with the queries while the lanes that keys and values have work for are about half
// of what the GPU holds at once; else windows of 64 in a launch of their own, the queries' beside it.  One launch and two,
// 8/32 heads of bf16: 256 tokens 6.7 and 5.7 us, 512 7.0 and 9.2, 1024 8.9 and 10.8, 2048 17.3 and 16.8, 8192 61 and
// 49; 16/64 heads: 600 tokens 10.9 and 14.8, 1024 20.2 and 17.3; 512 requests of one token 6.2 and 9.3.  (Tokens that
// follow one another in pages of 64 and more of few heads would rather have two: 600 of 1/8 heads 13.2 and 10.6 us, of 4/32
// heads of 64 6.5 and 4.8; the rule does not know how long runs are.)
constexpr int kFewLanes = 160 * 1024;
// Three blocks of 256 threads and 64 rows per SM: a prompt of 8192 tokens 49 us.  Two of them 54, four 48 (but 41 for
// 39 where eleven ragged chunks meet); earlier, at 51, four of 128 threads and 32 rows took 60.  Blocks that stay and take the heads of a
// window one after the other, its runs found once and the next head's rows on their way, took 52.
constexpr int kKvThreads = 256, kKvWindow = 64, kKvBlocks = 3;
constexpr int kQueryBatch = 3;      // heads a lane group has in flight
constexpr int kQueryMaxTokens = 4;  // tokens of a block of queries

template <typename S>
__device__ __forceinline__ void queries(const Store8Params& p, Turn<S::D>* turns, unsigned block) {
  using T = typename S::T;
  constexpr int D = S::D, E = S::E, LPH = S::LPH, GP = S::ROWS, THREADS = S::THREADS;
  const int gl = threadIdx.x % LPH, group = threadIdx.x / LPH;
  const int gt = GP / p.tokens, tk = group / gt;
  const int64_t row0 = (int64_t)(block / p.splits) * p.tokens, row = row0 + tk;
  const int step = gt * p.splits, h0 = group % gt + block % p.splits * gt;
  const unsigned mask = (LPH == 32 ? 0xffffffffu : ((1u << LPH) - 1u)) << ((threadIdx.x & 31) / LPH * LPH);
  const bool in = row < p.N;
  const T* x = static_cast<const T*>(p.x) + (in ? row : 0) * p.ld_x + gl * E;
  __nv_bfloat16* q = p.q + row * p.ld_q + gl * E;
  int pos = -1;
  for (int h = h0; h < p.Hq || h == h0; h += kQueryBatch * step) {
    Raw<T, E> ra[kQueryBatch], rb[kQueryBatch];
#pragma unroll
    for (int k = 0; k < kQueryBatch; ++k) {
      const int hk = h + k * step;
      if (hk < p.Hq) {
        ra[k].load(x + hk * D);
        rb[k].load(x + hk * D + D / 2);
      }
    }
    if (h == h0) {
      if (in) pos = p.positions[row];
      for (int i = threadIdx.x; i < p.tokens * (D / 2); i += THREADS) {
        const int64_t r = row0 + i / (D / 2);
        make_turn<D>(turns[i / (D / 2)], i % (D / 2), p, r < p.N ? p.positions[r] : 0);
      }
      __syncthreads();
    }
    if (pos < 0) break;  // left out (whole lane groups; the shuffles name their lanes only)
#pragma unroll
    for (int k = 0; k < kQueryBatch; ++k) {
      const int hk = h + k * step;
      if (hk >= p.Hq) break;
      float a[E], b[E];
      ra[k].get(a);
      rb[k].get(b);
      norm_turn<E, D>(a, b, turns[tk], gl, p.q_gamma != nullptr, p.eps, mask);
      store_half<E>(q + hk * D, a);
      store_half<E>(q + hk * D + D / 2, b);
    }
  }
}

// Keys and values first, then the queries, in one launch.  Threads that an SM holds are worth a few spilled registers: 777
// rows of f32 with 768 of them 7.2 us, with 512 8.6; 1024 tokens of bf16 with 512 8.6, with 384 9.8.
template <typename T>
constexpr int kMixedThreads = sizeof(T) == 4 ? 768 : 512;
// BEHIND: beside a launch that looks for pages of two runs (check8_kernel); the last block ends behind it.
template <typename S, bool BEHIND>
__global__ void __launch_bounds__(S::THREADS, kMixedThreads<typename S::T> / S::THREADS) store8_kernel(const __grid_constant__ Store8Params p) {
  __shared__ union alignas(16) Any {
    __device__ Any() {}
    Runs<S::WINDOW, S::D> runs;
    Turn<S::D> turns[kQueryMaxTokens];
    Seen seen;
  } sm;
  const unsigned block = blockIdx.x;
  if (block < p.checks) check_runs<S::THREADS>(p, sm.seen, block);
  else if (block < p.checks + p.kv_blocks) store_runs<S>(p, sm.runs, block - p.checks);
  else queries<S>(p, sm.turns, block - p.checks - p.kv_blocks);
  if (BEHIND && block == gridDim.x - 1) ptx::wait_dependency();
}
// Keys and values alone
template <typename S, bool BEHIND>
__global__ void __launch_bounds__(S::THREADS, kKvBlocks) store8_kv_kernel(const __grid_constant__ Store8Params p) {
  __shared__ union alignas(16) Either {
    __device__ Either() {}
    Runs<S::WINDOW, S::D> runs;
    Seen seen;
  } sm;
  ptx::launch_dependents();  // the queries' blocks follow as these end
  if (blockIdx.x < p.checks) check_runs<S::THREADS>(p, sm.seen, blockIdx.x);
  else store_runs<S>(p, sm.runs, blockIdx.x - p.checks);
  if (BEHIND && blockIdx.x == gridDim.x - 1) ptx::wait_dependency();
}
constexpr int kCheckThreads = 1024;
__global__ void __launch_bounds__(kCheckThreads, 1) check8_kernel(const __grid_constant__ Store8Params p) {
  __shared__ Seen seen;
  ptx::launch_dependents();  // the stores' blocks follow
  check_runs<kCheckThreads>(p, seen, blockIdx.x);
}

// Rows of a thread (windows of 16) and of a call (windows of 64) up to which the stores' launch looks for pages of two
// runs, in the time that the stores take anyway.  In it and in a launch of its own: 1024 tokens of 32/4 heads of 64 6.5 and
// 7.0 us, 1536 8.3 and 7.4 (6.5 without looking); 2000 requests of one head 8.6 and 5.1; 16000 tokens of one head 37 and
// 11.8 (10.5 without).  60000 tokens of 8/2 heads 93 us in a launch of its own.
constexpr int kCheckRows = 16, kKvCheckRows = 16384;

template <typename T, int D>
cudaError_t launch_store8(Store8Params& p, int sms, cudaStream_t stream) {
  constexpr int E = kElems<T>, LPH = D / 2 / E;
  const auto kv_blocks = [&](int window) { return (unsigned)(((int64_t)p.N + window - 1) / window * 2 * p.Hkv); };
  // the blocks that look for pages of two runs (which have a row of another between them): in the stores' launch up to
  // `rows` rows, else in one that the stores follow beside
  p.checks = p.status && p.N > 2 ? (unsigned)((p.num_pages - 1) / kSeen + 1) : 0;
  const auto launch = [&](auto* kernel, auto* kernel_behind, int rows, unsigned blocks, int threads) {
    if (p.checks == 0 || p.N <= rows) {
      kernel<<<p.checks + blocks, threads, 0, stream>>>(p);
      return cudaGetLastError();
    }
    check8_kernel<<<p.checks, kCheckThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.checks = 0;
    return launch_early(kernel_behind, dim3(blocks), dim3(threads), 0, stream, p);
  };
  if ((int64_t)p.N * 2 * p.Hkv * LPH > kFewLanes) {
    using S = Shape<T, D, kKvThreads, kKvWindow, kKvWindow / (kKvThreads / LPH)>;
    const cudaError_t e = launch(store8_kv_kernel<S, false>, store8_kv_kernel<S, true>, kKvCheckRows, kv_blocks(S::WINDOW),
                                 S::THREADS);
    if (e != cudaSuccess) return e;
    return launch_queries(p, sizeof(T) == 4 ? MK_F32 : MK_BF16, D, sms, stream);
  }
  using S = Shape<T, D, 16 * LPH, 16, 5>;
  constexpr int GP = S::ROWS;
  // tokens whose heads fill a block's batch; few tokens: a head per lane group, over several blocks
  p.tokens = 1;
  while (p.tokens < kQueryMaxTokens && 2 * p.tokens * p.Hq <= kQueryBatch * GP) p.tokens *= 2;
  while (p.tokens > 1 && (p.N + p.tokens - 1) / p.tokens < 2 * sms) p.tokens /= 2;
  p.splits = p.N < sms ? (p.Hq + GP - 1) / GP : 1;
  p.kv_blocks = kv_blocks(S::WINDOW);
  const unsigned blocks = p.kv_blocks + (unsigned)((p.N + p.tokens - 1) / p.tokens * p.splits);
  return launch(store8_kernel<S, false>, store8_kernel<S, true>, kCheckRows * S::THREADS, blocks, S::THREADS);
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_qk_norm_rope_e4m3(void* stream, int N, int Hq, int Hkv, int D, const void* qkv, int qkv_dtype,
                                    int64_t ld_qkv, const void* q_gamma, const void* k_gamma, float eps,
                                    double rope_theta, const int32_t* positions, const int32_t* slots, void* q_out,
                                    int64_t ld_q, void* kpool, void* vpool, float* kscale, float* vscale,
                                    int num_pages, int page_size, int32_t* status) try {
  const char* who = "mk_qk_norm_rope_e4m3";
  if (int rc = check_norm(who, N, Hq, Hkv, D, qkv, qkv_dtype, ld_qkv, q_gamma, k_gamma, eps, rope_theta, positions,
                          slots, q_out, ld_q, kpool, vpool, num_pages, page_size))
    return rc;
  if (!kscale || !vscale) return fail(MK_ERR_ARG, "mk_qk_norm_rope_e4m3: null argument");
  // (blocks of a launch)
  if (((int64_t)N + 63) / 64 * 2 * Hkv + num_pages / kSeen + 1 > INT32_MAX || (int64_t)N * ((Hq + 2 * Hkv) / 8 + 1) > INT32_MAX)
    return fail(MK_ERR_LIMIT, "mk_qk_norm_rope_e4m3: too many rows");
  if (int rc = pending_error(who)) return rc;
  if (N == 0) return MK_OK;
  Store8Params p{};
  p.x = qkv; p.ld_x = ld_qkv; p.ld_q = ld_q;
  p.q_gamma = static_cast<const __nv_bfloat16*>(q_gamma);
  p.k_gamma = static_cast<const __nv_bfloat16*>(k_gamma);
  p.positions = positions; p.slots = slots;
  p.q = static_cast<__nv_bfloat16*>(q_out);
  p.kcodes = static_cast<uint8_t*>(kpool);
  p.vcodes = static_cast<uint8_t*>(vpool);
  p.kscale = kscale; p.vscale = vscale;
  p.status = status; p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.num_pages = num_pages; p.eps = eps;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  rope_frequencies(rope_theta, D, p.freq);
  int sms = 0;
  if (int rc = device_sms(who, &sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (qkv_dtype == MK_F32) e = D == 128 ? launch_store8<float, 128>(p, sms, s) : launch_store8<float, 64>(p, sms, s);
  else e = D == 128 ? launch_store8<__nv_bfloat16, 128>(p, sms, s) : launch_store8<__nv_bfloat16, 64>(p, sms, s);
  return launch_result(e, who);
} catch (...) {
  return MK_ERR_NOMEM;
}
