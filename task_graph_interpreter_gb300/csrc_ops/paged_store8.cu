// Norms of queries and keys for each head, the rotary embedding, and the
// stores of keys and values into pages of e4m3 with a scale for each page and
// head.
//
//   s = the smallest power of two, at least 2^-126, with max |x| <= 448 s
//
// over the page's new tokens and, where the page is begun (its first token is not
// among them), s at least its old scale; if that grows, what the page holds is
// rounded to the new one, e4m3(code s_old / s).  A power of two makes that exact but for codes that
// become subnormal, and a stored value does not depend on the steps in which
// the page was filled.
//
// Bound by bytes, as the bf16 form is (paged.cu): activations are read once,
// queries written in 16 bits, keys and values in 8.  A page's maximum has to
// be known before its first value is stored, so the unit of work is a run: the
// neighbouring rows that go to one page, of one key or value head.  A block
// takes the runs that begin in its window of 16 rows, a row per lane group,
// follows the last of them over up to four more windows, whose values stay in
// registers between the maximum and the store (rows of longer runs are read
// again), and holds a row's angles in shared memory, one window at a time.
// Blocks of queries follow those of keys and values in the same launch.
#include <cuda_fp16.h>

#include "paged_norm.cuh"

namespace mk {
namespace {

constexpr int kGap = 15;  // rows that are not stored which a run may have between two that are

struct Store8Params : NormParams {
  uint8_t *kcodes, *vcodes;
  float *kscale, *vscale;
  unsigned kv_blocks;
};

template <typename T>
constexpr int kElems = sizeof(T) == 4 ? 4 : 8;  // of each half of a head, per lane
// A block of THREADS takes the runs that begin among WINDOW rows, ROWS at a time; the values of KEPT such passes stay in
// registers.
template <typename T_, int D_, int THREADS_, int WINDOW_, int VALUES>
struct Shape {
  using T = T_;
  static constexpr int D = D_, THREADS = THREADS_, WINDOW = WINDOW_;
  static constexpr int E = kElems<T>, LPH = D / 2 / E, ROWS = THREADS / LPH;
  static constexpr int PASSES = WINDOW / ROWS, KEPT = VALUES / (2 * E);
  static_assert(THREADS % (D / 2) == 0, "a thread keeps its pair of the rows' angles");
  static_assert(PASSES >= 1 && KEPT >= PASSES && WINDOW <= 64, "the window's own rows are kept");
};

// Four coefficients of a pair, gains folded in: y_a = r (a ca + b sb), y_b = r (b cb + a sa).
template <int D>
struct Turn {
  float ca[D / 2], sb[D / 2], cb[D / 2], sa[D / 2];
};
// What a thread knows of its pair j of every row (its frequency is a constant that differs from lane to lane, which
// takes a read per lane: once a block, not once a row).
struct Pair {
  uint64_t freq;
  float ga, gb;
};
template <int D>
__device__ __forceinline__ Pair pair_of(int j, const Store8Params& p, const __nv_bfloat16* gamma) {
  return {p.freq[j], gamma ? __bfloat162float(gamma[j]) : 1.f, gamma ? __bfloat162float(gamma[j + D / 2]) : 1.f};
}
// KEYS: with the hardware's sine and cosine, which are off by under 2^-20: keys are rounded to e4m3 (2^-4).
template <int D, bool KEYS>
__device__ __forceinline__ void make_turn(Turn<D>& t, int j, const Pair& q, int pos) {
  const uint64_t turn = (uint64_t)(uint32_t)pos * q.freq;
  const float half_turns = (float)(int32_t)(turn >> 32) * 0x1p-31f;  // in [-1, 1)
  float s, c;
  if constexpr (KEYS) {
    s = __sinf(half_turns * 3.14159265f);
    c = __cosf(half_turns * 3.14159265f);
  } else {
    sincospif(half_turns, &s, &c);
  }
  t.ca[j] = c * q.ga;
  t.sb[j] = -s * q.gb;
  t.cb[j] = c * q.gb;
  t.sa[j] = s * q.ga;
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

// The rows of a run go to one page, each at a higher offset than the one before.
template <typename S>
__device__ __forceinline__ void store_runs(const Store8Params& p, Turn<S::D>* turns, unsigned block) {
  using T = typename S::T;
  constexpr int D = S::D, E = S::E, LPH = S::LPH, THREADS = S::THREADS, ROWS = S::ROWS, WINDOW = S::WINDOW;
  constexpr int BACK = kGap + 1, SPAN = BACK + WINDOW + THREADS;  // rows around the window that are looked at at once
  __shared__ int near_slot[SPAN], near_pos[SPAN];
  __shared__ unsigned leads[2], breaks[2];   // rows of the window that begin a run, and others that end one
  __shared__ int stop, beyond, grown;
  __shared__ unsigned top[WINDOW];           // maxima of the runs, by first row
  __shared__ unsigned written[WINDOW][8];    // offsets that a run writes, where what a page holds is looked at again
  __shared__ int upto[WINDOW];               // the last one
  __shared__ float inv_of[WINDOW], again[WINDOW];  // 1 / scale; what held codes are multiplied with (1: they stay)
  const int tid = threadIdx.x, gl = tid % LPH, group = tid / LPH;
  const int heads = 2 * p.Hkv, hh = block % heads;
  const int64_t r0 = (int64_t)(block / heads) * WINDOW;
  const bool is_v = hh >= p.Hkv;
  const int head = is_v ? hh - p.Hkv : hh, page = 1 << p.page_shift;
  const unsigned mask = (LPH == 32 ? 0xffffffffu : ((1u << LPH) - 1u)) << ((tid & 31) / LPH * LPH);
  // the window's rows are on their way while their runs are found (where a page may be larger than the window, many
  // windows have no run of their own)
  const T* base = static_cast<const T*>(p.x) + (int64_t)(p.Hq + hh) * D + gl * E;
  const bool early = page <= WINDOW;
  Raw<T, E> ra[S::KEPT], rb[S::KEPT];
  const auto load = [&](int w) {
    const int64_t row = r0 + w * ROWS + group;
    ra[w].load(base + row * p.ld_x);
    rb[w].load(base + row * p.ld_x + D / 2);
  };
  // a row's slot, and its position; -1 for one that is not stored
  const auto slot_at = [&](int64_t r, int& pos) {
    if (r < 0 || r >= p.N) return pos = -1;
    const int slot = p.slots[r];
    pos = p.positions[r];
    return pos >= 0 ? slot : -1;
  };
  for (int i = tid; i < SPAN; i += THREADS) near_slot[i] = slot_at(r0 - BACK + i, near_pos[i]);
  if (early) {
#pragma unroll
    for (int w = 0; w < S::PASSES; ++w)
      if (r0 + w * ROWS + group < p.N) load(w);
  }
  if (tid == 0) {
    stop = INT32_MAX;
    beyond = grown = 0;
    leads[1] = breaks[1] = 0;
  }
  for (int i = tid; i < WINDOW; i += THREADS) top[i] = 0;
  __syncthreads();
  const auto in_pool = [&](int slot) { return slot >= 0 && (slot >> p.page_shift) < p.num_pages; };
  const auto same_page = [&](int a, int b) { return b >= 0 && (a >> p.page_shift) == (b >> p.page_shift); };
  // the slot of the nearest stored row before row r0 + i
  const auto before_of = [&](int i) {
    int b = -1, pos;
#pragma unroll 1
    for (int k = 1; k <= BACK && b < 0; ++k)
      b = i - k < SPAN - BACK ? near_slot[BACK + i - k] : slot_at(r0 + i - k, pos);
    return b;
  };
  if (tid < WINDOW) {
    const unsigned who = WINDOW < 32 ? (1u << (WINDOW & 31)) - 1u : 0xffffffffu;
    const int slot = near_slot[BACK + tid], before = slot >= 0 ? before_of(tid) : -1;
    const bool in = in_pool(slot), again_page = in && same_page(slot, before);
    // a page that comes again in another order: two runs would both set its scale
    const bool twice = again_page && slot <= before;
    if (hh == 0 && ((slot >= 0 && !in) || twice)) set_status(p.status, MK_DEV_BAD_INDEX);
    const unsigned l = __ballot_sync(who, in && !again_page), t = __ballot_sync(who, twice || (slot >= 0 && !in));
    if (tid % 32 == 0) {
      leads[tid / 32] = l;
      breaks[tid / 32] = t;
    }
  }
  __syncthreads();
  const uint64_t lead_bits = leads[0] | (uint64_t)leads[1] << 32;
  if (lead_bits == 0) return;
  const uint64_t ends = lead_bits | breaks[0] | (uint64_t)breaks[1] << 32;
  // the run that a row of the window belongs to, by its first row (-1: another block's, or none)
  const auto run_of = [&](int row) {
    const uint64_t e = ends & ((2ull << row) - 1ull);
    const int at = e ? 63 - __clzll((long long)e) : -1;
    return at >= 0 && (lead_bits >> at & 1) ? at : -1;
  };
  const int last = run_of(WINDOW - 1);
  // the last run's rows behind the window
  for (int i0 = WINDOW; last >= 0; i0 += THREADS) {
    const int i = i0 + tid;
    int pos;
    const int slot = i0 == WINDOW ? near_slot[BACK + i] : slot_at(r0 + i, pos), before = slot >= 0 ? before_of(i) : -1;
    const bool on = in_pool(slot) && same_page(slot, before) && slot > before;
    if (slot >= 0 && !on) atomicMin(&stop, i);
    if (!__syncthreads_or(on)) break;  // (a run goes on within BACK rows)
    const int end = stop;
    if (on && i < end) atomicMax(&beyond, i + 1 - WINDOW);
    if (end != INT32_MAX) break;
    __syncthreads();
  }
  __syncthreads();
  const Pair pair = is_v ? Pair{} : pair_of<D>(tid % (D / 2), p, p.k_gamma);
  const int more = beyond, passes = S::PASSES + (more + ROWS - 1) / ROWS;

  // this group's row of a pass: its run, and its slot (-1: none of this block's)
  const auto run_in = [&](int w) { return w < S::PASSES ? run_of(w * ROWS + group) : last; };
  const auto slot_in = [&](int w) {
    const int i = w * ROWS + group;
    int pos;
    if (w < S::PASSES) return run_of(i) >= 0 ? near_slot[BACK + i] : -1;
    return i - WINDOW >= more ? -1 : i < SPAN - BACK ? near_slot[BACK + i] : slot_at(r0 + i, pos);
  };
  const auto turn_rows = [&](int w) {
    if (is_v) return;
    __syncthreads();
    for (int i = tid / (D / 2); i < ROWS; i += THREADS / (D / 2)) {
      const int k = w * ROWS + i;
      int pos;
      if (k < SPAN - BACK) pos = near_pos[BACK + k];
      else slot_at(r0 + k, pos);
      make_turn<D, true>(turns[i], tid % (D / 2), pair, pos);
    }
    __syncthreads();
  };
  // a pass's values, as floats to be stored (zero where there is no row)
  const auto values = [&](int w, int slot, const Raw<T, E>& ra, const Raw<T, E>& rb, float (&a)[E], float (&b)[E]) {
    turn_rows(w);
#pragma unroll
    for (int i = 0; i < E; ++i) a[i] = b[i] = 0.f;
    if (slot >= 0) {
      ra.get(a);
      rb.get(b);
      if (!is_v) norm_turn<E, D>(a, b, turns[group], gl, p.k_gamma != nullptr, p.eps, mask);
#pragma unroll
      for (int i = 0; i < E; i += 2) {  // an infinity becomes NaN
        const uint64_t u = ptx::pair_f32(a[i], a[i + 1]), v = ptx::pair_f32(b[i], b[i + 1]);
        const float2 x = ptx::unpair_f32(ptx::fma2(u, 0, u)), y = ptx::unpair_f32(ptx::fma2(v, 0, v));
        a[i] = x.x;
        a[i + 1] = x.y;
        b[i] = y.x;
        b[i + 1] = y.y;
      }
    }
  };
  // the same of a pass that is not kept
  const auto read = [&](int w, int slot, float (&a)[E], float (&b)[E]) {
    Raw<T, E> xa, xb;
    if (slot >= 0) {
      xa.load(base + (r0 + w * ROWS + group) * p.ld_x);
      xb.load(base + (r0 + w * ROWS + group) * p.ld_x + D / 2);
    }
    values(w, slot, xa, xb, a, b);
  };
  const auto raise = [&](int run, const float (&a)[E], const float (&b)[E]) {
    float m = 0.f;  // (a maximum leaves NaN out)
#pragma unroll
    for (int i = 0; i < E; ++i) m = fmaxf(m, fmaxf(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
    if (gl == 0 && m > 0.f) atomicMax(&top[run], __float_as_uint(m));
  };
  int slot_k[S::KEPT], run_k[S::KEPT];
#pragma unroll
  for (int w = 0; w < S::KEPT; ++w) {
    slot_k[w] = w < passes ? slot_in(w) : -1;
    run_k[w] = max(run_in(w), 0);
    if ((w >= S::PASSES || !early) && slot_k[w] >= 0) load(w);
  }
  float ka[S::KEPT][E], kb[S::KEPT][E];
#pragma unroll
  for (int w = 0; w < S::KEPT; ++w) {
    if (w >= passes) break;
    values(w, slot_k[w], ra[w], rb[w], ka[w], kb[w]);
    raise(run_k[w], ka[w], kb[w]);
  }
  for (int w = S::KEPT; w < passes; ++w) {
    float a[E], b[E];
    read(w, slot_in(w), a, b);
    raise(last, a, b);
  }
  __syncthreads();
  float* scales = is_v ? p.vscale : p.kscale;
  uint8_t* codes = is_v ? p.vcodes : p.kcodes;
  if (tid < WINDOW && (lead_bits >> tid & 1)) {
    const int slot = near_slot[BACK + tid];
    float* at = scales + (int64_t)(slot >> p.page_shift) * p.Hkv + head;
    float s = scale_for(__uint_as_float(top[tid])), by = 1.f;
    if ((slot & (page - 1)) != 0) {  // a page that is begun
      const float old = *at;
      if (old >= s) s = old;
      else by = old / s;
      if (by != 1.f) grown = 1;
    }
    *at = s;
    inv_of[tid] = 1.f / s;
    again[tid] = by;
  }
  __syncthreads();
  if (grown) {
    // pages whose scale grew: what they hold below the last new row, but for what is new
    for (int i = tid; i < WINDOW; i += THREADS) upto[i] = 0;
    for (int i = tid; i < WINDOW * 8; i += THREADS) written[i / 8][i % 8] = 0;
    __syncthreads();
    for (int w = 0; w < passes; ++w) {
      const int slot = slot_in(w), off = slot & (page - 1);
      if (gl != 0 || slot < 0) continue;
      atomicOr(&written[run_in(w)][off / 32], 1u << (off % 32));
      atomicMax(&upto[run_in(w)], off);
    }
    __syncthreads();
    for (uint64_t rest = lead_bits; rest; rest &= rest - 1) {
      const int i = __ffsll((long long)rest) - 1;
      const float by = again[i];
      if (by == 1.f) continue;
      uint4* at = reinterpret_cast<uint4*>(
          codes + (((int64_t)(near_slot[BACK + i] >> p.page_shift) * p.Hkv + head) << p.page_shift) * D);
      for (int j = tid; j < upto[i] * (D / 16); j += THREADS) {
        const int off = j / (D / 16);
        if (written[i][off / 32] >> (off % 32) & 1) continue;
        uint4 v = at[j];
        v.x = rescale4(v.x, by); v.y = rescale4(v.y, by); v.z = rescale4(v.z, by); v.w = rescale4(v.w, by);
        at[j] = v;
      }
    }
  }
  const auto put = [&](int slot, int run, const float (&a)[E], const float (&b)[E]) {
    if (slot < 0) return;
    uint8_t* dst = codes + ((((int64_t)(slot >> p.page_shift) * p.Hkv + head) << p.page_shift) + (slot & (page - 1))) * D +
                   gl * E;
    const float inv = inv_of[run];
    store_codes<E>(dst, a, inv);
    store_codes<E>(dst + D / 2, b, inv);
  };
#pragma unroll
  for (int w = 0; w < S::KEPT; ++w) put(slot_k[w], run_k[w], ka[w], kb[w]);
  for (int w = S::KEPT; w < passes; ++w) {
    float a[E], b[E];
    const int slot = slot_in(w);
    read(w, slot, a, b);
    put(slot, last, a, b);
  }
}

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
      const int j = threadIdx.x % (D / 2);
      const Pair pair = pair_of<D>(j, p, p.q_gamma);
      for (int i = threadIdx.x / (D / 2); i < p.tokens; i += THREADS / (D / 2)) {
        const int64_t r = row0 + i;
        make_turn<D, false>(turns[i], j, pair, r < p.N ? p.positions[r] : 0);
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

// Keys and values first, then the queries, in one launch
template <typename S>
__global__ void __launch_bounds__(S::THREADS) store8_kernel(const __grid_constant__ Store8Params p) {
  __shared__ __align__(16) Turn<S::D> turns[S::ROWS];
  if (blockIdx.x < p.kv_blocks) store_runs<S>(p, turns, blockIdx.x);
  else queries<S>(p, turns, blockIdx.x - p.kv_blocks);
}
// Keys and values alone
template <typename S>
__global__ void __launch_bounds__(S::THREADS, 2) store8_kv_kernel(const __grid_constant__ Store8Params p) {
  ptx::launch_dependents();  // the queries' blocks follow as these end
  __shared__ __align__(16) Turn<S::D> turns[S::ROWS];
  store_runs<S>(p, turns, blockIdx.x);
}

#ifndef FEW_ROWS
#define FEW_ROWS 512
#endif
template <typename T, int D>
cudaError_t launch_store8(Store8Params& p, int sms, cudaStream_t stream) {
  constexpr int E = kElems<T>, LPH = D / 2 / E;
  if (p.N > FEW_ROWS) {
    using S = Shape<T, D, 256, 64, 64>;
    const int64_t kv = (((int64_t)p.N + S::WINDOW - 1) / S::WINDOW) * 2 * p.Hkv;
    store8_kv_kernel<S><<<(unsigned)kv, S::THREADS, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_queries(p, sizeof(T) == 4 ? MK_F32 : MK_BF16, D, sms, stream);
  }
  using S = Shape<T, D, 16 * LPH, 16, 10 * E>;
  constexpr int GP = S::ROWS;
  // tokens whose heads fill a block's batch; few tokens: a head per lane group, over several blocks
  p.tokens = 1;
  while (p.tokens < kQueryMaxTokens && 2 * p.tokens * p.Hq <= kQueryBatch * GP) p.tokens *= 2;
  while (p.tokens > 1 && (p.N + p.tokens - 1) / p.tokens < 2 * sms) p.tokens /= 2;
  p.splits = p.N < sms ? (p.Hq + GP - 1) / GP : 1;
  p.kv_blocks = (unsigned)((p.N + S::WINDOW - 1) / S::WINDOW * 2 * p.Hkv);
  const unsigned blocks = p.kv_blocks + (unsigned)((p.N + p.tokens - 1) / p.tokens * p.splits);
  store8_kernel<S><<<blocks, S::THREADS, 0, stream>>>(p);
  return cudaGetLastError();
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
  if (((int64_t)N + 63) / 64 * 2 * Hkv > INT32_MAX || (int64_t)N * ((Hq + 2 * Hkv) / 8 + 1) > INT32_MAX)
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
