// Log probabilities of given tokens, the entropy of their distributions, and
// the likeliest alternatives, from rows of logits.
//
//   m = max x,  s = sum 2^((x - m) log2 e),  u = sum 2^((x - m) log2 e) (x - m)
//   log p_t = (x_t - m) - ln s        H = ln s - u / s
//
// in one pass with running (m, s, u) per thread, so HBM bounds it.  A row
// belongs to a cluster of one to eight CTAs (few rows would leave SMs without
// work), each with an even part of it; the parts' sums and alternatives meet
// in the first CTA's shared memory.
//
// The alternatives are the largest of unique 64-bit keys (the logit's order,
// then the lower index), so their order never depends on the order of work.
// The pass over the row does nothing for them: it leaves each thread's maximum,
// the top-th largest of 64 thread groups' maxima is a lower bound of the top-th
// largest logit, and only the logits of threads whose maximum reaches it are
// looked at again (about `top` of 256 threads; out of the L2), by the whole CTA.
// Should more reach the bound than there is room for (equal logits), each warp
// goes through its part with a buffer that is cut down to its `top` largest when
// it is full.  A key's rank is the number of larger keys, counted by four threads.
//
// 2048 rows of 128256: f32 158 us (6.6 TB/s, a copy's rate), bf16 94 (5.6 TB/s:
// twice the arithmetic per byte) and 101 with one
// alternative, 120 with 20.  61 rows of f32 with 20 alternatives 12.5 us, of
// which 4.2 are those; one row 4.4 us, 8.1 with 20: start, one trip to memory
// and the cluster's meeting, then the chain bound, hits, logits, ranks.
#include <cuda_bf16.h>

#include "paged.h"
#include "ptx_ops.cuh"

namespace mk {
namespace {

using namespace ptx;

constexpr int kCap = 128;                     // candidates of a warp, where there are too many
constexpr int kMaxTop = 32, kMaxCluster = 8;
constexpr int kGroups = 64;                   // groups of threads whose maxima give a bound
constexpr int kFirst = 64;                    // logits that a part is filled up from with -inf
// A CTA of THREADS, whose threads take STEP bytes of logits at a time (with the next step's on their way).
template <typename T_, int THREADS_, int STEP_, int CTAS_>
struct Shape {
  using T = T_;
  static constexpr int THREADS = THREADS_, WARPS = THREADS / 32, STEP = STEP_, CTAS = CTAS_;
  static constexpr int VEC = 16 / sizeof(T), U = STEP / 16;
  static constexpr int MATES = THREADS / kGroups;  // threads of a group; threads that count a key's rank
  static constexpr int FEW = WARPS * kCap;         // candidates
  static_assert(FEW >= (kMaxTop - 1) * MATES * 8 + 16 && FEW >= kMaxTop + kFirst, "parts of fewer groups than `top` fit");
};

struct LogprobParams {
  const void* x;
  int64_t ld;
  const int32_t* tokens;
  float *logprobs, *entropy, *top_logprobs;
  int32_t *top_ids, *status;
  int V, top, cluster;
};

// (m, s, u) of a part of a row: its maximum, sum of 2^((x - m) log2 e), and that sum weighted with x - m
struct Sums {
  float m, s, u;
};
__device__ __forceinline__ Sums merge(Sums a, Sums b) {
  const float m = fmaxf(a.m, b.m), at = m == -INFINITY ? 0.f : m;
  constexpr float kLog2e = 1.4426950408889634f;
  const float da = a.m - at, db = b.m - at, fa = ex2(da * kLog2e), fb = ex2(db * kLog2e);
  // (a part without weight adds nothing, although its maximum may be -inf, and s (x - m) past the largest f32 where it
  // is finite, as masks of the type's lowest value make it: zero times infinity would be NaN)
  const float ua = a.s == 0.f || fa == 0.f ? 0.f : fa * fmaf(a.s, da, a.u);
  const float ub = b.s == 0.f || fb == 0.f ? 0.f : fb * fmaf(b.s, db, b.u);
  return {m, a.s * fa + b.s * fb, ua + ub};
}

// A logit's place in the order: larger ones first, of equal ones the lower index; 0: not in it (NaN).
__device__ __forceinline__ uint64_t key_of(float x, int index) {
  const uint32_t b = __float_as_uint(x + 0.f);  // (-0 is 0)
  const uint32_t order = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return x != x ? 0 : (uint64_t)order << 32 | (uint32_t)~index;
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t order = (uint32_t)(key >> 32);
  return __uint_as_float(order & 0x80000000u ? order ^ 0x80000000u : ~order);
}

template <typename S>
struct Shared {
  uint64_t few[S::FEW], best[kMaxTop], group[kGroups];
  uint64_t all[kMaxCluster][kMaxTop];  // of the first CTA: every part's alternatives, and sums
  Sums sums[kMaxCluster], warp[S::WARPS];
  uint64_t bound;
  int few_count, hit_count, odd;
  uint8_t hits[S::THREADS];            // threads whose maximum reaches the bound
};

// The number of keys[0 .. n) larger than `key`, counted by MATES neighbouring lanes.
template <int MATES>
__device__ __forceinline__ int rank_of(const uint64_t* keys, int n, uint64_t key) {
  int r = 0;
#pragma unroll 4
  for (int i = threadIdx.x % MATES; i < n; i += MATES) r += keys[i] > key;
#pragma unroll
  for (int o = 1; o < MATES; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  return r;
}

// The top-th largest of 64 thread groups' largest keys: at least `top` keys are as large.  0: fewer groups have one.
// The whole CTA.
template <typename S>
__device__ __forceinline__ uint64_t group_bound(Shared<S>& sm, uint64_t own, int top) {
  constexpr int MATES = S::MATES;
#pragma unroll
  for (int o = 1; o < MATES; o <<= 1) {
    const uint64_t other = __shfl_xor_sync(0xffffffffu, own, o);
    own = other > own ? other : own;
  }
  if (threadIdx.x % MATES == 0) sm.group[threadIdx.x / MATES] = own;
  if (threadIdx.x == 0) sm.bound = 0;
  __syncthreads();
  const int r = rank_of<MATES>(sm.group, kGroups, own);
  if (own != 0 && r == top - 1 && threadIdx.x % MATES == 0) sm.bound = own;
  __syncthreads();
  return sm.bound;
}

// best[0 .. top) = the largest of keys[0 .. n), in order, 0 where there are fewer.  The whole CTA; keys are there.
template <typename S>
__device__ __forceinline__ void rank_all(Shared<S>& sm, const uint64_t* keys, int n, int top) {
  constexpr int MATES = S::MATES;
  if (threadIdx.x < kMaxTop) sm.best[threadIdx.x] = 0;
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += kGroups) {
    const int i = i0 + threadIdx.x / MATES;
    const uint64_t key = i < n ? keys[i] : 0;
    const int r = rank_of<MATES>(keys, n, key);
    if (key != 0 && r < top && threadIdx.x % MATES == 0) sm.best[r] = key;
  }
  __syncthreads();
}

// A warp's buffer of n keys cut down to its `top` largest, in order; the last of them.
__device__ __noinline__ uint64_t cut_down(uint64_t* buf, int n, int top) {
  const int lane = threadIdx.x % 32;
  __syncwarp();
  uint64_t k[kCap / 32], last = 0;
#pragma unroll
  for (int i = 0; i < kCap / 32; ++i) k[i] = i * 32 + lane < n ? buf[i * 32 + lane] : 0;
  __syncwarp();
  for (int t = 0; t < top; ++t) {
    uint64_t most = 0;
#pragma unroll
    for (int i = 0; i < kCap / 32; ++i) most = k[i] > most ? k[i] : most;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, most, o);
      most = other > most ? other : most;
    }
#pragma unroll
    for (int i = 0; i < kCap / 32; ++i)
      if (k[i] == most) k[i] = 0;
    if (lane == 0) buf[t] = most;
    last = most;
  }
  __syncwarp();
  return last;
}

__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// 16 bytes of logits
__device__ __forceinline__ void widen(const uint4& v, float* f, float) {
  f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void widen(const uint4& v, float* f, __nv_bfloat16) {
  f[0] = bf_lo(v.x); f[1] = bf_hi(v.x); f[2] = bf_lo(v.y); f[3] = bf_hi(v.y);
  f[4] = bf_lo(v.z); f[5] = bf_hi(v.z); f[6] = bf_lo(v.w); f[7] = bf_hi(v.w);
}
// the largest of a step's logits, NaN left out
template <int U>
__device__ __forceinline__ float most_of(const uint4 (&v)[U], float) {
  float m[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    m[u] = fmaxf(fmaxf(__uint_as_float(v[u].x), __uint_as_float(v[u].y)),
                 fmaxf(__uint_as_float(v[u].z), __uint_as_float(v[u].w)));
#pragma unroll
  for (int u = 1; u < U; ++u) m[0] = fmaxf(m[0], m[u]);
  return m[0];
}
template <int U>
__device__ __forceinline__ float most_of(const uint4 (&v)[U], __nv_bfloat16) {
  const auto two = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
  __nv_bfloat162 m[U];
#pragma unroll
  for (int u = 0; u < U; ++u) m[u] = __hmax2(__hmax2(two(v[u].x), two(v[u].y)), __hmax2(two(v[u].z), two(v[u].w)));
#pragma unroll
  for (int u = 1; u < U; ++u) m[0] = __hmax2(m[0], m[u]);
  return fmaxf(__low2float(m[0]), __high2float(m[0]));
}
__device__ __forceinline__ float widen1(float x) { return x; }
__device__ __forceinline__ float widen1(__nv_bfloat16 x) { return __bfloat162float(x); }

// A CTA's part of a row: logits before the first 16-byte boundary (of the row's first part), vectors, logits behind
// the last (of its last part).
template <typename T>
struct Part {
  const T* x;          // the row
  int head, v0, v1;    // index of vector 0's first logit; the part's vectors
  int lead, trail;     // logits before, and behind the vectors
  int behind;          // index of the first of those behind
  __device__ __forceinline__ const uint4* vectors() const { return reinterpret_cast<const uint4*>(x + head); }
  // the i-th logit that is in no vector, by index; -1: there are fewer
  __device__ __forceinline__ int end(int i) const { return i < lead ? i : i - lead < trail ? behind + i - lead : -1; }
};

// Candidates of a part where too many logits reach a bound: every warp's `top` largest, in few[].  The whole CTA.
template <typename S>
__device__ __noinline__ int sift(Shared<S>& sm, const Part<typename S::T>& p, int top, float bound) {
  using T = typename S::T;
  constexpr int VEC = S::VEC, kWarps = S::WARPS, kThreads = S::THREADS;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint64_t* buf = sm.few + warp * kCap;
  int count = 0, before = INT32_MAX;  // a logit equal to the bound has to lie before this index
  __syncthreads();
  const auto offer = [&](float v, int index, bool there) {
    bool yes = there && (v > bound || (v == bound && index < before));
    unsigned who = __ballot_sync(0xffffffffu, yes);
    if (who == 0) return;
    if (count > kCap - 32) {
      const uint64_t last = cut_down(buf, count, top);
      count = top;
      bound = logit_of(last);
      before = (int32_t)~(uint32_t)last;
      yes = there && (v > bound || (v == bound && index < before));
      who = __ballot_sync(0xffffffffu, yes);
    }
    if (yes) buf[count + __popc(who & ((1u << lane) - 1))] = key_of(v, index);
    count += __popc(who);
  };
  for (int v = p.v0 + warp * 32; v < p.v1; v += kThreads) {
    const bool there = v + lane < p.v1;
    float f[VEC];
    widen(there ? __ldg(p.vectors() + v + lane) : make_uint4(0, 0, 0, 0), f, T());
#pragma unroll
    for (int e = 0; e < VEC; ++e) offer(f[e], p.head + (v + lane) * VEC + e, there);
  }
  if (warp == 0) {
    const int i = p.end(lane);
    offer(i >= 0 ? widen1(p.x[i]) : 0.f, i, i >= 0);
  }
  if (count > top) {
    cut_down(buf, count, top);
    count = top;
  }
  if (lane >= count && lane < top) buf[lane] = 0;
  __syncthreads();
  // the warps' lists side by side
  const uint64_t key = threadIdx.x < kWarps * top ? sm.few[threadIdx.x / top * kCap + threadIdx.x % top] : 0;
  __syncthreads();
  if (threadIdx.x < kWarps * top) sm.few[threadIdx.x] = key;
  __syncthreads();
  return kWarps * top;
}

// best[0 .. top): a part's largest logits.  `most`: the largest of this thread's (vectors v0 + tid + i * kThreads, and
// the end tid), `odd` whether there is a NaN among them.  The whole CTA.
template <typename S>
__device__ __forceinline__ void alternatives(Shared<S>& sm, const Part<typename S::T>& p, int top, float most, bool odd) {
  using T = typename S::T;
  constexpr int VEC = S::VEC, kThreads = S::THREADS;
  const int tid = threadIdx.x, per = (p.v1 - p.v0 + kThreads - 1) / kThreads;  // vectors of a thread
  const bool some = p.v0 + tid < p.v1 || p.end(tid) >= 0;
  const uint64_t least = group_bound(sm, some ? key_of(most, tid) : 0, top);
  // without a bound, every logit but NaN is a candidate
  const float bound = least ? logit_of(least) : -INFINITY;
  if (tid == 0) sm.few_count = sm.hit_count = sm.odd = 0;
  __syncthreads();
  const bool finite = least != 0 && bound == -INFINITY;  // (only those over -inf)
  if (some && (finite ? most > bound : most >= bound)) sm.hits[atomicAdd(&sm.hit_count, 1)] = (uint8_t)tid;
  if (odd) sm.odd = 1;
  __syncthreads();
  const auto offer = [&](float v, int index) {
    if (!(finite ? v > bound : v >= bound)) return;
    const int at = atomicAdd(&sm.few_count, 1);
    if (at < S::FEW) sm.few[at] = key_of(v, index);
  };
  const int items = sm.hit_count * per;
  constexpr int B = 4;  // loads in flight
  for (int i0 = tid; i0 < items; i0 += B * kThreads) {
    uint4 raw[B];
    int v[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int i = i0 + k * kThreads;
      v[k] = i < items ? p.v0 + sm.hits[i / per] + i % per * kThreads : p.v1;
      if (v[k] < p.v1) raw[k] = __ldg(p.vectors() + v[k]);
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      if (v[k] >= p.v1) continue;
      float f[VEC];
      widen(raw[k], f, T());
#pragma unroll
      for (int e = 0; e < VEC; ++e) offer(f[e], p.head + v[k] * VEC + e);
    }
  }
  const int e = p.end(tid);
  if (e >= 0) offer(widen1(p.x[e]), e);
  __syncthreads();
  int n = sm.few_count;
  if (n < top && finite && !sm.odd) {
    // fewer logits than alternatives have a probability: the first ones without follow (of kFirst neighbours fewer
    // than `top` have one)
    const int first = p.lead > 0 ? 0 : p.head + p.v0 * VEC;
    const int end = p.trail > 0 ? p.behind + p.trail : p.head + p.v1 * VEC;
    __syncthreads();
    if (tid < kFirst && first + tid < end && widen1(p.x[first + tid]) == -INFINITY)
      sm.few[atomicAdd(&sm.few_count, 1)] = key_of(-INFINITY, first + tid);
    __syncthreads();
    n = sm.few_count;
  } else if (n > S::FEW || (n < top && sm.odd)) {
    n = sift(sm, p, top, bound);
  }
  rank_all(sm, sm.few, n, top);
}

template <typename S>
__global__ void __launch_bounds__(S::THREADS, S::CTAS) logprob_kernel(const __grid_constant__ LogprobParams p) {
  using T = typename S::T;
  constexpr int VEC = S::VEC, U = S::U, kThreads = S::THREADS, kWarps = S::WARPS;
  constexpr float kLog2e = 1.4426950408889634f;
  __shared__ Shared<S> sm;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, C = p.cluster, rank = blockIdx.x % C;
  const int64_t row = blockIdx.x / C;
  int token = -1;
  if (p.tokens) {
    token = p.tokens[row];
    if (token < 0) return;  // left out (the whole cluster)
  }
  if (C > 1) cluster_arrive();
  Part<T> part;
  {
    const T* x = static_cast<const T*>(p.x) + row * p.ld;
    const int head = min(p.V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T));
    const int nv = (p.V - head) / VEC, per = (nv + C - 1) / C;
    part.x = x;
    part.head = head;
    part.v0 = min(nv, rank * per);
    part.v1 = min(nv, part.v0 + per);
    part.lead = rank == 0 ? head : 0;
    part.behind = head + nv * VEC;
    part.trail = rank == C - 1 ? p.V - part.behind : 0;
  }
  const int steps = (part.v1 - part.v0 + kThreads * U - 1) / (kThreads * U);
  uint4 next[U];
  const uint32_t fill = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;  // -inf
  auto load = [&](int c) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = part.v0 + (c * U + u) * kThreads + tid;
      next[u] = v < part.v1 ? __ldg(part.vectors() + v) : make_uint4(fill, fill, fill, fill);
    }
  };
  if (steps > 0) load(0);
  Sums own = {-INFINITY, 0.f, 0.f};
  if (part.end(tid) >= 0) {  // (at most 14 threads)
    own.m = widen1(part.x[part.end(tid)]);
    own.s = ex2((own.m == -INFINITY ? own.m : own.m - own.m) * kLog2e);  // 1, 0 or NaN
    if (own.m != own.m) own.m = -INFINITY;
  }
  for (int c = 0; c < steps; ++c) {
    uint4 now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = next[u];
    if (c + 1 < steps) load(c + 1);
    const float most = most_of(now, T());
    if (most > own.m) own = merge(own, {most, 0.f, 0.f});
    const float at = own.m == -INFINITY ? 0.f : own.m;
    const uint64_t at2 = pair_f32(-at, -at), log2 = pair_f32(kLog2e, kLog2e);
    uint64_t s2[2] = {0, 0}, u2[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[VEC];
      widen(now[u], f, T());
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        const uint64_t d = add2(pair_f32(f[e], f[e + 1]), at2);
        const float2 t = unpair_f32(mul2(d, log2)), dd = unpair_f32(d);
        const uint64_t w = pair_f32(ex2(t.x), ex2(t.y));
        s2[(e >> 1) & 1] = add2(s2[(e >> 1) & 1], w);
        // (a weight of zero times -inf would be NaN)
        u2[(e >> 1) & 1] = fma2(w, pair_f32(fmaxf(dd.x, -1e30f), fmaxf(dd.y, -1e30f)), u2[(e >> 1) & 1]);
      }
    }
    const float2 s = unpair_f32(add2(s2[0], s2[1])), u = unpair_f32(add2(u2[0], u2[1]));
    own.s += s.x + s.y;
    own.u += u.x + u.y;
  }
  const float most = own.m;
  const bool odd = own.s != own.s;

  // the part's sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    own = merge(own, {__shfl_xor_sync(0xffffffffu, own.m, o), __shfl_xor_sync(0xffffffffu, own.s, o),
                      __shfl_xor_sync(0xffffffffu, own.u, o)});
  if (lane == 0) sm.warp[warp] = own;
  if (p.top > 0) alternatives(sm, part, p.top, most, odd);
  else __syncthreads();
  own = sm.warp[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) own = merge(own, sm.warp[w]);
  if (C > 1) {
    __syncwarp();
    cluster_wait();  // the first CTA is there
    if (tid == 0) {
      const uint32_t a = cluster_addr(&sm.sums[rank], 0);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(own.m) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 4), "f"(own.s) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 8), "f"(own.u) : "memory");
    }
    if (tid < p.top)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr(&sm.all[0][rank * p.top + tid], 0)),
                   "l"(sm.best[tid])
                   : "memory");
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    own = sm.sums[0];
    for (int r = 1; r < C; ++r) own = merge(own, sm.sums[r]);
    if (p.top > 0) {
      const int n = C * p.top;
      if (n <= kGroups) {
        rank_all(sm, sm.all[0], n, p.top);
      } else {
        uint64_t key = 0;
        for (int i = tid; i < n; i += kThreads) key = sm.all[0][i] > key ? sm.all[0][i] : key;
        const uint64_t bound = group_bound(sm, key, p.top);
        if (tid == 0) sm.few_count = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads)
          if (sm.all[0][i] != 0 && sm.all[0][i] >= bound) sm.few[atomicAdd(&sm.few_count, 1)] = sm.all[0][i];
        __syncthreads();
        rank_all(sm, sm.few, sm.few_count, p.top);
      }
    }
  }
  const float ln_s = logf(own.s);
  if (tid == 0) {
    p.entropy[row] = ln_s - own.u / own.s;
    if (p.tokens) {
      float lp = __uint_as_float(0x7FC00000u);
      if (token < p.V) lp = (widen1(part.x[token]) - own.m) - ln_s;
      else set_status(p.status, MK_DEV_BAD_INDEX);
      p.logprobs[row] = lp;
    }
  }
  if (tid < p.top) {
    const uint64_t key = sm.best[tid];
    p.top_ids[row * p.top + tid] = key ? (int32_t)~(uint32_t)key : -1;
    p.top_logprobs[row * p.top + tid] = key ? (logit_of(key) - own.m) - ln_s : __uint_as_float(0x7FC00000u);
  }
}

template <typename S>
cudaError_t launch_shape(LogprobParams& p, int N, int sms, cudaStream_t stream) {
  // parts of a row while they all run at once, none under two vectors a thread
  p.cluster = 1;
  while (p.cluster < kMaxCluster && (int64_t)N * p.cluster * 2 <= S::CTAS * sms &&
         p.V / (2 * p.cluster) >= S::THREADS * S::VEC * 2)
    p.cluster *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(N * p.cluster));
  cfg.blockDim = dim3(S::THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)p.cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprob_kernel<S>, p);
}

// Many short rows: smaller CTAs, whose start, alternatives and end overlap better with others' passes (2048 rows of
// bf16, top 5: V 1000 21.4 us with 256 threads, 12.5 with 128; 8192 23.1 and 16.2; 32768 38.1 and 33.9; 50257 53.4 and
// 49.8; 80000 69.7 and 69.8; f32 at 50257 83.3 and 82.8, at 80000 117 and 125; 64 threads lose from 8192 on).  At f32
// 128 bytes a thread and step in three CTAs per SM stream best (2048 rows of 128256: 158 us, 6.6 TB/s, a copy's rate;
// 64 bytes in four 168), at bf16, where a step is more arithmetic, 64 in four (512 rows 31 us, 35 the other way; 2048
// rows 101 and 98).
constexpr int kShortRow = 65536;
template <typename T>
cudaError_t launch_logprobs(LogprobParams& p, int N, int sms, cudaStream_t stream) {
  constexpr bool f32 = sizeof(T) == 4;
  if (p.V <= kShortRow && N > sms) return launch_shape<Shape<T, 128, 64, 8>>(p, N, sms, stream);
  return launch_shape<Shape<T, 256, f32 ? 128 : 64, f32 ? 3 : 4>>(p, N, sms, stream);
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_token_logprobs(void* stream, int N, int V, const void* logits, int logits_dtype, int64_t ld,
                                 const int32_t* tokens, int top, float* logprobs, float* entropy, int32_t* top_ids,
                                 float* top_logprobs, int32_t* status) try {
  if (!logits || !entropy || (tokens && !logprobs) || (top > 0 && (!top_ids || !top_logprobs)))
    return fail(MK_ERR_ARG, "mk_token_logprobs: null argument");
  if (N < 0 || V < 1 || V > INT32_MAX / 2) return fail(MK_ERR_ARG, "mk_token_logprobs: need N >= 0 and 1 <= V < 2^30");
  if (N > INT32_MAX / kMaxCluster) return fail(MK_ERR_LIMIT, "mk_token_logprobs: need N < 2^28");
  if (top < 0 || top > kMaxTop || top > V) return fail(MK_ERR_ARG, "mk_token_logprobs: need 0 <= top <= min(32, V)");
  if (logits_dtype != MK_F32 && logits_dtype != MK_BF16)
    return fail(MK_ERR_ARG, "mk_token_logprobs: logits must be f32 or bf16");
  if (ld < 0 || (N > 1 && ld < V)) return fail(MK_ERR_ARG, "mk_token_logprobs: rows may not overlap");
  if (reinterpret_cast<uintptr_t>(logits) % (logits_dtype == MK_F32 ? 4 : 2))
    return fail(MK_ERR_ARG, "mk_token_logprobs: logits must be aligned to their type");
  if (int rc = pending_error("mk_token_logprobs")) return rc;
  if (N == 0) return MK_OK;
  int sms = 0;
  if (int rc = device_sms("mk_token_logprobs", &sms)) return rc;
  LogprobParams p{logits, ld, tokens, logprobs, entropy, top_logprobs, top_ids, status, V, top, 1};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_result(logits_dtype == MK_F32 ? launch_logprobs<float>(p, N, sms, s)
                                              : launch_logprobs<__nv_bfloat16>(p, N, sms, s),
                       "mk_token_logprobs");
} catch (...) {
  return MK_ERR_NOMEM;
}
