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
// Each CTA keeps a buffer of candidates: after its first 8192 logits the
// top-th largest of 64 thread groups' maxima is a lower bound of the top-th
// largest logit, what exceeds the bound goes to the buffer (about `top` per
// 8192 logits), and a buffer that fills up is cut down to its `top` largest,
// which raises the bound.  A key's rank is the number of larger keys, counted
// by a thread per key.
#include <cuda_bf16.h>

#include "paged.h"
#include "ptx_ops.cuh"

namespace mk {
namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kPer = 32;                      // logits of a thread and step
constexpr int kCap = 2048, kHigh = 512;       // candidates: room, and the count from which they are cut down
constexpr int kMaxTop = 32, kMaxCluster = 8;
constexpr int kGroups = 64;                   // groups whose maxima give the first bound

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
  // (a part without weight may have a maximum of -inf)
  const float ua = a.s == 0.f ? 0.f : fa * fmaf(a.s, da, a.u), ub = b.s == 0.f ? 0.f : fb * fmaf(b.s, db, b.u);
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

struct Shared {
  uint64_t buf[kCap], few[kCap / kGroups * kMaxTop], best[kMaxTop], group[kGroups];
  uint64_t all[kMaxCluster][kMaxTop];  // of the first CTA: every part's alternatives, and sums
  Sums sums[kMaxCluster], warp[kThreads / 32];
  uint64_t bound;
  int count, few_count;
};

// The number of keys[0 .. n) larger than `key`.
__device__ __forceinline__ int rank_of(const uint64_t* keys, int n, uint64_t key) {
  int r = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) r += keys[i] > key;
  return r;
}

// The top-th largest of 64 thread groups' largest keys: at least `top` keys are as large.  0: fewer groups have one.
__device__ __forceinline__ uint64_t group_bound(Shared& sm, uint64_t own, int top) {
  for (int o = 1; o < kThreads / kGroups; o <<= 1) {
    const uint64_t other = __shfl_xor_sync(0xffffffffu, own, o);
    own = other > own ? other : own;
  }
  if (threadIdx.x % (kThreads / kGroups) == 0) sm.group[threadIdx.x / (kThreads / kGroups)] = own;
  if (threadIdx.x == 0) sm.bound = 0;
  __syncthreads();
  if (threadIdx.x < kGroups) {
    const uint64_t key = sm.group[threadIdx.x];
    if (key != 0 && rank_of(sm.group, kGroups, key) == top - 1) sm.bound = key;
  }
  __syncthreads();
  return sm.bound;
}

// best[0 .. top) = the largest of buf[0 .. n), in order, 0 where there are fewer.  The whole CTA.
__device__ __noinline__ void select(Shared& sm, int n, int top) {
  const uint64_t* from = sm.buf;
  if (threadIdx.x < kMaxTop) sm.best[threadIdx.x] = 0;
  if (n > kThreads) {
    uint64_t own = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) own = max(own, sm.buf[i]);
    const uint64_t bound = group_bound(sm, own, top);
    if (threadIdx.x == 0) sm.few_count = 0;
    __syncthreads();
    // at most top groups reach the bound, with kCap / kGroups keys each
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t key = sm.buf[i];
      if (key >= bound) sm.few[atomicAdd(&sm.few_count, 1)] = key;
    }
    __syncthreads();
    from = sm.few;
    n = sm.few_count;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int r = rank_of(from, n, from[i]);
    if (r < top) sm.best[r] = from[i];
  }
  __syncthreads();
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
__device__ __forceinline__ float widen1(float x) { return x; }
__device__ __forceinline__ float widen1(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) logprob_kernel(const __grid_constant__ LogprobParams p) {
  constexpr int VEC = 16 / sizeof(T), U = kPer / VEC;
  constexpr float kLog2e = 1.4426950408889634f;
  __shared__ Shared sm;
  const int tid = threadIdx.x, C = p.cluster, rank = blockIdx.x % C;
  const int64_t row = blockIdx.x / C;
  int token = -1;
  if (p.tokens) {
    token = p.tokens[row];
    if (token < 0) return;  // left out (the whole cluster)
  }
  if (C > 1) cluster_arrive();
  const T* x = static_cast<const T*>(p.x) + row * p.ld;
  // logits before the first 16-byte boundary, vectors, logits behind the last
  const int head = min(p.V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T));
  const int nv = (p.V - head) / VEC, tail = p.V - head - nv * VEC;
  const int per = (nv + C - 1) / C, v0 = min(nv, rank * per), v1 = min(nv, v0 + per);
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  const int steps = max(1, (v1 - v0 + kThreads * U - 1) / (kThreads * U));

  uint4 raw[U];
  const uint32_t fill = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;  // -inf
  auto load = [&](int c) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + (c * U + u) * kThreads + tid;
      raw[u] = v < v1 ? __ldg(xv + v) : make_uint4(fill, fill, fill, fill);
    }
  };
  load(0);
  if (tid == 0) sm.count = 0;
  Sums own = {-INFINITY, 0.f, 0.f};
  float bound = -INFINITY;   // what a logit has to exceed to be a candidate
  bool open = true;          // no bound yet
  for (int c = 0; c < steps; ++c) {
    float f[kPer];
#pragma unroll
    for (int u = 0; u < U; ++u) widen(raw[u], f + u * VEC, T());
    if (c + 1 < steps) load(c + 1);
    // at most one of the row's ends: the first part has those before the vectors, the last those behind
    int ends = -1;
    if (c == 0 && rank == 0 && tid < head) ends = tid;
    if (c == steps - 1 && rank == C - 1 && tid >= kThreads / 2 && tid - kThreads / 2 < tail)
      ends = head + nv * VEC + tid - kThreads / 2;
    const float fe = ends >= 0 ? widen1(x[ends]) : -INFINITY;
    float top[4] = {fmaxf(f[0], fe), f[1], f[2], f[3]};
#pragma unroll
    for (int e = 4; e < kPer; ++e) top[e & 3] = fmaxf(top[e & 3], f[e]);
    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    if (most > own.m) own = merge(own, {most, 0.f, 0.f});
    const float at = own.m == -INFINITY ? 0.f : own.m;
    const uint64_t at2 = pair_f32(-at, -at), log2 = pair_f32(kLog2e, kLog2e);
    uint64_t s2[2] = {0, 0}, u2[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
      const uint64_t d = add2(pair_f32(f[e], f[e + 1]), at2);
      const float2 t = unpair_f32(mul2(d, log2)), dd = unpair_f32(d);
      const uint64_t w = pair_f32(ex2(t.x), ex2(t.y));
      s2[(e >> 1) & 1] = add2(s2[(e >> 1) & 1], w);
      // (a weight of zero times -inf would be NaN)
      u2[(e >> 1) & 1] = fma2(w, pair_f32(fmaxf(dd.x, -1e30f), fmaxf(dd.y, -1e30f)), u2[(e >> 1) & 1]);
    }
    const float2 s = unpair_f32(add2(s2[0], s2[1])), u = unpair_f32(add2(u2[0], u2[1]));
    own.s += s.x + s.y;
    own.u += u.x + u.y;
    if (ends >= 0) {
      const float w = ex2((fe - at) * kLog2e);
      own.s += w;
      own.u += w * fmaxf(fe - at, -1e30f);
    }
    if (p.top == 0) continue;

    // candidates: keys from `least` on
    const int first = head + (v0 + c * U * kThreads + tid) * VEC;
    auto each = [&](auto&& use) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int v = v0 + (c * U + e / VEC) * kThreads + tid;
        if (v < v1) use(f[e], first + (e / VEC) * kThreads * VEC + e % VEC);
      }
      if (ends >= 0) use(fe, ends);
    };
    uint64_t least;
    if (open) {
      uint64_t largest = 0;
      each([&](float v, int i) {
        const uint64_t key = key_of(v, i);
        largest = key > largest ? key : largest;
      });
      least = group_bound(sm, largest, p.top);
      if (least == 0) least = 1;
    } else {
      least = ((key_of(bound, 0) >> 32) + 1) << 32;
    }
    bool scan = open || most > bound;
    __syncthreads();  // (everyone has read the last step's count)
    const int before = sm.count;
    __syncthreads();
    for (;;) {
      if (scan) {
        each([&](float v, int i) {
          const uint64_t key = key_of(v, i);
          if (key >= least) {
            const int at_buf = atomicAdd(&sm.count, 1);
            if (at_buf < kCap) sm.buf[at_buf] = key;
          }
        });
      }
      __syncthreads();
      const int n = sm.count;
      if (n <= kCap) break;
      // too many: the bound rises to what the buffer holds, and this step's logits are looked at again
      select(sm, kCap, p.top);
      least = sm.best[p.top - 1];
      if (tid == 0) sm.count = before;
      __syncthreads();
    }
    const int n = sm.count;
    if (n > kHigh || open) {
      select(sm, n, p.top);
      const uint64_t last = sm.best[p.top - 1];
      open = last == 0;
      if (!open) bound = logit_of(last);
      if (n > kHigh) {
        if (tid < p.top) sm.buf[tid] = sm.best[tid];
        if (tid == 0) sm.count = open ? n : p.top;
      }
      __syncthreads();
    }
  }

  // the part's sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    own = merge(own, {__shfl_xor_sync(0xffffffffu, own.m, o), __shfl_xor_sync(0xffffffffu, own.s, o),
                      __shfl_xor_sync(0xffffffffu, own.u, o)});
  if (tid % 32 == 0) sm.warp[tid / 32] = own;
  __syncthreads();
  if (p.top > 0) select(sm, sm.count, p.top);
  if (tid == 0) {
    for (int w = 1; w < kThreads / 32; ++w) own = merge(own, sm.warp[w]);
  }
  __syncwarp();
  if (C > 1) {
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
    if (tid < kMaxTop) sm.best[tid] = 0;
    __syncthreads();
    for (int i = tid; i < C * p.top; i += kThreads) {
      const uint64_t key = sm.all[0][i];
      const int r = key ? rank_of(sm.all[0], C * p.top, key) : p.top;
      if (r < p.top) sm.best[r] = key;
    }
  } else {
    if (tid == 0) sm.sums[0] = own;
    __syncthreads();
    own = sm.sums[0];
  }
  __syncthreads();
  const float ln_s = logf(own.s);
  if (tid == 0) {
    p.entropy[row] = ln_s - own.u / own.s;
    if (p.tokens) {
      float lp = __uint_as_float(0x7FC00000u);
      if (token < p.V) lp = (widen1(x[token]) - own.m) - ln_s;
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

template <typename T>
cudaError_t launch_logprobs(const LogprobParams& p, int N, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(N * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)p.cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprob_kernel<T>, p);
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
  // parts of a row while there are SMs without one, none under a step of a CTA
  while (p.cluster < kMaxCluster && (int64_t)N * p.cluster * 2 <= 4 * sms && V / (2 * p.cluster) >= kThreads * kPer)
    p.cluster *= 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_result(logits_dtype == MK_F32 ? launch_logprobs<float>(p, N, s) : launch_logprobs<__nv_bfloat16>(p, N, s),
                       "mk_token_logprobs");
} catch (...) {
  return MK_ERR_NOMEM;
}
