// Verification of drafted tokens against the target's probabilities, from
// given random numbers (speculative sampling).
//
// Draft t of a request is accepted while u_t q_t(x_t) < p_t(x_t).  After the
// first rejection a token is drawn from max(p_t - q_t, 0), after the last
// accepted draft from p_t itself: the smallest i whose sum of weights up to
// i exceeds u_K times the sum of all.
//
// Only the rows of that one position are read: 2 V floats per request, which
// bound a batch (HBM); few requests are bound by the chain of reads (drafts,
// their probabilities, the row, the chosen segment).  A cluster serves a
// request; each warp sums a contiguous segment of the vocabulary, the
// segments' sums are exchanged through distributed shared memory, and the
// CTA that owns the segment holding the draw reads that segment once more
// (out of L2), all its warps together, to find the token.
//
// The product of two floats is exact in double.  The sums decide between
// neighbouring tokens of a vocabulary of 10^5, so they are carried far below
// float precision: every weight as an unevaluated pair (difference and its
// rounding error), pairs added without loss to about 2^-48, in float
// arithmetic, since a warp's double addition takes 16 cycles of an SM; only
// one warp at a time adds the sums of segments in double.
#include <cfloat>

#include "paged.h"
#include "ptx_ops.cuh"

namespace mk {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCtas = 8;  // portable cluster size

struct VerifyParams {
  const float *p, *q, *u;
  const int32_t *drafts, *draft_len;
  int32_t *tokens, *accepted, *status;
  int64_t ld_p, ld_q;  // elements between rows
  int B, K, V, ctas, seg;  // seg: vocabulary entries per warp, a multiple of 128
  int vec;             // rows 16-byte aligned
};

__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_addr(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The row the last token is drawn from, and what is taken off it.
struct Weights {
  const float* p;
  const float* q;  // subtracted, or null
  int hole;        // entry of weight zero (a draft without probabilities), or -1
  int V;
  __device__ __forceinline__ float2 pair(float a, float b) const {
    // a - b as a pair: the rounding error of a difference of a >= b >= 0 is exact
    if (!(a > b)) return make_float2(0.f, 0.f);
    const float d = a - b;
    return make_float2(d, (a - d) - b);
  }
  __device__ __forceinline__ double at(int i) const {
    if (i >= V || i == hole) return 0.0;
    const double a = p[i], b = q ? (double)q[i] : 0.0;
    return a > b ? a - b : 0.0;
  }
};

struct PairSum {
  float s = 0.f, c = 0.f;
  __device__ __forceinline__ void add(float2 w) {
    const float t = s + w.x, z = t - s;
    c += ((s - (t - z)) + (w.x - z)) + w.y;
    s = t;
  }
  // the warp's sum, in a fixed order
  __device__ __forceinline__ double reduce() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float2 w = make_float2(__shfl_xor_sync(0xffffffffu, s, o), __shfl_xor_sync(0xffffffffu, c, o));
      add(w);
    }
    return (double)s + (double)c;
  }
};

// Inclusive sums over the lanes.
__device__ __forceinline__ double lane_scan(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// The lane whose range of the running sum holds the target: the first with a weight whose end exceeds it, or
// the last with a weight where none does (u at 1 or beyond, or the rounding of sums taken in another order).
__device__ __forceinline__ int pick_lane(double own, double end, double target) {
  const unsigned hits = __ballot_sync(0xffffffffu, own > 0.0 && end > target);
  const unsigned some = __ballot_sync(0xffffffffu, own > 0.0);
  return hits ? __ffs(hits) - 1 : 31 - __clz(some);
}

// Sum of entries [i0, i1) over the warp (every lane gets it), in a fixed order.
template <bool Q>
__device__ __forceinline__ double segment_sum(const Weights& w, int i0, int i1, bool vec, int lane) {
  PairSum acc;
  if (vec) {
    int i = i0 + lane * 4;
    const auto add4 = [&](int j, float4 a, float4 b) {
      const float2 d[4] = {w.pair(a.x, b.x), w.pair(a.y, b.y), w.pair(a.z, b.z), w.pair(a.w, b.w)};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (Q || j + k != w.hole) acc.add(d[k]);
    };
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 4;  // groups of each row in flight
    for (; i + (U - 1) * 128 + 4 <= i1; i += U * 128) {
      float4 a[U], b[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        a[k] = __ldg(reinterpret_cast<const float4*>(w.p + i + k * 128));
        b[k] = Q ? __ldg(reinterpret_cast<const float4*>(w.q + i + k * 128)) : none;
      }
#pragma unroll
      for (int k = 0; k < U; ++k) add4(i + k * 128, a[k], b[k]);
    }
#pragma unroll 1
    for (; i + 4 <= i1; i += 128)
      add4(i, __ldg(reinterpret_cast<const float4*>(w.p + i)),
           Q ? __ldg(reinterpret_cast<const float4*>(w.q + i)) : none);
    for (int k = i; k < i1 && k < i + 4; ++k)  // the row's last, partial group
      if (Q || k != w.hole) acc.add(w.pair(w.p[k], Q ? w.q[k] : 0.f));
  } else {
#pragma unroll 4
    for (int i = i0 + lane; i < i1; i += 32) {
      const float a = __ldg(w.p + i), b = Q ? __ldg(w.q + i) : 0.f;
      if (Q || i != w.hole) acc.add(w.pair(a, b));
    }
  }
  return acc.reduce();
}

__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams v) {
  __shared__ double seg_sum[2][kVerifyMaxCtas * kVerifyWarps];
  __shared__ double sub_sum[kVerifyWarps];
  __shared__ double base_s, target_s, sub_base_s;
  __shared__ int at_s, mode_s, seg_s, sub_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / v.ctas, rank = blockIdx.x % v.ctas;
  const int32_t* tok = v.drafts + (int64_t)b * v.K;
  const float* u = v.u + (int64_t)b * (v.K + 1);
  // (waited for before another CTA's shared memory is written: it has to be running)
  if (v.ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (warp == 0) {
    const int len = v.draft_len ? min(max(v.draft_len[b], 0), v.K) : v.K;
    int at = len, mode = 0;  // mode 1: rejected, the draft's row is taken off
#pragma unroll 1
    for (int t0 = 0; t0 < v.K; t0 += 32) {
      const int t = t0 + lane;
      bool valid = false, yes = false;
      if (t < v.K) {
        const int x = tok[t];  // (not behind the draft's length, so that both loads are in flight)
        valid = t < len && (unsigned)x < (unsigned)v.V;
        if (valid) {
          const double pt = v.p[((int64_t)b * (v.K + 1) + t) * v.ld_p + x];
          const double qt = v.q ? (double)v.q[((int64_t)b * v.K + t) * v.ld_q + x] : 1.0;
          yes = (double)u[t] * qt < pt;
        }
      }
      const unsigned stop = __ballot_sync(0xffffffffu, t < len && !yes);
      if (stop) {
        const int k = __ffs(stop) - 1;
        at = t0 + k;
        mode = (__ballot_sync(0xffffffffu, valid) >> k) & 1;
        if (!mode && lane == 0 && rank == 0) set_status(v.status, MK_DEV_BAD_INDEX);
        break;
      }
    }
    if (lane == 0) {
      at_s = at;
      mode_s = mode;
    }
  }
  __syncthreads();
  const int at = at_s;
  int mode = mode_s;
  Weights w;
  w.V = v.V;
  w.p = v.p + ((int64_t)b * (v.K + 1) + at) * v.ld_p;
  const int segs = v.ctas * kVerifyWarps, mine = rank * kVerifyWarps + warp;
  const int i0 = min(mine * v.seg, v.V), i1 = min(i0 + v.seg, v.V);
  if (v.ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    w.q = mode && v.q ? v.q + ((int64_t)b * v.K + at) * v.ld_q : nullptr;
    w.hole = mode && !v.q ? tok[at] : -1;
    const double s = w.q ? segment_sum<true>(w, i0, i1, v.vec, lane) : segment_sum<false>(w, i0, i1, v.vec, lane);
    if (lane < v.ctas)
      asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(cluster_addr(&seg_sum[pass][mine], lane)), "d"(s)
                   : "memory");
    if (v.ctas > 1) cluster_barrier();
    else __syncthreads();
    if (warp == 0) {
      // the segment of the draw: lanes hold consecutive segments, summed in order
      const int per = (segs + 31) / 32;
      double own = 0.0;
#pragma unroll 1
      for (int k = 0; k < per; ++k)
        if (lane * per + k < segs) own += seg_sum[pass][lane * per + k];
      const double end = lane_scan(own, lane), total = __shfl_sync(0xffffffffu, end, 31);
      int seg = -1;
      double r = u[v.K], base = 0.0;
      r = r >= 0.0 ? r : 0.0;  // a NaN counts as zero
      const double target = r * total;
      if (total > 0.0) {
        const int src = pick_lane(own, end, target);
        double run = end - own;
  #pragma unroll 1
      for (int k = 0; k < per; ++k) {
          const int g = lane * per + k;
          const double x = g < segs ? seg_sum[pass][g] : 0.0;
          if (x > 0.0) {
            seg = g;
            base = run;
            if (run + x > target) break;
          }
          run += x;
        }
        seg = __shfl_sync(0xffffffffu, seg, src);
        base = __shfl_sync(0xffffffffu, base, src);
      }
      if (lane == 0) {
        seg_s = seg;
        base_s = base;
        target_s = target;
      }
    }
    __syncthreads();
    if (seg_s >= 0 || !mode) break;
    mode = 0;  // nothing is left of the target over the draft: draw from the target
    __syncthreads();
  }
  const int seg = seg_s;
  if (seg < 0) {
    if (rank == 0 && warp == 0) {
#pragma unroll 1
      for (int t = lane; t <= v.K; t += 32) v.tokens[(int64_t)b * (v.K + 1) + t] = t < at ? tok[t] : -1;
      if (lane == 0) v.accepted[b] = at;
    }
    return;
  }
  if (rank != seg / kVerifyWarps) return;
  // the token: each warp sums a sixteenth of the segment, a lane consecutive entries
  const int s0 = min(seg * v.seg, v.V), s1 = min(s0 + v.seg, v.V), sub = v.seg / kVerifyWarps;
  const int per = (sub + 31) / 32, e0 = s0 + warp * sub, e1 = min(e0 + sub, s1);
  const int l0 = min(e0 + lane * per, e1), l1 = min(l0 + per, e1);
  PairSum acc;
#pragma unroll 4
  for (int i = l0; i < l1; ++i)
    if (i != w.hole) acc.add(w.pair(__ldg(w.p + i), w.q ? __ldg(w.q + i) : 0.f));
  const double own = (double)acc.s + (double)acc.c;
  const double all = acc.reduce();
  if (lane == 0) sub_sum[warp] = all;
  __syncthreads();
  const double target = target_s;
  if (warp == 0) {
    const double x = lane < kVerifyWarps ? sub_sum[lane] : 0.0, end = base_s + lane_scan(x, lane);
    const int src = pick_lane(x, end, target);
    if (lane == src) {
      sub_s = src;
      sub_base_s = end - x;
    }
  }
  __syncthreads();
  if (warp != sub_s) return;
  const double end = sub_base_s + lane_scan(own, lane);
  const int src = pick_lane(own, end, target);
  int pick = -1;
  if (lane == src) {
    double run = end - own;
#pragma unroll 1
    for (int i = l0; i < l1; ++i) {
      const double x = w.at(i);
      run += x;
      if (x > 0.0) {
        pick = i;
        if (run > target) break;
      }
    }
  }
  pick = __shfl_sync(0xffffffffu, pick, src);
#pragma unroll 1
  for (int t = lane; t <= v.K; t += 32)
    v.tokens[(int64_t)b * (v.K + 1) + t] = t < at ? tok[t] : t == at ? pick : -1;
  if (lane == 0) v.accepted[b] = at;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_verify_drafts(void* stream, int B, int K, int V, const float* p, int64_t ld_p, const float* q,
                                int64_t ld_q, const int32_t* drafts, const int32_t* draft_len, const float* u,
                                int32_t* tokens, int32_t* accepted, int32_t* status) try {
  if (!p || !u || !tokens || !accepted || (K > 0 && !drafts))
    return fail(MK_ERR_ARG, "mk_verify_drafts: null argument");
  if (B < 0 || K < 0 || K > 1024 || V < 1) return fail(MK_ERR_ARG, "mk_verify_drafts: need B >= 0, 0 <= K <= 1024, V >= 1");
  if (ld_p < V || (q && ld_q < V)) return fail(MK_ERR_ARG, "mk_verify_drafts: row strides must cover a row");
  if (V > (1 << 28) || B > (1 << 24)) return fail(MK_ERR_LIMIT, "mk_verify_drafts: V at most 2^28, B at most 2^24");
  if (int rc = pending_error("mk_verify_drafts")) return rc;
  if (B == 0) return MK_OK;
  int sms = 0;
  if (int rc = device_sms("mk_verify_drafts", &sms)) return rc;
  VerifyParams v{};
  v.p = p; v.q = q; v.u = u; v.drafts = drafts; v.draft_len = draft_len;
  v.tokens = tokens; v.accepted = accepted; v.status = status;
  v.ld_p = ld_p; v.ld_q = ld_q; v.B = B; v.K = K; v.V = V;
  v.vec = aligned16(p) && ld_p % 4 == 0 && (!q || (aligned16(q) && ld_q % 4 == 0));
  // as many CTAs per request as still give every warp a few 128-entry steps,
  // fewer once two CTAs per SM are there (64 requests of 128256 entries: 3, 4,
  // 6, 8 CTAs each took 16.6, 14.3, 14.9 and 17.6 us, one request 8.8 us with 8;
  // in a graph, with the rows in the L2: on changing rows the 64 take 20 us)
  int ctas = kVerifyMaxCtas;
  while (ctas > 1 && ((int64_t)V < (int64_t)ctas * kVerifyWarps * 256 || (int64_t)B * ctas > 2 * (int64_t)sms)) ctas /= 2;
  v.ctas = ctas;
  const int64_t warps = (int64_t)ctas * kVerifyWarps;
  v.seg = (int)((((int64_t)V + warps - 1) / warps + 127) / 128 * 128);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)B * (unsigned)ctas);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return launch_result(cudaLaunchKernelEx(&cfg, verify_kernel, v), "mk_verify_drafts");
} catch (...) {
  return MK_ERR_NOMEM;
}
