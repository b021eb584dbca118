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
// warp that owns the segment holding the draw reads that segment once more
// (out of L2) to find the token.
//
// The product of two floats is exact in double.  The sums decide between
// neighbouring tokens of a vocabulary of 10^5, so they are carried far below
// float precision: every weight as an unevaluated pair (difference and its
// rounding error), pairs added without loss to about 2^-48, in float
// arithmetic, since the card's double adders are 64 times slower; segments
// and the final search use double.
#include <cfloat>

#include "paged.h"
#include "ptx.cuh"

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
};

// Sum of entries [i0, i1) over the warp (every lane gets it), in a fixed order.
template <bool Q>
__device__ __forceinline__ double segment_sum(const Weights& w, int i0, int i1, bool vec, int lane) {
  PairSum acc;
  if (vec) {
    int i = i0 + lane * 4;
#pragma unroll 4
    for (; i + 4 <= i1; i += 128) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(w.p + i));
      float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
      if (Q) b = __ldg(reinterpret_cast<const float4*>(w.q + i));
      float2 d[4] = {w.pair(a.x, b.x), w.pair(a.y, b.y), w.pair(a.z, b.z), w.pair(a.w, b.w)};
      const int h = w.hole - i;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (!Q && k == h) d[k] = make_float2(0.f, 0.f);
        acc.add(d[k]);
      }
    }
    for (int k = i; k < i1 && k < i + 4; ++k)  // the row's last, partial group
      if (Q || k != w.hole) acc.add(w.pair(w.p[k], Q ? w.q[k] : 0.f));
  } else {
#pragma unroll 4
    for (int i = i0 + lane; i < i1; i += 32) {
      const float a = __ldg(w.p + i), b = Q ? __ldg(w.q + i) : 0.f;
      if (Q || i != w.hole) acc.add(w.pair(a, b));
    }
  }
  double s = (double)acc.s + (double)acc.c;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams v) {
  __shared__ double seg_sum[2][kVerifyMaxCtas * kVerifyWarps];
  __shared__ int at_s, mode_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / v.ctas, rank = blockIdx.x % v.ctas;
  const int32_t* tok = v.drafts + (int64_t)b * v.K;
  const float* u = v.u + (int64_t)b * (v.K + 1);
  if (warp == 0) {
    const int len = v.draft_len ? min(max(v.draft_len[b], 0), v.K) : v.K;
    int at = len, mode = 0;  // mode 1: rejected, the draft's row is taken off
    for (int t0 = 0; t0 < len; t0 += 32) {
      const int t = t0 + lane;
      bool valid = false, yes = false;
      if (t < len) {
        const int x = tok[t];
        valid = (unsigned)x < (unsigned)v.V;
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
  bool found = false;
  int seg_at = 0;
  double base = 0.0, target = 0.0;
  if (v.ctas > 1) cluster_barrier();  // every CTA of the cluster runs before its shared memory is written
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
    // every warp finds the segment of the draw for itself: lanes hold
    // consecutive segments, summed in order
    const int per = segs / 32 > 0 ? segs / 32 : 1;
    double own = 0.0;
    for (int k = 0; k < per; ++k) {
      const int g = lane * per + k;
      if (g < segs) own += seg_sum[pass][g];
    }
    double end = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += up;
    }
    const double total = __shfl_sync(0xffffffffu, end, 31);
    if (!(total > 0.0)) {
      if (!mode) break;
      mode = 0;  // nothing is left of the target over the draft: draw from the target
      continue;
    }
    double r = u[v.K];
    r = r >= 0.0 ? r : 0.0;  // a NaN counts as zero
    target = r * total;
    // the first segment whose end exceeds the target; at u >= 1 (or by the
    // rounding of the sums) none does, and the last one of any weight is it
    double run = end - own;
    int hit = -1, last = -1;
    double hit_base = 0.0, last_base = 0.0;
    for (int k = 0; k < per; ++k) {
      const int g = lane * per + k;
      if (g >= segs) break;
      const double sg = seg_sum[pass][g];
      if (sg > 0.0) {
        last = g;
        last_base = run;
        if (hit < 0 && run + sg > target) {
          hit = g;
          hit_base = run;
        }
      }
      run += sg;
    }
    const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0), lasts = __ballot_sync(0xffffffffu, last >= 0);
    const int src = hits ? __ffs(hits) - 1 : 31 - __clz(lasts);
    seg_at = __shfl_sync(0xffffffffu, hits ? hit : last, src);
    base = __shfl_sync(0xffffffffu, hits ? hit_base : last_base, src);
    found = true;
    break;
  }
  if (!found) {
    if (rank == 0 && warp == 0) {
      for (int t = lane; t <= v.K; t += 32) v.tokens[(int64_t)b * (v.K + 1) + t] = t < at ? tok[t] : -1;
      if (lane == 0) v.accepted[b] = at;
    }
    return;
  }
  if (rank != seg_at / kVerifyWarps || warp != 0) return;
  // the token: the first entry of the segment whose running sum exceeds the target
  const int s0 = min(seg_at * v.seg, v.V), s1 = min(s0 + v.seg, v.V);
  int pick = -1, last = -1;
  for (int i = s0; i < s1 && pick < 0; i += 128) {
    double x[4], own = 0.0;
    int mine_last = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int g = i + lane * 4 + k;
      x[k] = g < s1 ? w.at(g) : 0.0;
      own += x[k];
      if (x[k] > 0.0) mine_last = g;
    }
    double end = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += up;
    }
    double run = base + (end - own);
    int hit = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      run += x[k];
      if (hit < 0 && x[k] > 0.0 && run > target) hit = i + lane * 4 + k;
    }
    const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0), some = __ballot_sync(0xffffffffu, mine_last >= 0);
    if (some) last = __shfl_sync(0xffffffffu, mine_last, 31 - __clz(some));
    if (hits) pick = __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1);
    base += __shfl_sync(0xffffffffu, end, 31);
  }
  if (pick < 0) pick = last;
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
  // fewer once the requests alone fill the SMs twice
  int ctas = kVerifyMaxCtas;
  while (ctas > 1 && ((int64_t)V < (int64_t)ctas * kVerifyWarps * 256 || (int64_t)B * ctas > 4 * (int64_t)sms)) ctas /= 2;
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
