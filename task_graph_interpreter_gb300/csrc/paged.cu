// Paged KV cache: the step plan (block tables, slot maps) and the per-head
// norms with the rotary position embedding and the stores into pages.
#include <cmath>

#include <cuda_bf16.h>

#include "paged.h"
#include "ptx.cuh"

namespace mk {
namespace {

// ------------------------------------------------------------------ plan
//
// Request b needs want = ceil((ctx + new) / page) pages and holds `held`.
// Pages beyond `want` go on top of the stack of free pages in the order of
// requests; then each growing request takes its pages from the top.  With
// the exclusive sums of new tokens, taken and returned pages over the
// requests, every output element is a function of its index alone, so all
// threads work without order: the a-th page taken is virtual stack entry
// top - 1 - a, below `count` a free page, above it the returned page number
// (entry - count), found by a search in the returned pages' sums.
//
// Bound by latency, not bytes (a full server's step moves under 1 MB): one
// cluster, whose CTAs each compute the sums for themselves (a block scan of
// up to 4096 requests) rather than exchange them, and the only barrier
// before the held pages, the count and the returned pages are stored, since
// those may be the arrays that other CTAs still read.
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 4096;
constexpr int kPlanCtas = 8;

struct PlanParams {
  const int32_t *ctx, *len, *held, *count;
  int32_t *table, *free_pages, *held_out, *count_out, *cu, *positions, *slots, *status;
  int B, page_shift, max_pages, num_pages, max_tokens;
  int vec;  // positions and slots 16-byte aligned
};

__device__ __forceinline__ int plan_want(const PlanParams& p, int b) {
  return (int)(((int64_t)p.ctx[b] + p.len[b] + (1 << p.page_shift) - 1) >> p.page_shift);
}

struct PlanPages {
  const PlanParams& p;
  const int32_t *goff, *boff;
  int count, top;
  // the a-th page taken from the stack
  __device__ int taken(int a) const {
    const int v = top - 1 - a;
    if (v < count) return p.free_pages[v];
    return returned(v - count);
  }
  __device__ int returned(int f) const {
    const int b = upper_row(boff, p.B, f);
    return p.table[(size_t)b * p.max_pages + plan_want(p, b) + (f - boff[b])];
  }
  // the page holding page index j of request b after the step
  __device__ int of(int b, int j, int held) const {
    if (j < held) return p.table[(size_t)b * p.max_pages + j];
    return taken(goff[b] + j - held);
  }
};

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  extern __shared__ int32_t sm[];
  int32_t* cu = sm;                 // [B + 1]
  int32_t* goff = cu + p.B + 1;     // [B + 1] pages taken
  int32_t* boff = goff + p.B + 1;   // [B + 1] pages returned
  __shared__ long long warp_sum[3][kPlanThreads / 32];
  __shared__ int err_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, ctas = gridDim.x;
  if (tid == 0) err_s = MK_DEV_OK;
  __syncthreads();
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long sum[3] = {0, 0, 0};
  int err = MK_DEV_OK;
  for (int b = b0; b < b1; ++b) {
    const int c = p.ctx[b], n = p.len[b], h = p.held[b];
    if (c < 0 || n < 0 || h < 0 || h > p.max_pages) {
      err = MK_DEV_BAD_INDEX;
      continue;
    }
    const int64_t w = ((int64_t)c + n + (1 << p.page_shift) - 1) >> p.page_shift;
    if (w > p.max_pages) {
      if (err == MK_DEV_OK) err = MK_DEV_CAPACITY;
      continue;
    }
    sum[0] += n;
    sum[1] += max((int)w - h, 0);
    sum[2] += max(h - (int)w, 0);
  }
  if (err != MK_DEV_OK) atomicCAS(&err_s, MK_DEV_OK, err);
  // exclusive scan of the three sums over the block
  long long ex[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long v = sum[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) warp_sum[k][warp] = v;
    ex[k] = v - sum[k];
  }
  __syncthreads();
  long long total[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long before = 0, all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) before += warp_sum[k][w];
      all += warp_sum[k][w];
    }
    ex[k] += before;
    total[k] = all;
  }
  const int count = *p.count;
  int code = err_s;
  if (code == MK_DEV_OK) {
    if (count < 0 || count > p.num_pages || count + total[2] > p.num_pages) code = MK_DEV_BAD_INDEX;
    else if (total[0] > p.max_tokens || total[1] > count + total[2]) code = MK_DEV_CAPACITY;
  }
  const bool ok = code == MK_DEV_OK;
  const int ntok = ok ? (int)total[0] : 0, ngrow = ok ? (int)total[1] : 0, nback = ok ? (int)total[2] : 0;
  if (ok) {
    for (int b = b0; b < b1; ++b) {
      const int n = p.len[b], h = p.held[b], w = plan_want(p, b);
      cu[b] = (int)ex[0];
      goff[b] = (int)ex[1];
      boff[b] = (int)ex[2];
      ex[0] += n;
      ex[1] += max(w - h, 0);
      ex[2] += max(h - w, 0);
    }
  } else {
    for (int b = b0; b < b1; ++b) cu[b] = goff[b] = boff[b] = 0;
  }
  if (tid == 0) {
    cu[p.B] = ntok;
    goff[p.B] = ngrow;
    boff[p.B] = nback;
  }
  __syncthreads();
  const PlanPages pages{p, goff, boff, count, count + nback};
  const int gtid = rank * kPlanThreads + tid, nthr = ctas * kPlanThreads;
  // block tables: the pages taken
  for (int a = gtid; a < ngrow; a += nthr) {
    const int b = upper_row(goff, p.B, a);
    const int held = plan_want(p, b) - (goff[b + 1] - goff[b]);
    const int id = pages.taken(a);
    p.table[(size_t)b * p.max_pages + held + (a - goff[b])] = id;
    if ((unsigned)id >= (unsigned)p.num_pages) set_status(p.status, MK_DEV_BAD_INDEX);
  }
  // positions and slots, four tokens a thread
  const int pmask = (1 << p.page_shift) - 1;
  for (int i0 = gtid * 4; i0 < p.max_tokens; i0 += nthr * 4) {
    int pos[4], slot[4];
    int b = i0 < ntok ? upper_row(cu, p.B, i0) : 0, at_b = -1, at_j = -1, id = -1, ctx = 0, held = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k;
      pos[k] = slot[k] = -1;
      if (i < ntok) {
        while (cu[b + 1] <= i) ++b;
        if (b != at_b) {
          ctx = p.ctx[b];
          // pages kept from before: all of the held ones, or the wanted ones
          held = plan_want(p, b) - (goff[b + 1] - goff[b]);
          at_b = b;
          at_j = -1;
        }
        pos[k] = ctx + (i - cu[b]);
        const int j = pos[k] >> p.page_shift;
        if (j != at_j) {
          id = pages.of(b, j, held);
          at_j = j;
        }
        if ((unsigned)id < (unsigned)p.num_pages) slot[k] = (id << p.page_shift) + (pos[k] & pmask);
        else set_status(p.status, MK_DEV_BAD_INDEX);
      }
    }
    if (p.vec && i0 + 4 <= p.max_tokens) {
      *reinterpret_cast<int4*>(p.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(p.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
      for (int k = 0; k < 4 && i0 + k < p.max_tokens; ++k) {
        p.positions[i0 + k] = pos[k];
        p.slots[i0 + k] = slot[k];
      }
    }
  }
  // the returned pages that stay on the stack
  const int left = count + nback - ngrow;
  for (int f = gtid; f < nback && count + f < left; f += nthr) p.free_pages[count + f] = pages.returned(f);
  // held pages and the count may be the arrays that every CTA reads above
  if (ctas > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  if (rank != 0) return;
  for (int b = tid; b < p.B; b += kPlanThreads) {
    const int h = p.held[b];
    p.held_out[b] = ok ? plan_want(p, b) : h;
  }
  for (int b = tid; b <= p.B; b += kPlanThreads) p.cu[b] = cu[b];
  if (tid == 0) {
    *p.count_out = ok ? left : count;
    if (!ok) set_status(p.status, code);
  }
}

// ------------------------------------------------------------------ norms, rotation, store
//
//   y = x / sqrt(mean(x^2) + eps) * gamma        over a head's D elements
//   (y_i, y_{i + D/2}) turned by pos * theta^(-2i/D)
//
// for query and key heads; query heads go to q (bf16), key and value heads
// to the pages.  Bound by bytes: every element is read once and written
// once.  A head belongs to D / (2 E) neighbouring lanes, E = 4 (f32) or 8
// (16 bits) elements of each half per lane, so loads are 16 bytes and the
// two halves of a pair meet in one lane.  A lane group keeps its token's
// angles in registers over the heads it does in turn; the launch gives it
// as many as leave a thousand threads per SM.
//
// The angle in revolutions is pos * f mod 1, f = theta^(-2i/D) / (2 pi): with
// f as a 64-bit fraction (units of 2^-64) the product modulo 2^64 is that
// remainder without rounding, for any position, and its upper 32 bits give
// the angle to 2^-32 of a turn; sincospif then works on [-1, 1).
constexpr int kNormThreads = 256;

struct NormParams {
  const void* x;
  int64_t ld_x, ld_q;
  const __nv_bfloat16 *q_gamma, *k_gamma;
  const int32_t *positions, *slots;
  __nv_bfloat16 *q, *kpool, *vpool;
  int32_t* status;
  int N, Hq, Hkv, page_shift, num_pages, splits;
  float eps;
  uint64_t freq[64];  // [D / 2]
};

template <int E>
__device__ __forceinline__ void load_half(const float* p, float (&v)[E]) {
#pragma unroll
  for (int i = 0; i < E; i += 4) {
    const float4 t = __ldg(reinterpret_cast<const float4*>(p + i));
    v[i] = t.x; v[i + 1] = t.y; v[i + 2] = t.z; v[i + 3] = t.w;
  }
}
template <int E>
__device__ __forceinline__ void load_half(const __nv_bfloat16* p, float (&v)[E]) {
  if constexpr (E == 8) {
    const uint4 t = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = ptx::bf_lo(w[i]);
      v[2 * i + 1] = ptx::bf_hi(w[i]);
    }
  } else {
    const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = ptx::bf_lo(t.x); v[1] = ptx::bf_hi(t.x); v[2] = ptx::bf_lo(t.y); v[3] = ptx::bf_hi(t.y);
  }
}
using ptx::pack_bf16;
template <int E>
__device__ __forceinline__ void store_half(__nv_bfloat16* p, const float (&v)[E]) {
  if constexpr (E == 8)
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

template <typename T, int D>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ NormParams p) {
  constexpr int E = sizeof(T) == 4 ? 4 : 8;
  constexpr int LPH = D / 2 / E;  // lanes per head
  const int gl = threadIdx.x % LPH;
  const int64_t unit = (int64_t)blockIdx.x * (kNormThreads / LPH) + threadIdx.x / LPH;
  const int row = (int)(unit / p.splits), split = (int)(unit % p.splits);
  if (row >= p.N) return;  // whole lane groups leave; the shuffles below name their group's lanes only
  const int pos = p.positions[row], slot = p.slots[row];
  if (pos < 0) return;
  const unsigned mask = (LPH == 32 ? 0xffffffffu : ((1u << LPH) - 1u)) << ((threadIdx.x & 31) / LPH * LPH);
  float cs[E], sn[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint64_t turn = (uint64_t)(uint32_t)pos * p.freq[gl * E + i];
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn[i], &cs[i]);
  }
  const int heads = p.Hq + 2 * p.Hkv;
  const T* x = static_cast<const T*>(p.x) + (int64_t)row * p.ld_x + gl * E;
  const int pg = slot >> p.page_shift, off = slot & ((1 << p.page_shift) - 1);
  const bool store = slot >= 0 && pg < p.num_pages;
  if (slot >= 0 && !store && gl == 0 && split == 0) set_status(p.status, MK_DEV_BAD_INDEX);
#pragma unroll 2
  for (int h = split; h < heads; h += p.splits) {
    float a[E], b[E];
    load_half<E>(x + (int64_t)h * D, a);
    load_half<E>(x + (int64_t)h * D + D / 2, b);
    const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
    if (!is_v) {
      const __nv_bfloat16* gamma = is_q ? p.q_gamma : p.k_gamma;
      if (gamma) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
        const float r = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
        float ga[E], gb[E];
        load_half<E>(gamma + gl * E, ga);
        load_half<E>(gamma + gl * E + D / 2, gb);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          a[i] *= r * ga[i];
          b[i] *= r * gb[i];
        }
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float u = a[i], w = b[i];
        a[i] = u * cs[i] - w * sn[i];
        b[i] = w * cs[i] + u * sn[i];
      }
    }
    __nv_bfloat16* dst;
    if (is_q) {
      dst = p.q + (int64_t)row * p.ld_q + (int64_t)h * D;
    } else {
      if (!store) continue;
      const int g = h - p.Hq - (is_v ? p.Hkv : 0);
      dst = (is_v ? p.vpool : p.kpool) + ((((int64_t)pg * p.Hkv + g) << p.page_shift) + off) * D;
    }
    store_half<E>(dst + gl * E, a);
    store_half<E>(dst + gl * E + D / 2, b);
  }
}

template <typename T, int D>
cudaError_t launch_norm(NormParams& p, int sms, cudaStream_t stream) {
  constexpr int E = sizeof(T) == 4 ? 4 : 8;
  constexpr int LPH = D / 2 / E;
  const int heads = p.Hq + 2 * p.Hkv;
  // heads in turn per lane group: fewer while the launch would hold under a
  // thousand threads per SM
  int turns = 8;
  while (turns > 1 && (int64_t)p.N * ((heads + turns - 1) / turns) * LPH < (int64_t)sms * 1024) turns >>= 1;
  p.splits = (heads + turns - 1) / turns;
  const int64_t units = (int64_t)p.N * p.splits, per = kNormThreads / LPH;
  norm_rope_kernel<T, D><<<(unsigned)((units + per - 1) / per), kNormThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_paged_plan(void* stream, int B, int page_size, int max_pages, int num_pages, int max_tokens,
                             const int32_t* ctx_len, const int32_t* new_len, int32_t* table, const int32_t* held,
                             int32_t* held_out, int32_t* free_pages, const int32_t* free_count,
                             int32_t* free_count_out, int32_t* cu, int32_t* positions, int32_t* slots,
                             int32_t* status) try {
  if (!ctx_len || !new_len || !table || !held || !held_out || !free_pages || !free_count || !free_count_out || !cu ||
      !positions || !slots)
    return fail(MK_ERR_ARG, "mk_paged_plan: null argument");
  if (B < 1 || B > kPlanMaxB) return fail(MK_ERR_ARG, "mk_paged_plan: need 1 <= B <= 4096");
  if (!page_size_ok(page_size)) return fail(MK_ERR_ARG, "mk_paged_plan: page_size must be 16, 32, 64, 128 or 256");
  if (max_pages < 1 || num_pages < 1 || max_tokens < 1)
    return fail(MK_ERR_ARG, "mk_paged_plan: max_pages, num_pages and max_tokens must be positive");
  if ((int64_t)num_pages * page_size > INT32_MAX || (int64_t)max_pages * page_size > INT32_MAX ||
      max_tokens > INT32_MAX - kPlanCtas * kPlanThreads * 4)
    return fail(MK_ERR_LIMIT, "mk_paged_plan: slots and positions must fit int32");
  if (int rc = pending_error("mk_paged_plan")) return rc;
  PlanParams p{};
  p.ctx = ctx_len; p.len = new_len; p.held = held; p.count = free_count;
  p.table = table; p.free_pages = free_pages; p.held_out = held_out; p.count_out = free_count_out;
  p.cu = cu; p.positions = positions; p.slots = slots; p.status = status;
  p.B = B; p.max_pages = max_pages; p.num_pages = num_pages; p.max_tokens = max_tokens;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.vec = aligned16(positions) && aligned16(slots);
  const size_t smem = (size_t)3 * (B + 1) * 4;
  if (smem > 48 * 1024 - 512) {
    const cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return launch_result(e, "mk_paged_plan");
  }
  // one CTA does 2048 tokens in one pass of its threads; the sums are the rest of its time
  int ctas = 1;
  while (ctas < kPlanCtas && max_tokens > ctas * kPlanThreads * 4) ctas *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return launch_result(cudaLaunchKernelEx(&cfg, plan_kernel, p), "mk_paged_plan");
} catch (...) {
  return MK_ERR_NOMEM;
}

extern "C" int mk_qk_norm_rope(void* stream, int N, int Hq, int Hkv, int D, const void* qkv, int qkv_dtype,
                               int64_t ld_qkv, const void* q_gamma, const void* k_gamma, float eps, double rope_theta,
                               const int32_t* positions, const int32_t* slots, void* q_out, int64_t ld_q, void* kpool,
                               void* vpool, int num_pages, int page_size, int32_t* status) try {
  if (!qkv || !positions || !slots || !q_out || !kpool || !vpool)
    return fail(MK_ERR_ARG, "mk_qk_norm_rope: null argument");
  if (N < 0 || Hq < 1 || Hkv < 1 || Hq > 1024 || Hkv > 1024)
    return fail(MK_ERR_ARG, "mk_qk_norm_rope: need N >= 0 and 1 to 1024 heads");
  if (D != 64 && D != 128) return fail(MK_ERR_ARG, "mk_qk_norm_rope: D must be 64 or 128");
  if (qkv_dtype != MK_F32 && qkv_dtype != MK_BF16) return fail(MK_ERR_ARG, "mk_qk_norm_rope: qkv must be f32 or bf16");
  if (!page_size_ok(page_size)) return fail(MK_ERR_ARG, "mk_qk_norm_rope: page_size must be 16, 32, 64, 128 or 256");
  if (num_pages < 1 || (int64_t)num_pages * page_size > INT32_MAX)
    return fail(MK_ERR_ARG, "mk_qk_norm_rope: num_pages * page_size must be in [1, 2^31)");
  if (!(rope_theta > 0.0) || !std::isfinite(rope_theta) || !(eps >= 0.f) || !std::isfinite(eps))
    return fail(MK_ERR_ARG, "mk_qk_norm_rope: bad rope_theta or eps");
  const int64_t width = (int64_t)(Hq + 2 * Hkv) * D, unit = qkv_dtype == MK_F32 ? 4 : 8;
  if (ld_qkv < width || ld_qkv % unit || ld_q < (int64_t)Hq * D || ld_q % 8)
    return fail(MK_ERR_ARG, "mk_qk_norm_rope: row strides must cover a row and be multiples of 16 bytes");
  if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(kpool) || !aligned16(vpool) || !aligned16(q_gamma) ||
      !aligned16(k_gamma))
    return fail(MK_ERR_ARG, "mk_qk_norm_rope: pointers must be 16-byte aligned");
  if (int rc = pending_error("mk_qk_norm_rope")) return rc;
  if (N == 0) return MK_OK;
  NormParams p{};
  p.x = qkv; p.ld_x = ld_qkv; p.ld_q = ld_q;
  p.q_gamma = static_cast<const __nv_bfloat16*>(q_gamma);
  p.k_gamma = static_cast<const __nv_bfloat16*>(k_gamma);
  p.positions = positions; p.slots = slots;
  p.q = static_cast<__nv_bfloat16*>(q_out);
  p.kpool = static_cast<__nv_bfloat16*>(kpool);
  p.vpool = static_cast<__nv_bfloat16*>(vpool);
  p.status = status; p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.num_pages = num_pages; p.eps = eps;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  // the last base's frequencies: a decoder asks for the same ones in every layer
  thread_local struct {
    double theta = 0.0;
    int D = 0;
    uint64_t f[64];
  } known;
  if (known.theta != rope_theta || known.D != D) {
    for (int i = 0; i < D / 2; ++i) {
      // revolutions per position, reduced below one, in units of 2^-64
      const double f = std::fmod(std::pow(rope_theta, -2.0 * i / D) / 6.283185307179586476925, 1.0);
      known.f[i] = (uint64_t)std::ldexp(f, 64);
    }
    known.theta = rope_theta;
    known.D = D;
  }
  for (int i = 0; i < D / 2; ++i) p.freq[i] = known.f[i];
  int sms = 0;
  if (int rc = device_sms("mk_qk_norm_rope", &sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (qkv_dtype == MK_F32) e = D == 128 ? launch_norm<float, 128>(p, sms, s) : launch_norm<float, 64>(p, sms, s);
  else e = D == 128 ? launch_norm<__nv_bfloat16, 128>(p, sms, s) : launch_norm<__nv_bfloat16, 64>(p, sms, s);
  return launch_result(e, "mk_qk_norm_rope");
} catch (...) {
  return MK_ERR_NOMEM;
}
