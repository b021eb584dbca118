// Paged KV cache: the step plan (block tables, slot maps) and the per-head
// norms with the rotary position embedding and the stores into pages.
#include "paged_norm.cuh"

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
// up to 4096 requests) rather than exchange them.  One barrier: before it the
// tables get their new pages, after it tokens look their pages up there and
// the held pages, the count and the returned pages are stored, which may be
// the arrays that were read before.  (509 requests, 65,000 tokens: 39 us of
// work for one CTA, so eight; tokens that resolved new pages themselves took
// twice as long.)
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanMaxB = 4096;
constexpr int kPlanCtas = 8;

struct PlanParams {
  const int32_t *ctx, *len, *held, *count;
  int32_t *table, *free_pages, *held_out, *count_out, *cu, *positions, *slots, *status;
  int B, page_shift, max_pages, num_pages, max_tokens;
  int vec;  // positions and slots 16-byte aligned
};

// What a CTA knows of every request, in shared memory: exclusive sums of new
// tokens, of pages taken and of pages returned [B + 1 each], cached tokens,
// and the pages kept from before, min(held, want).
struct PlanPages {
  const PlanParams& p;
  int32_t *cu, *goff, *boff, *ctx, *kept;
  int count, top;
  __device__ PlanPages(const PlanParams& p_, int32_t* sm) : p(p_) {
    cu = sm;
    goff = cu + p.B + 1;
    boff = goff + p.B + 1;
    ctx = boff + p.B + 1;
    kept = ctx + p.B;
  }
  // a returned page, and the a-th page taken from the stack
  __device__ int returned(int f) const {
    const int b = upper_row(boff, p.B, f);
    return p.table[(size_t)b * p.max_pages + kept[b] + (f - boff[b])];
  }
  __device__ int taken(int a) const {
    const int v = top - 1 - a;
    return v < count ? p.free_pages[v] : returned(v - count);
  }
};

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  extern __shared__ int32_t sm[];
  __shared__ long long warp_sum[3][kPlanWarps];
  __shared__ int err_s;
  PlanPages pages(p, sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, ctas = gridDim.x, threads = blockDim.x;
  const int count = *p.count;
  if (tid == 0) err_s = MK_DEV_OK;
  __syncthreads();
  const int per = (p.B + threads - 1) / threads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long sum[3] = {0, 0, 0};
  int err = MK_DEV_OK;
  for (int b = b0; b < b1; ++b) {
    const int c = p.ctx[b], n = p.len[b], h = p.held[b];
    const int64_t w = ((int64_t)c + n + (1 << p.page_shift) - 1) >> p.page_shift;
    if (c < 0 || n < 0 || h < 0 || h > p.max_pages) {
      err = MK_DEV_BAD_INDEX;
      continue;
    }
    if (w > p.max_pages) {
      if (err == MK_DEV_OK) err = MK_DEV_CAPACITY;
      continue;
    }
    const int grow = max((int)w - h, 0), back = max(h - (int)w, 0);
    // (each request's own counts, until the sums before them are known)
    pages.cu[b] = n;
    pages.goff[b] = grow;
    pages.boff[b] = back;
    pages.ctx[b] = c;
    pages.kept[b] = min(h, (int)w);
    sum[0] += n;
    sum[1] += grow;
    sum[2] += back;
  }
  if (err != MK_DEV_OK) atomicCAS(&err_s, MK_DEV_OK, err);
  // exclusive scan of the three sums over the block
  long long ex[3], total[3];
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
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long v = lane < threads / 32 ? warp_sum[k][lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    total[k] = __shfl_sync(0xffffffffu, v, 31);
    const long long before = __shfl_sync(0xffffffffu, v, max(warp - 1, 0));
    if (warp > 0) ex[k] += before;
  }
  int code = err_s;
  if (code == MK_DEV_OK) {
    if (count < 0 || count > p.num_pages || count + total[2] > p.num_pages) code = MK_DEV_BAD_INDEX;
    else if (total[0] > p.max_tokens || total[1] > count + total[2]) code = MK_DEV_CAPACITY;
  }
  const bool ok = code == MK_DEV_OK;
  const int ntok = ok ? (int)total[0] : 0, ngrow = ok ? (int)total[1] : 0, nback = ok ? (int)total[2] : 0;
  for (int b = b0; b < b1; ++b) {
    const int n = ok ? pages.cu[b] : 0, grow = ok ? pages.goff[b] : 0, back = ok ? pages.boff[b] : 0;
    pages.cu[b] = ok ? (int)ex[0] : 0;
    pages.goff[b] = ok ? (int)ex[1] : 0;
    pages.boff[b] = ok ? (int)ex[2] : 0;
    ex[0] += n;
    ex[1] += grow;
    ex[2] += back;
  }
  if (tid == 0) {
    pages.cu[p.B] = ntok;
    pages.goff[p.B] = ngrow;
    pages.boff[p.B] = nback;
  }
  pages.count = count;
  pages.top = count + nback;
  __syncthreads();
  const int gtid = rank * threads + tid, nthr = ctas * threads;
  // block tables: the pages taken
  for (int a = gtid; a < ngrow; a += nthr) {
    const int b = upper_row(pages.goff, p.B, a);
    const int id = pages.taken(a);
    p.table[(size_t)b * p.max_pages + pages.kept[b] + (a - pages.goff[b])] = id;
    if ((unsigned)id >= (unsigned)p.num_pages) set_status(p.status, MK_DEV_BAD_INDEX);
  }
  // the tables are whole, and every CTA has read the held pages and the count, which may be stored in place
  if (ctas > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  // positions and slots, four tokens a thread
  const int pmask = (1 << p.page_shift) - 1;
  for (int i0 = gtid * 4; i0 < p.max_tokens; i0 += nthr * 4) {
    int pos[4], slot[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) pos[k] = slot[k] = -1;
    if (i0 < ntok) {
      int b = upper_row(pages.cu, p.B, i0);
      const int n = min(4, ntok - i0);
      if (pages.cu[b + 1] >= i0 + n) {  // one request: at most two pages
        const int p0 = pages.ctx[b] + (i0 - pages.cu[b]), j0 = p0 >> p.page_shift, j1 = (p0 + n - 1) >> p.page_shift;
        const int32_t* at = p.table + (size_t)b * p.max_pages;
        const int id0 = __ldcg(at + j0), id1 = __ldcg(at + j1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k >= n) break;
          pos[k] = p0 + k;
          slot[k] = (pos[k] >> p.page_shift) == j0 ? id0 : id1;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k >= n) break;
          while (pages.cu[b + 1] <= i0 + k) ++b;
          pos[k] = pages.ctx[b] + (i0 + k - pages.cu[b]);
          slot[k] = __ldcg(p.table + (size_t)b * p.max_pages + (pos[k] >> p.page_shift));
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k >= n) break;
        if ((unsigned)slot[k] < (unsigned)p.num_pages) {
          slot[k] = (slot[k] << p.page_shift) + (pos[k] & pmask);
        } else {
          slot[k] = -1;
          set_status(p.status, MK_DEV_BAD_INDEX);
        }
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
  if (rank != 0) return;
  for (int b = tid; b < p.B; b += threads) {
    const int h = p.held[b];
    p.held_out[b] = ok ? pages.kept[b] + (pages.goff[b + 1] - pages.goff[b]) : h;
  }
  for (int b = tid; b <= p.B; b += threads) p.cu[b] = pages.cu[b];
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
// two halves of a pair meet in one lane.  A block takes the heads of one to
// four tokens: each lane group loads its heads of one token, the block works
// out the tokens' angles with the gains folded in,
//   y_a = r (a ca - b sb),  y_b = r (b cb + a sa),
// once in shared memory, and the heads are then done in packed pairs of
// floats: at 16 bits the instructions per element are the second bound.
//
// The angle in revolutions is pos * f mod 1, f = theta^(-2i/D) / (2 pi): with
// f as a 64-bit fraction (units of 2^-64) the product modulo 2^64 is that
// remainder without rounding, for any position, and its upper 32 bits give
// the angle to 2^-32 of a turn; sincospif then works on [-1, 1).

constexpr int kNormBatch = 3;      // heads a lane group has in flight
constexpr int kNormMaxTokens = 4;  // tokens of a block
// Small blocks: a block's loads, angles and stores follow one another, and
// many of them overlap better (8192 tokens of 48 heads of 128 in 16 bits:
// 64 threads 35.5 us, 5.7 TB/s; 128 39; 256 42).
template <typename T, int D>
constexpr int kNormThreads = sizeof(T) == 4 ? (D == 128 ? 128 : 64) : 64;

template <typename T, int D>
__global__ void __launch_bounds__((kNormThreads<T, D>), (768 / kNormThreads<T, D>)) norm_rope_kernel(const __grid_constant__ NormParams p) {
  constexpr int E = sizeof(T) == 4 ? 4 : 8;
  constexpr int LPH = D / 2 / E;              // lanes per head
  constexpr int GP = kNormThreads<T, D> / LPH;  // lane groups of a block
  // per token, for query and key heads: ca, -sb, cb, sa
  __shared__ __align__(16) float coef[kNormMaxTokens][2][4][D / 2];
  const int gl = threadIdx.x % LPH, group = threadIdx.x / LPH;
  const int gt = GP / p.tokens;                          // lane groups of a token
  const int tk = group / gt;
  const int row0 = blockIdx.x / p.splits * p.tokens, row = row0 + tk;
  const int step = gt * p.splits, h0 = group % gt + blockIdx.x % p.splits * gt;
  const int hk0 = p.Hq, hv0 = p.Hq + p.Hkv, heads = p.Hq + 2 * p.Hkv;
  const unsigned mask = (LPH == 32 ? 0xffffffffu : ((1u << LPH) - 1u)) << ((threadIdx.x & 31) / LPH * LPH);
  const bool there = row < p.N;
  const T* x = static_cast<const T*>(p.x) + (int64_t)(there ? row : 0) * p.ld_x + gl * E;
  __nv_bfloat16* q = p.q + (int64_t)row * p.ld_q + gl * E;
  int pos = -1, slot = -1;
  int64_t at = 0;  // head 0's row in its page
  bool store = false;
  for (int h = h0; h < heads || h == h0; h += kNormBatch * step) {
    Raw<T, E> ra[kNormBatch], rb[kNormBatch];
#pragma unroll
    for (int k = 0; k < kNormBatch; ++k) {
      const int hk = h + k * step;
      if (hk < heads) {  // (left-out rows too: the position is still on its way)
        ra[k].load(x + hk * D);
        rb[k].load(x + hk * D + D / 2);
      }
    }
    if (h == h0) {
      if (there) {
        pos = p.positions[row];
        slot = p.slots[row];
      }
      for (int i = threadIdx.x; i < p.tokens * (D / 2); i += kNormThreads<T, D>) {
        const int t = i / (D / 2), j = i % (D / 2), r = row0 + t;
        const int at_pos = r < p.N ? p.positions[r] : 0;
        float gain[2][2];
#pragma unroll
        for (int cl = 0; cl < 2; ++cl) {
          const __nv_bfloat16* g = cl ? p.k_gamma : p.q_gamma;
          gain[cl][0] = g ? __bfloat162float(g[j]) : 1.f;
          gain[cl][1] = g ? __bfloat162float(g[j + D / 2]) : 1.f;
        }
        const uint64_t turn = (uint64_t)(uint32_t)at_pos * p.freq[j];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
#pragma unroll
        for (int cl = 0; cl < 2; ++cl) {
          const float ga = gain[cl][0], gb = gain[cl][1];
          coef[t][cl][0][j] = c * ga;
          coef[t][cl][1][j] = -s * gb;
          coef[t][cl][2][j] = c * gb;
          coef[t][cl][3][j] = s * ga;
        }
      }
      __syncthreads();
      const int pg = slot >> p.page_shift, off = slot & ((1 << p.page_shift) - 1);
      store = slot >= 0 && pg < p.num_pages;
      at = (((int64_t)pg * p.Hkv << p.page_shift) + off) * D + gl * E;
      if (pos >= 0 && slot >= 0 && !store && gl == 0 && group % gt == 0) set_status(p.status, MK_DEV_BAD_INDEX);
    }
    if (pos < 0) break;  // left out (whole lane groups; the shuffles name their lanes only)
#pragma unroll
    for (int k = 0; k < kNormBatch; ++k) {
      const int hk = h + k * step;
      if (hk >= heads) break;
      float a[E], b[E];
      ra[k].get(a);
      rb[k].get(b);
      if (hk < hv0) {
        const bool is_q = hk < hk0;
        float r = 1.f;
        if ((is_q ? p.q_gamma : p.k_gamma) != nullptr) {
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
        const uint64_t r2 = ptx::pair_f32(r, r);
        const float* cf = &coef[tk][is_q ? 0 : 1][0][gl * E];
#pragma unroll
        for (int i = 0; i < E; i += 4) {
          const float4 ca = *reinterpret_cast<const float4*>(cf + i), sb = *reinterpret_cast<const float4*>(cf + D / 2 + i);
          const float4 cb = *reinterpret_cast<const float4*>(cf + D + i),
                       sa = *reinterpret_cast<const float4*>(cf + 3 * D / 2 + i);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint64_t u = ptx::mul2(r2, ptx::pair_f32(a[i + 2 * e], a[i + 2 * e + 1]));
            const uint64_t v = ptx::mul2(r2, ptx::pair_f32(b[i + 2 * e], b[i + 2 * e + 1]));
            const uint64_t c1 = e ? ptx::pair_f32(ca.z, ca.w) : ptx::pair_f32(ca.x, ca.y);
            const uint64_t s1 = e ? ptx::pair_f32(sb.z, sb.w) : ptx::pair_f32(sb.x, sb.y);
            const uint64_t c2 = e ? ptx::pair_f32(cb.z, cb.w) : ptx::pair_f32(cb.x, cb.y);
            const uint64_t s2 = e ? ptx::pair_f32(sa.z, sa.w) : ptx::pair_f32(sa.x, sa.y);
            const float2 ya = ptx::unpair_f32(ptx::fma2(v, s1, ptx::mul2(u, c1)));
            const float2 yb = ptx::unpair_f32(ptx::fma2(u, s2, ptx::mul2(v, c2)));
            a[i + 2 * e] = ya.x;
            a[i + 2 * e + 1] = ya.y;
            b[i + 2 * e] = yb.x;
            b[i + 2 * e + 1] = yb.y;
          }
        }
      }
      __nv_bfloat16* dst = q + hk * D;
      if (hk >= hk0) {
        if (!store) continue;
        dst = hk < hv0 ? p.kpool + at + ((int64_t)(hk - hk0) << p.page_shift) * D
                       : p.vpool + at + ((int64_t)(hk - hv0) << p.page_shift) * D;
      }
      store_half<E>(dst, a);
      store_half<E>(dst + D / 2, b);
    }
  }
  ptx::wait_dependency();  // (where it was launched beside another: this one ends behind it)
}

// `beside`: beside the launch before it, which makes nothing that this one reads (the kernel ends behind it)
template <typename T, int D>
cudaError_t launch_norm(NormParams& p, int sms, cudaStream_t stream, bool beside = false) {
  constexpr int E = sizeof(T) == 4 ? 4 : 8;
  constexpr int GP = kNormThreads<T, D> / (D / 2 / E);
  const int heads = p.Hq + 2 * p.Hkv;
  // tokens whose heads fill a block's batch; few tokens: a head per lane group, over several blocks
  p.tokens = 1;
  while (p.tokens < kNormMaxTokens && 2 * p.tokens * heads <= kNormBatch * GP) p.tokens *= 2;
  while (p.tokens > 1 && (p.N + p.tokens - 1) / p.tokens < 2 * sms) p.tokens /= 2;
  p.splits = p.N < sms ? (heads + GP - 1) / GP : 1;
  const int64_t blocks = (int64_t)((p.N + p.tokens - 1) / p.tokens) * p.splits;
  if (beside) return launch_early(norm_rope_kernel<T, D>, dim3((unsigned)blocks), dim3(kNormThreads<T, D>), 0, stream, p);
  norm_rope_kernel<T, D><<<(unsigned)blocks, kNormThreads<T, D>, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_queries(const NormParams& all, int dtype, int D, int sms, cudaStream_t stream) {
  NormParams p = all;
  p.Hkv = 0;  // (a row then ends with its queries)
  if (dtype == MK_F32)
    return D == 128 ? launch_norm<float, 128>(p, sms, stream, true) : launch_norm<float, 64>(p, sms, stream, true);
  return D == 128 ? launch_norm<__nv_bfloat16, 128>(p, sms, stream, true)
                  : launch_norm<__nv_bfloat16, 64>(p, sms, stream, true);
}

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
  const size_t smem = (size_t)5 * (B + 1) * 4;
  if (smem > 48 * 1024 - 1024) {
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(plan_kernel, 5 * (kPlanMaxB + 1) * 4, &allowed);
    if (e != cudaSuccess) return launch_result(e, "mk_paged_plan");
  }
  // one CTA does 4096 tokens in one pass of its threads; the sums are the rest of its time, and fewer warps
  // scan and meet sooner where they cover requests and tokens
  int ctas = 1, threads = 128;
  while (threads < kPlanThreads && (B > threads || max_tokens > threads * 4)) threads *= 2;
  while (ctas < kPlanCtas && max_tokens > ctas * kPlanThreads * 4) ctas *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
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
  if (int rc = check_norm("mk_qk_norm_rope", N, Hq, Hkv, D, qkv, qkv_dtype, ld_qkv, q_gamma, k_gamma, eps, rope_theta,
                          positions, slots, q_out, ld_q, kpool, vpool, num_pages, page_size))
    return rc;
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
  rope_frequencies(rope_theta, D, p.freq);
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
