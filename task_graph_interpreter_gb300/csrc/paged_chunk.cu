// Paged attention of chunks: prompts, or any request with more query rows
// than the few-rows kernel takes, on the tcgen05 tensor cores.
//
// An item is a pair of 128-row query tiles of one request and key/value
// head; a row is a (token, query head) with the group's heads side by side,
// so one pass over the keys serves the whole group.  One persistent CTA per
// SM walks its part of the work line:
//
//   warp 8   copies: query tiles, then key and value blocks of 128 keys, pages
//            gathered by TMA into 128-byte-swizzled tiles, a ring of blocks
//   warp 9   products: S_w = Q_w K^T, O_w += P_w V for the tiles w = 0, 1
//   warp 10  division of the work: one descriptor per part of an item
//   warp 11  values of blocks that some row does not wholly see: what was not
//            loaded becomes zero and what is not finite is set aside, since
//            0 * NaN would reach rows behind the mask; the rows that do see
//            such a value get it when they store their result
//   warps 0-3, 4-7   softmax of tile 0 and tile 1, one row per thread
//
// Tensor memory holds S_0, S_1 (128 columns each) and O_0, O_1 (D columns):
// all of it at D = 128, so P (bf16) overwrites S and enters the second
// product from there, and the tiles take turns: while one tile's softmax
// runs, the tensor cores do P V and the next S of the other.  The issue order
// P_w V (block j), S_w (block j + 1) keeps S_w from being overwritten before
// P_w is read, since products execute in order, and makes the barrier of
// S_w (j + 1) cover P_w V (j) too.
//
// The running maximum moves only when a block exceeds it by 2^8 (the sums
// have that much room in f32 and the probabilities' relative precision in
// bf16 does not depend on their scale), so O is rarely rescaled; the softmax
// warps do it themselves, before they hand over P.
//
// Probabilities are rounded to bf16 (2^-9 each, in the mean far less in the
// sum), the form the tensor cores multiply with bf16 values; maxima, sums
// and O are f32.
#include "paged_attention.cuh"

namespace mk {
namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kStages = 5;
constexpr int kSegRing = 4;
// registers: the launch's 3 x 128 threads x 168, moved to the softmax warpgroups
constexpr int kLaunchRegs = 168, kConsumerRegs = 224, kOtherRegs = 56;
static_assert(2 * kConsumerRegs + kOtherRegs <= 3 * kLaunchRegs, "register shares within the launch's");

struct Segment {
  int row0;       // first query row of the item (token index in q)
  int b, g;       // request, key/value head
  int ctx, t0;    // cached tokens; the item's first token in its request
  int n;          // new tokens of the request
  int k0, k1;     // key blocks of this part
  int end[2];     // end of each tile's key blocks, >= k0
  int slot;       // partial record, or -1: the part is the whole item
  int valid;      // 0: no more parts
};

template <int D>
struct Smem {
  static constexpr int kHalf = 128 * 128;        // 128 rows of 128 bytes
  static constexpr int kTile = kHalf * (D / 64);
  static constexpr int kBytes = 1024 + 2 * kTile + kStages * kTile;
};

__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs)); }
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs)); }

// The first key block with a key that the item's first row does not see.
__device__ __forceinline__ int first_masked(const Segment& s) { return (s.ctx + s.t0 + 1) >> 7; }

// Zero the rows of a value block from `valid` on and those of missing pages,
// and let the tensor cores see it.  A whole warp.
template <int D>
__device__ __forceinline__ void zero_values(uint32_t v0, int valid, uint32_t miss, int page_shift, int lane) {
  constexpr int NH = D / 64;
  for (int e = lane; e < 128 * NH * 8; e += 32) {
    const int key = e / (NH * 8), c = e % (NH * 8);
    if (key >= valid || ((miss >> (key >> page_shift)) & 1))
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v0 + (c >> 3) * Smem<D>::kHalf + key * 128 +
                                                                   (c & 7) * 16),
                   "r"(0)
                   : "memory");
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Bits of a bf16 pair that belong to a value that is not finite.
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) { return __vcmpeq2(w & 0x7F807F80u, 0x7F807F80u); }

// For 32 columns of a row's result, the sum of the values that are not finite, of the
// keys it sees in this part's masked blocks (they were set aside).
__device__ __noinline__ void add_odd_values(const AttnParams& p, const Segment& s, int lim, int D, int c, float* add) {
  const int pmask = (1 << p.page_shift) - 1;
  for (int key = max(s.k0, first_masked(s)) * 128; key <= min(lim, s.k1 * 128 - 1); ++key) {
    const int id = p.table[(size_t)s.b * p.max_pages + (key >> p.page_shift)];
    if ((unsigned)id >= (unsigned)p.num_pages) continue;
    const __nv_bfloat16* v =
        p.v + ((((int64_t)id * p.Hkv + s.g) << p.page_shift) + (key & pmask)) * D + c;
    for (int e = 0; e < 32; ++e) {
      const float x = __bfloat162float(v[e]);
      if (!isfinite(x)) add[e] += x;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap qmap,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<D>;
  constexpr int NH = D / 64;
  constexpr uint32_t kSCol = 0, kOCol = 256;  // tensor memory columns of S_0, S_1 and O_0, O_1
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t kv_full[kStages], kv_empty[kStages], q_full, q_empty, s_full[2], p_full[2],
      o_done[2], v_raw[kStages], seg_full[kSegRing], seg_empty[kSegRing], drained;
  __shared__ Segment segs[kSegRing];
  __shared__ int odd[kSegRing];  // a value set aside in this part
  __shared__ uint32_t tmem_s;
  __shared__ int gave_up;
  __shared__ uint32_t missing[8];  // per key block (ring): pages of it that are not in the pool, one bit each
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* qt = base;                  // [2][NH][128 rows][128 B]
  uint8_t* ring = base + 2 * S::kTile;  // [kStages][NH][128 keys][128 B]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    gave_up = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
      mbar_init(&v_raw[i], 1);
    }
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&drained, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 11);  // 8 softmax warps, the copy, product and value warps
    }
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&tmem_s, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();
  const uint32_t tmem = tmem_s;
  const int pmask = (1 << p.page_shift) - 1;

  if (warp >= 8) {
    reg_dec();
    if (warp == 10) {
      // ------------------------------------------------ division of the work
      bool bad;
      const int64_t u = line_length<D, true>(p, lane, &bad);
      if (bad && blockIdx.x == 0 && lane == 0) set_status(p.status, MK_DEV_BAD_INDEX);
      const int64_t x0 = border(u, blockIdx.x, p.workers), x1 = border(u, blockIdx.x + 1, p.workers);
      Cursor<D, true> c;
      bool more = !bad && x0 < x1;
      if (more) c.find(p, x0, lane);
      for (uint32_t i = 0;; ++i) {
        int k0 = 0, k1 = 0, nk = 0;
        while (more) {
          nk = c.blocks(p);
          k0 = c.block_at(x0, nk);
          k1 = c.block_at(x1, nk);
          if (k0 < k1) break;
          c.next(p);
          more = c.b < p.B && c.start < x1;
        }
        const int st = i % kSegRing;
        if (!wait_phase(&seg_empty[st], ((i / kSegRing) & 1) ^ 1, &gave_up)) break;
        if (lane == 0) {
          Segment s;
          s.valid = more ? 1 : 0;
          if (more) {
            s.b = c.b;
            s.g = c.g;
            s.ctx = c.s.ctx;
            s.n = c.s.n;
            s.t0 = c.i * 2 * p.tq;
            s.row0 = p.cu[c.b] + s.t0;
            s.k0 = k0;
            s.k1 = k1;
            s.slot = k0 == 0 && k1 == nk ? -1 : 2 * (int)blockIdx.x + (k0 == 0 ? 1 : 0);
            for (int w = 0; w < 2; ++w) {
              const int first = s.t0 + w * p.tq, last = min(first + p.tq, s.n) - 1;
              s.end[w] = first < s.n ? max(k0, min(k1, (s.ctx + last) / 128 + 1)) : k0;
            }
          }
          segs[st] = s;
          odd[st] = 0;
          mbar_arrive(&seg_full[st]);
        }
        __syncwarp();
        if (!more) break;
        c.next(p);
        more = c.b < p.B && c.start < x1;
      }
    } else if (warp == 8) {
      // ------------------------------------------------ copies
      const int box = min(128, pmask + 1), npg = 128 / box;
      uint32_t it = 0, nq = 0;  // key and value blocks; query tiles
      uint32_t raw_at = 0, raw_phase = 0;  // stages last filled through v_raw, and its phases
      for (uint32_t i = 0;; ++i) {
        const int sst = i % kSegRing;
        if (!wait_phase(&seg_full[sst], (i / kSegRing) & 1, &gave_up)) break;
        const Segment s = segs[sst];
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[sst]);
        if (!s.valid) break;
        if (!wait_phase(&q_empty, (nq & 1) ^ 1, &gave_up)) break;
        ++nq;
        if (lane == 0) {
          const int tiles = s.t0 + p.tq < s.n ? 2 : 1;
          mbar_arrive_expect_tx(&q_full, tiles * NH * p.tq * p.G * 128);
          for (int w = 0; w < tiles; ++w)
            for (int h = 0; h < NH; ++h)
              tma_load_3d(qt + w * S::kTile + h * S::kHalf, &qmap, h * 64, s.g * p.G, s.row0 + w * p.tq, &q_full);
        }
        const int L = s.ctx + s.n, jd = first_masked(s);
        bool ok = true;
        for (int k = s.k0; k < s.k1 && ok; ++k) {
          // lane = page * NH + column half
          const int pg = lane / NH, half = lane % NH, key = k * 128 + pg * box;
          int id = -1;
          const bool in = pg < npg && key < L;
          if (in) id = p.table[(size_t)s.b * p.max_pages + (key >> p.page_shift)];
          const bool good = in && (unsigned)id < (unsigned)p.num_pages;
          if (in && !good) set_status(p.status, MK_DEV_BAD_INDEX);
          const unsigned lanes = __ballot_sync(0xffffffffu, good);
          unsigned miss = __ballot_sync(0xffffffffu, in && !good && half == 0);
          if (NH == 2) {  // one bit per page
            unsigned m2 = 0;
            for (int j = 0; j < npg; ++j) m2 |= ((miss >> (2 * j)) & 1) << j;
            miss = m2;
          }
          const int row = ((id * p.Hkv + s.g) << p.page_shift) + (key & pmask);
          for (int v = 0; v < 2; ++v, ++it) {
            const int st = it % kStages;
            if (!wait_phase(&kv_empty[st], ((it / kStages) & 1) ^ 1, &gave_up)) {
              ok = false;
              break;
            }
            // values of a masked block go by the value warp, which passes them on as full
            const bool raw = v == 1 && k >= jd;
            uint64_t* bar = raw ? &v_raw[st] : &kv_full[st];
            raw_at = raw ? raw_at | 1u << st : raw_at & ~(1u << st);
            raw_phase ^= raw ? 1u << st : 0u;
            if (lane == 0) {
              if (v == 0) missing[(it >> 1) & 7] = miss;
              mbar_arrive_expect_tx(bar, __popc(lanes) * box * 128);
            }
            __syncwarp();
            if (good)
              tma_load_2d(ring + st * S::kTile + half * S::kHalf + pg * box * 128, v ? &vmap : &kmap, half * 64, row,
                          bar);
          }
        }
        if (!ok) break;
      }
      if (*(volatile int*)&gave_up) {
        if (lane == 0) set_status(p.status, MK_DEV_RING_TIMEOUT);
        // copies in flight land before the shared memory goes
        for (uint32_t d = it > kStages ? it - kStages : 0; d < it; ++d) {
          const int st = d % kStages;
          const bool raw = (raw_at >> st) & 1;
          for (int j = 0; j < 100000 && !mbar_try_wait(raw ? &v_raw[st] : &kv_full[st],
                                                       raw ? ((raw_phase >> st) & 1) ^ 1 : (d / kStages) & 1);
               ++j) {
          }
        }
        if (nq)
          for (int j = 0; j < 100000 && !mbar_try_wait(&q_full, (nq - 1) & 1); ++j) {
          }
      }
    } else if (warp == 9) {
      // ------------------------------------------------ products
      const uint32_t idesc_s = idesc_bf16_f32(128, 128);
      const uint32_t idesc_o = idesc_bf16_f32(128, D) | kIdescBMnMajor;
      const uint32_t q0 = smem_addr(qt), r0 = smem_addr(ring);
      uint32_t it = 0, blk = 0, np[2] = {0, 0};
      bool ok = true;
      for (uint32_t i = 0; ok; ++i) {
        const int sst = i % kSegRing;
        if (!(ok = wait_phase(&seg_full[sst], (i / kSegRing) & 1, &gave_up))) break;
        const Segment s = segs[sst];
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[sst]);
        if (!s.valid) break;
        if (!(ok = wait_phase(&q_full, i & 1, &gave_up))) break;
        const int nt = s.k1 - s.k0, jd = first_masked(s);
        const int ntw[2] = {s.end[0] - s.k0, s.end[1] - s.k0};
        auto product_s = [&](int w, uint32_t kit) {
          const uint32_t a0 = q0 + w * S::kTile, b0 = r0 + (kit % kStages) * S::kTile;
          if (lane == 0) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc_mma_bf16(tmem + kSCol + w * 128, smem_desc_sw128(a0 + (kk >> 2) * S::kHalf, 1024u) + (kk & 3) * 2u,
                          smem_desc_sw128(b0 + (kk >> 2) * S::kHalf, 1024u) + (kk & 3) * 2u, idesc_s, kk != 0 ? 1u : 0u);
            tc_commit(&s_full[w]);
          }
          __syncwarp();
        };
        if (!(ok = wait_phase(&kv_full[it % kStages], (it / kStages) & 1, &gave_up))) break;
        tc_fence_after();
        for (int w = 0; w < 2; ++w)
          if (ntw[w] > 0) product_s(w, it);
        if (lane == 0) {
          tc_commit(&kv_empty[it % kStages]);
          if (nt == 1) tc_commit(&q_empty);
        }
        for (int j = 0; j < nt && ok; ++j) {
          const uint32_t vit = it + 2 * j + 1, kit = it + 2 * j + 2;
          bool have_v = false, have_k = false;
          for (int w = 0; w < 2 && ok; ++w) {
            if (j >= ntw[w]) continue;
            if (!have_v) {
              if (!(ok = wait_phase(&kv_full[vit % kStages], (vit / kStages) & 1, &gave_up))) break;
              have_v = true;
              // (in masked blocks the value warp has seen to missing pages)
              const uint32_t miss = s.k0 + j < jd ? missing[(blk + j) & 7] : 0u;
              if (miss) zero_values<D>(r0 + (vit % kStages) * S::kTile, 128, miss, p.page_shift, lane);
            }
            if (!(ok = wait_phase(&p_full[w], np[w] & 1, &gave_up))) break;
            ++np[w];
            tc_fence_after();
            if (lane == 0) {
              const uint32_t v0 = r0 + (vit % kStages) * S::kTile;
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc_mma_bf16_ts(tmem + kOCol + w * D, tmem + kSCol + w * 128 + kk * 8,
                               smem_desc_sw128_mn(v0 + kk * 2048u, S::kHalf, 1024u), idesc_o, (j | kk) != 0 ? 1u : 0u);
            }
            __syncwarp();
            if (j + 1 < ntw[w]) {
              if (!have_k) {
                if (!(ok = wait_phase(&kv_full[kit % kStages], (kit / kStages) & 1, &gave_up))) break;
                have_k = true;
                tc_fence_after();
              }
              product_s(w, kit);
            } else if (lane == 0) {
              tc_commit(&o_done[w]);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (lane == 0) {
            tc_commit(&kv_empty[vit % kStages]);
            if (j + 1 < nt) tc_commit(&kv_empty[kit % kStages]);
            if (j + 2 == nt) tc_commit(&q_empty);
          }
          __syncwarp();
        }
        it += 2 * nt;
        blk += nt;
      }
      if (*(volatile int*)&gave_up) {
        // products in flight end before the tensor memory is freed
        if (lane == 0) tc_commit(&drained);
        for (int j = 0; j < 100000 && !mbar_try_wait(&drained, 0); ++j) {
        }
      }
    } else {
      // ------------------------------------------------ values behind masks
      const uint32_t r0 = smem_addr(ring);
      uint32_t it = 0, blk = 0, raw_phase = 0;
      bool ok = true;
      for (uint32_t i = 0; ok; ++i) {
        const int sst = i % kSegRing;
        if (!wait_phase(&seg_full[sst], (i / kSegRing) & 1, &gave_up)) break;
        const Segment s = segs[sst];
        if (!s.valid) break;
        for (int k = max(s.k0, first_masked(s)); k < s.k1; ++k) {
          const uint32_t vit = it + 2 * (k - s.k0) + 1;
          const int st = vit % kStages;
          if (!(ok = wait_phase(&v_raw[st], (raw_phase >> st) & 1, &gave_up))) break;
          raw_phase ^= 1u << st;
          const uint32_t v0 = r0 + st * S::kTile;
          const int valid = min(128, s.ctx + s.n - k * 128);
          const uint32_t miss = missing[(blk + k - s.k0) & 7];
          if (valid < 128 || miss) zero_values<D>(v0, valid, miss, p.page_shift, lane);
          uint32_t any = 0;
#pragma unroll 4
          for (int e = lane; e < valid * 8; e += 32) {
#pragma unroll
            for (int h = 0; h < NH; ++h) {
              const uint4 v = lds128(v0 + h * S::kHalf + e * 16);
              any |= odd_bits(v.x) | odd_bits(v.y) | odd_bits(v.z) | odd_bits(v.w);
            }
          }
          if (__any_sync(0xffffffffu, any != 0)) {
            for (int e = lane; e < valid * 32; e += 32) {
              for (int h = 0; h < NH; ++h) {
                const uint32_t a = v0 + h * S::kHalf + e * 4, v = lds32(a), o = odd_bits(v);
                if (o) sts32(a, v & ~o);
              }
            }
            if (lane == 0) odd[sst] = 1;
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&kv_full[st]);
          __syncwarp();
        }
        it += 2 * (s.k1 - s.k0);
        blk += s.k1 - s.k0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[sst]);
      }
    }
  } else {
    // -------------------------------------------------- softmax: one row per thread
    reg_inc();
    const int w = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's tensor-memory lanes (lane field, bits 16 up)
    const uint32_t ts = tmem + lanes + kSCol + w * 128, to = tmem + lanes + kOCol + w * D;
    const int tok_in = row / p.G, head = row % p.G;
    uint32_t ns = 0, no = 0, blk = 0;
    for (uint32_t i = 0;; ++i) {
      const int sst = i % kSegRing;
      if (!wait_phase(&seg_full[sst], (i / kSegRing) & 1, &gave_up)) break;
      const Segment s = segs[sst];
      if (!s.valid) break;
      const int tok = s.t0 + w * p.tq + tok_in;  // in the request
      const bool mine = tok_in < p.tq && tok < s.n;
      const int lim = min(s.ctx + tok, s.ctx + s.n - 1);  // the last key this row sees
      const int lim0 = s.ctx + s.t0 + w * p.tq;           // ... and the tile's first row
      const int nt = s.end[w] - s.k0;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < nt; ++j) {
        if (!(ok = wait_phase(&s_full[w], ns & 1, &gave_up))) break;
        ++ns;
        tc_fence_after();
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, x + c * 32);
        tmem_wait_ld();
        const int key0 = (s.k0 + j) * 128;
        const uint32_t miss = missing[(blk + j) & 7];
        if (key0 + 127 > lim0 || miss) {
          const int last = lim - key0;
          if (miss) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if ((miss >> (c >> p.page_shift)) & 1) x[c] = -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > last) x[c] = -INFINITY;
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < 128; c += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = c + 4 + e < 128 ? fmaxf(fmaxf(mx[e], x[c + e]), x[c + 4 + e]) : fmaxf(mx[e], x[c + e]);
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale;
        if (j == 0) {
          m = top;
        } else {
          const bool far = top > m + 8.f;
          if (__any_sync(0xffffffffu, far)) {
            // every product into O is complete: the barrier of this block's S covers them
            const float f = far ? ex2(m - top) : 1.f;
            if (far) m = top;
            l *= f;
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
        }
        const float mu = m == -INFINITY ? 0.f : -m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float a = ex2(fmaf(x[c * 32 + 2 * e], p.scale, mu)), b = ex2(fmaf(x[c * 32 + 2 * e + 1], p.scale, mu));
            sum[(2 * e) & 3] += a;
            sum[(2 * e + 1) & 3] += b;
            r[e] = pack_bf16(a, b);
          }
          tmem_st16(ts + c * 16, r);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      if (!ok) break;
      blk += s.k1 - s.k0;
      if (nt > 0) {
        if (!wait_phase(&o_done[w], no & 1, &gave_up)) break;
        ++no;
        tc_fence_after();
      }
      const bool set_aside = nt > 0 && odd[sst];
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[sst]);
      const float f = l == 0.f ? 0.f : 1.0f / l;  // a row without keys is zero
      const int64_t token = (int64_t)s.row0 + w * p.tq + tok_in;
      if (s.slot < 0) {
        __nv_bfloat16* dst = p.out + token * p.ld_out + (int64_t)(s.g * p.G + head) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          if (nt > 0) {
            tmem_ld32(to + c, o);
            tmem_wait_ld();
          }
          if (set_aside && mine) {
            float add[32] = {};
            add_odd_values(p, s, lim, D, c, add);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] += add[e];
          }
          if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (nt > 0 && l != 0.f)
                v = make_uint4(pack_bf16(o[e] * f, o[e + 1] * f), pack_bf16(o[e + 2] * f, o[e + 3] * f),
                               pack_bf16(o[e + 4] * f, o[e + 5] * f), pack_bf16(o[e + 6] * f, o[e + 7] * f));
              *reinterpret_cast<uint4*>(dst + c + e) = v;
            }
          }
        }
      } else if (p.part) {
        const int rec = w * 128 + row;
        if (mine) *reinterpret_cast<float2*>(part_ml(p, D, s.slot, rec)) = make_float2(m, l);
        if (nt > 0) {
          float* dst = part_o(p, D, s.slot, rec);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(to + c, o);
            tmem_wait_ld();
            if (set_aside && mine) {
              float add[32] = {};
              add_odd_values(p, s, lim, D, c, add);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] += add[e];
            }
            if (mine) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(dst + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
        }
      }
      tc_fence_before();  // O is read before the next part's first P is handed over
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_chunk_t(const AttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes a;
  if ((e = cudaFuncGetAttributes(&a, chunk_kernel<D>)) != cudaSuccess) return e;
  // the register shares add up to this allocation: with fewer a warpgroup would wait for registers for ever
  if (a.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
  chunk_kernel<D><<<(unsigned)p.workers, kThreads, Smem<D>::kBytes, stream>>>(p, qmap, kmap, vmap);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk(const AttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, int D, cudaStream_t stream) {
  return D == 128 ? launch_chunk_t<128>(p, qmap, kmap, vmap, stream) : launch_chunk_t<64>(p, qmap, kmap, vmap, stream);
}

}  // namespace mk
