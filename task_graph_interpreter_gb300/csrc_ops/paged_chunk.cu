// Paged attention of chunks: prompts, or any request with more query rows
// than the few-rows kernel takes, on the tcgen05 tensor cores.
//
// An item is a pair of 128-row query tiles of one request and key/value
// head; a row is a (token, query head) with the group's heads side by side,
// so one pass over the keys serves the whole group.  One persistent CTA per
// SM walks its part of the work line:
//
//   warps 0-3, 4-7   softmax of tile 0 and tile 1, one row per thread
//   warp 8   copies: query tiles, then key and value blocks of 128 keys, pages
//            gathered by TMA into 128-byte-swizzled tiles, a ring of blocks
//   warps 9, 11   products of tile 0 and of tile 1: S_w = Q_w K^T, O_w += P_w V
//   warp 10  division of the work, one descriptor per part of an item; and the
//            values of blocks that some row does not wholly see: what was not
//            loaded becomes zero and what is not finite is set aside, since
//            0 * NaN would reach rows behind the mask; the rows that do see
//            such a value get it when they store their result
//
// Tensor memory holds S_0, S_1 (128 columns each) and O_0, O_1 (D columns):
// all of it at D = 128, so P (bf16) overwrites S and enters the second
// product from there, and the tiles take turns: while one tile's softmax
// runs, the tensor cores do P V and the next S of the other.  The issue order
// P_w V (block j), S_w (block j + 1) keeps S_w from being overwritten before
// P_w is read, since products execute in order, and makes the barrier of
// S_w (j + 1) cover P_w V (j) too.
//
// What bounds it at D = 128: the products, 1025 cycles per tile and block (16
// instructions of 64 cycles), 2050 for both tiles; an 8192-token prompt of 32
// heads takes 2300 per block and 314 us in all (1.75 PFLOP/s of causal
// arithmetic; 350 us once the card is at its power limit, at 1650 MHz).  A
// tile's chain is S, its softmax (128 powers per row at 4.4 cycles of the SM's
// quarter, the maximum, two transfers: 1250 cycles), P V and the next S; it
// fits beside the other tile's products only because the second product starts
// on half of P and hand-overs are few:
//  - each tile's products have a warp of their own (waits, instructions and
//    commits of a block take one some 1300 cycles), and the two pass a token:
//    instructions of both tiles mixed in the queue finish together, after which
//    both softmaxes run at once with the tensor cores idle (3600 cycles);
//  - two threads per row, which halves a thread's powers, exchange maxima and
//    hold fewer registers: 2900 cycles.
// At D = 64 P V is half the arithmetic in the same time (64-column products
// run at half rate): 786 cycles of products per tile.  Tensor memory has room
// for P beside S there, so the next scores are made while a softmax runs and
// no turns are needed; a block of both tiles takes 2150 cycles (2200 with P
// over S), which the two softmaxes set: 1370 of powers, 650 of loads and
// maxima, waits.  Making their powers take turns changed nothing.
//
// Short parts are bound by what surrounds their blocks: the first scores'
// wait, the last product and the store of the results, the values behind
// masks, and instructions.  Warps of four kinds go through all of their code
// for each part, which is more than the instruction cache keeps: bringing it
// from 109 KB to 66 (loops left rolled, each step written out once) and moving
// registers from the softmaxes to the others, which spilled, took eleven
// requests of 400 new tokens, 64 query heads on 8, from 87 to 75 us, eight
// requests of five tokens from 19 to 15.  Results by way of shared memory and TMA
// (two ring places lent at the end of a part) took 309 us for the long prompt but
// 82 for the eleven requests, for its code.
//
// The running maximum moves only when a block exceeds it by 2^8 (the sums
// have that much room in f32 and the probabilities' relative precision in
// bf16 does not depend on their scale), so O is rarely rescaled; the softmax
// warps do it themselves, before they hand over P.
//
// Probabilities are rounded to bf16 (2^-8 each, in the mean far less in the
// sum), the form the tensor cores multiply with bf16 values; maxima, sums
// and O are f32.
#include "paged_chunk.cuh"

namespace mk {
namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kStages = 5;
// registers: the launch's 3 x 128 threads x 168, moved to the softmax warpgroups
constexpr int kLaunchRegs = 168, kConsumerRegs = 208, kOtherRegs = 88;
static_assert(2 * kConsumerRegs + kOtherRegs <= 3 * kLaunchRegs, "register shares within the launch's");

template <int D>
struct Smem {
  static constexpr int kHalf = 128 * 128;        // 128 rows of 128 bytes
  static constexpr int kTile = kHalf * (D / 64);
  static constexpr int kControl = 1024;          // barriers, descriptors (struct Control)
  static constexpr int kBytes = kControl + 2 * kTile + kStages * kTile;
};
static_assert(Smem<128>::kBytes <= 232448, "227 KB of shared memory per CTA");

struct Control {
  uint64_t kv_full[kStages], kv_empty[kStages], v_raw[kStages], q_full[2], q_empty[2], s_full[2], p_full[2][2],
      o_done[2], s_free[2], turn[2], seg_full[kSegRing], seg_empty[kSegRing], drained[2], m_bar;
  Segment segs[kSegRing];
  int odd[kSegRing];      // a value set aside in this part
  uint32_t missing[8];    // per key block (ring): pages of it that are not in the pool, one bit each
  uint32_t tmem;
  Patience patience;
};
static_assert(sizeof(Control) <= Smem<128>::kControl, "control block");

__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs)); }
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs)); }

// Zero the rows of a value block from `valid` on and those of missing pages,
// and let the tensor cores see it.  A whole warp.
template <int D>
__device__ __forceinline__ void zero_values(uint32_t v0, int valid, uint32_t miss, int page_shift, int lane) {
  for (int key = (miss ? 0 : valid & ~3) + (lane >> 3); key < 128; key += 4) {
    if (key < valid && !((miss >> (key >> page_shift)) & 1)) continue;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v0 + h * Smem<D>::kHalf + key * 128 + (lane & 7) * 16),
                   "r"(0)
                   : "memory");
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Bits of a bf16 pair that belong to a value that is not finite.
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) { return __vcmpeq2(w & 0x7F807F80u, 0x7F807F80u); }

// For 32 columns of a row's result, the sum of the values that are not finite, of the
// keys it sees that other rows of the item do not (they were set aside).
__device__ __noinline__ void add_odd_values(const AttnParams& p, const Segment& s, int lim, int D, int c, float* add) {
  const int pmask = (1 << p.page_shift) - 1;
  for (int key = max(s.k0 * 128, masked_from(s)); key <= min(lim, s.k1 * 128 - 1); ++key) {
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

// Every kFold blocks of a part a row's results go from tensor memory to the place of the part's record (where the
// part is a whole item, to the worker's second, which is still free), and at the part's end what lies there is added
// to the rest (`last`); so does its sum of probabilities, l, whose new value is returned.  `m` is the row's maximum
// now, `some` whether results lie there already.  A whole warp, out of line: few parts are so long, and inside the loop over the blocks this cost 3 % of the long prompt's time, folding or
// not (314 us to 323; this way 313, seven chunks of 64-wide heads 40.0 to 40.3).
constexpr int kFold = kFoldKeys / 128;
__device__ __noinline__ float fold_results(const AttnParams& p, int D, int slot, int row, uint32_t to, float m, float l,
                                           bool mine, bool some, bool last) {
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
        x = make_float4(o[e] + x.x * f, o[e + 1] + x.y * f, o[e + 2] + x.z * f, o[e + 3] + x.w * f);
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap qmap,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = Smem<D>;
  constexpr int NH = D / 64;
  // tensor memory columns of S_0, S_1, of O_0, O_1, and of P_0, P_1: over the scores at D = 128, apart at D = 64
  constexpr bool kApart = D == 64;
  constexpr uint32_t kSCol = 0, kOCol = 256, kPCol = kApart ? 384 : 0, kPStep = kApart ? 64 : 128;
  // no static shared memory: the dynamic part starts 1024-byte aligned, as the swizzled tiles need
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Control& ctl = *reinterpret_cast<Control*>(smem_raw);
  auto &kv_full = ctl.kv_full, &kv_empty = ctl.kv_empty, &v_raw = ctl.v_raw;
  auto &q_full = ctl.q_full, &q_empty = ctl.q_empty, &s_full = ctl.s_full, &o_done = ctl.o_done,
       &turn = ctl.turn, &drained = ctl.drained, &s_free = ctl.s_free;
  auto &seg_full = ctl.seg_full, &seg_empty = ctl.seg_empty;
  auto& p_full = ctl.p_full;  // [tile][half of the scores handed over]
  auto& m_bar = ctl.m_bar;
  auto& segs = ctl.segs;
  auto& odd = ctl.odd;
  auto& missing = ctl.missing;
  auto& patience = ctl.patience;
  uint8_t* qt = smem_raw + S::kControl;  // [2][NH][128 rows][128 B]
  uint8_t* ring = qt + 2 * S::kTile;     // [kStages][NH][128 keys][128 B]
  // (broadcast, so that the compiler knows a warp's role and what follows from it uniform)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (smem_addr(smem_raw) & 1023u) {
    if (threadIdx.x == 0) set_status(p.status, MK_DEV_RING_TIMEOUT);
    return;
  }
  if (threadIdx.x == 0) {
    patience.gave_up = 0;
    patience.limit = p.wait_limit;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 2);
      mbar_init(&v_raw[i], 1);
    }
    mbar_init(&m_bar, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&drained[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i][0], 4);
      mbar_init(&p_full[i][1], 4);
      mbar_init(&turn[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], kThreads / 32);
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

  if (warp >= 8) {
    reg_dec();
    if (warp == 10) {
      // ------------------------------------------------ division of the work; values behind masks
      const Line line = measure_line<D, true>(p, lane);
      if (line.bad && blockIdx.x == 0 && lane == 0) set_status(p.status, MK_DEV_BAD_INDEX);
      const int64_t x0 = line.border(blockIdx.x), x1 = line.border(blockIdx.x + 1);
      if (lane == 0) *note_of(p, D, blockIdx.x) = Note{0, 0, 0, 0};
      Cursor<D, true> c;
      bool more = !line.bad && x0 < x1, told = false, begun = false;
      if (more) c.find(p, line, x0, lane);
      uint32_t made = 0;
      const uint32_t r0 = smem_addr(ring);
      uint32_t it = 0, blk = 0, raw_phase = 0;
      bool ok = true;
      // one part is made known ahead of the one whose values are looked after
      for (uint32_t i = 0;; ++i) {
        if (!told) {
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
          if (!wait_phase(&seg_empty[st], ((made / kSegRing) & 1) ^ 1, &patience)) break;
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
              s.slot = k0 == 0 && k1 == nk ? -1 : 2 * (int)blockIdx.x + (k0 == 0 ? 1 : 0);
              if (k0 != 0 && k1 == nk)
                *note_of(p, D, blockIdx.x) = Note{c.first_worker(line), s.row0, c.g, min(2 * p.tq, c.s.n - t0)};
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const int first = t0 + w * p.tq, last = min(first + p.tq, c.s.n) - 1;
                s.end[w] = first < c.s.n ? max(k0, min(k1, (c.s.ctx + last) / 128 + 1)) : k0;
              }
            }
            odd[st] = 0;
            mbar_arrive(&seg_full[st]);
          }
          __syncwarp();
          ++made;
          told = !more;
        }
        if (i < 1) continue;
        const int sst = (i - 1) % kSegRing;
        if (!segs[sst].valid) break;
        const int k0 = segs[sst].k0, k1 = segs[sst].k1, from = masked_from(segs[sst]), to = masked_to(segs[sst], p);
        for (int k = max(k0, from >> 7); k < k1; ++k) {
          const uint32_t vit = it + 2 * (k - k0) + 1;
          const int st = vit % kStages;
          if (!(ok = wait_phase(&v_raw[st], (raw_phase >> st) & 1, &patience))) break;
          raw_phase ^= 1u << st;
          const uint32_t v0 = r0 + st * S::kTile;
          const int first = max(0, from - k * 128), valid = min(128, to - k * 128);
          const uint32_t miss = missing[(blk + k - k0) & 7];
          if (valid < 128 || miss) zero_values<D>(v0, valid, miss, p.page_shift, lane);
          // 0 * v summed over the block is zero unless some v is not finite: one packed instruction per pair
          __nv_bfloat162 acc[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q] = __float2bfloat162_rn(0.f);
          const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
#pragma unroll 4
          for (int e = first * 8 + lane; e < valid * 8; e += 32) {
#pragma unroll
            for (int h = 0; h < NH; ++h) {
              const uint4 v = lds128(v0 + h * S::kHalf + e * 16);
              const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) acc[q] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u[q]), zero, acc[q]);
            }
          }
          const __nv_bfloat162 sum = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
          const bool any = __hisnan(__low2bfloat16(sum)) || __hisnan(__high2bfloat16(sum));
          if (__any_sync(0xffffffffu, any)) {
            for (int e = first * 32 + lane; e < valid * 32; e += 32) {
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
        if (!ok) break;
        it += 2 * (k1 - k0);
        blk += k1 - k0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[sst]);
      }
    } else if (warp == 8) {
      // ------------------------------------------------ copies
      const int box = min(128, pmask + 1), npg = 128 / box;
      uint32_t it = 0, nb = 0, nq = 0;  // places of the ring; blocks; query tile pairs
      uint32_t raw_at = 0, raw_phase = 0, misses = 0, hole = 0;  // stages last filled through v_raw, and its phases; uses of m_bar
      const auto load_q = [&](const Segment& s) {
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          if (!wait_phase(&q_empty[w], (nq & 1) ^ 1, &patience)) return false;
          if (lane == 0) {
            // (a second tile without tokens is not read)
            const bool some = w == 0 || s.t0 + p.tq < s.n;
            mbar_arrive_expect_tx(&q_full[w], some ? NH * p.tq * p.G * 128 : 0);
            for (int h = 0; h < NH && some; ++h)
              tma_load_3d(qt + w * S::kTile + h * S::kHalf, &qmap, h * 64, s.g * p.G, s.row0 + w * p.tq, &q_full[w]);
          }
          __syncwarp();
        }
        ++nq;
        return true;
      };
      for (uint32_t i = 0;; ++i) {
        const int sst = i % kSegRing;
        if (!wait_phase(&seg_full[sst], (i / kSegRing) & 1, &patience)) break;
        const Segment s = segs[sst];
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[sst]);
        if (!s.valid) break;
        const int L = masked_to(s, p), jd = masked_from(s) >> 7;
        // the query tiles, behind the first keys and values where the last item's products still read theirs
        const bool early = __all_sync(0xffffffffu, mbar_test_wait(&q_empty[0], (nq & 1) ^ 1) &&
                                                       mbar_test_wait(&q_empty[1], (nq & 1) ^ 1));
        bool ok = !early || load_q(s);
        // lane = page * NH + column half; table entries are read a block ahead
        const int pg = lane / NH, half = lane % NH;
        const int32_t* table = p.table + (size_t)s.b * p.max_pages;
        const auto entry = [&](int key) { return pg < npg && key < L ? table[key >> p.page_shift] : -1; };
        int next_id = entry(s.k0 * 128 + pg * box);
        for (int k = s.k0; k < s.k1 && ok; ++k) {
          const int key = k * 128 + pg * box, id = next_id;
          next_id = k + 1 < s.k1 ? entry(key + 128) : -1;  // (no key past the last block: it could pass 2^31)
          const bool in = pg < npg && key < L;
          const bool good = in && (unsigned)id < (unsigned)p.num_pages;
          if (in && !good) set_status(p.status, MK_DEV_BAD_INDEX);
          const unsigned lanes = __ballot_sync(0xffffffffu, good);
          unsigned miss = __ballot_sync(0xffffffffu, in && !good && half == 0);
          if (NH == 2 && miss) {  // one bit per page
            unsigned m2 = 0;
            for (int j = 0; j < npg; ++j) m2 |= ((miss >> (2 * j)) & 1) << j;
            miss = m2;
          }
          const int row = ((id * p.Hkv + s.g) << p.page_shift) + (key & pmask);
#pragma unroll 1
          for (int v = 0; v < 2; ++v, ++it) {
            const int st = it % kStages;
            if (!(ok = wait_phase(&kv_empty[st], ((it / kStages) & 1) ^ 1, &patience))) break;
            // values of a masked block go by warp 10, which passes them on as full; those of other
            // blocks with a missing page by this warp
            const bool raw = v == 1 && k >= jd, holes = v == 1 && k < jd && miss;
            uint64_t* bar = raw ? &v_raw[st] : holes ? &m_bar : &kv_full[st];
            raw_at = raw ? raw_at | 1u << st : raw_at & ~(1u << st);
            raw_phase ^= raw ? 1u << st : 0u;
            if (lane == 0) {
              if (v == 0) missing[nb & 7] = miss;
              mbar_arrive_expect_tx(bar, __popc(lanes) * box * 128);
            }
            __syncwarp();
            if (good)
              tma_load_2d(ring + st * S::kTile + half * S::kHalf + pg * box * 128, v ? &vmap : &kmap, half * 64, row,
                          bar);
            if (holes) {
              hole = 1;
              if (!(ok = wait_phase(&m_bar, misses & 1, &patience))) break;
              ++misses;
              hole = 0;
              zero_values<D>(smem_addr(ring) + st * S::kTile, 128, miss, p.page_shift, lane);
              if (lane == 0) mbar_arrive(&kv_full[st]);
            }
            __syncwarp();
          }
          ++nb;
          if (ok && k == s.k0 && !early) ok = load_q(s);
        }
        if (!ok) break;
      }
      if (*(volatile int*)&patience.gave_up) {
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
        for (int j = 0; hole && j < 100000 && !mbar_try_wait(&m_bar, misses & 1); ++j) {
        }
        for (int w = 0; w < 2 && nq; ++w)
          for (int j = 0; j < 100000 && !mbar_try_wait(&q_full[w], (nq - 1) & 1); ++j) {
          }
      }
    } else {
      // ------------------------------------------------ products of tile w
      // Whatever steers this loop or makes up a descriptor is a vote's or a broadcast's result: the compiler
      // then knows it uniform and keeps the descriptors in uniform registers (otherwise each instruction
      // took 70 to 100 cycles to issue, the tensor cores 64 to execute).
      const int w = warp == 9 ? 0 : 1;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_phase(bar, parity, &patience)) != 0;
      };
      const uint32_t idesc_s = idesc_bf16_f32(128, 128);
      const uint32_t idesc_o = idesc_bf16_f32(128, D) | kIdescBMnMajor;
      const uint32_t r0 = smem_addr(ring);
      // low words of the operands' descriptors; a 16-element step along a 128-byte row adds 32
      // bytes, 16 value rows 2048, a stage its size
      const uint64_t qd = smem_desc_sw128(smem_addr(qt) + w * S::kTile, 1024u), kd = smem_desc_sw128(r0, 1024u),
                     vd = smem_desc_sw128_mn(r0, S::kHalf, 1024u);
      const uint32_t khi = (uint32_t)(kd >> 32), vhi = (uint32_t)(vd >> 32);
      const uint32_t ts = tmem + kSCol + w * 128, to = tmem + kOCol + w * D, tp = tmem + kPCol + w * kPStep;
      const uint32_t a_lo = (uint32_t)qd;
      uint32_t it = 0, np = 0, nturn = 0;  // places of the ring; P handed over; turns taken (scores made, at D = 64)
      bool ok = true;
      for (uint32_t i = 0; ok; ++i) {
        const int sst = i % kSegRing;
        if (!(ok = wait(&seg_full[sst], (i / kSegRing) & 1))) break;
        const int valid = __shfl_sync(0xffffffffu, segs[sst].valid, 0), k0 = segs[sst].k0;
        const int nt = __shfl_sync(0xffffffffu, segs[sst].k1 - k0, 0);
        const int ntw = __shfl_sync(0xffffffffu, segs[sst].end[w] - k0, 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[sst]);
        if (!valid) break;
        if (!(ok = wait(&q_full[w], i & 1))) break;
        if (ntw == 0 && lane == 0) mbar_arrive(&q_empty[w]);
        // P V of block j out of ring place vst; as soon as half of P is there
        const auto values = [&](int j, uint32_t vst) {
          const uint32_t b_lo = (uint32_t)vd + vst * (S::kTile >> 4);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (c == 1) {
              if (!wait(&p_full[w][1], np & 1)) return false;
              tc_fence_after();
            }
            if (elect_one()) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int kk = c * 4 + e;  // 16 keys
                tc_mma_bf16_ts_lo(to, tp + kk * 8, b_lo + kk * 128, vhi, idesc_o, kk != 0 ? 1u : j != 0 ? 1u : 0u);
              }
              if (c == 1) {
                tc_commit(&kv_empty[vst]);
                if (kApart || j + 1 == ntw) tc_commit(&o_done[w]);
              }
            }
            __syncwarp();
          }
          ++np;
          return true;
        };
        // S of block j out of ring place kst
        const auto scores = [&](int j, uint32_t kst) {
          const uint32_t b_lo = (uint32_t)kd + kst * (S::kTile >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              tc_mma_bf16_lo(ts, a_lo + (kk >> 2) * (S::kHalf >> 4) + (kk & 3) * 2, khi,
                             b_lo + (kk >> 2) * (S::kHalf >> 4) + (kk & 3) * 2, khi, idesc_s, kk != 0 ? 1u : 0u);
              // the other tile's warp takes a while to see its turn
              if (!kApart && kk == D / 32 - 1) mbar_arrive(&turn[w ^ 1]);
            }
            tc_commit(&s_full[w]);
            tc_commit(&kv_empty[kst]);
            if (j + 1 == ntw) tc_commit(&q_empty[w]);
          }
          __syncwarp();
        };
        if constexpr (kApart) {
          // S (block j + 1) as soon as the softmax has S (block j) in registers, P V (block j) as P comes
          for (int j = -1; j < nt; ++j) {
            if (j + 1 < nt) {
              const uint32_t at = it + 2 * (j + 1), kst = at % kStages;
              if (!(ok = wait(&kv_full[kst], (at / kStages) & 1))) break;
              if (j + 1 < ntw) {
                if (!(ok = wait(&s_free[w], (nturn & 1) ^ 1))) break;
                ++nturn;
                tc_fence_after();
                scores(j + 1, kst);
              } else if (lane == 0) {
                mbar_arrive(&kv_empty[kst]);
              }
            }
            if (j >= 0) {
              const uint32_t at = it + 2 * j + 1, vst = at % kStages;
              if (!(ok = wait(&kv_full[vst], (at / kStages) & 1))) break;
              if (j < ntw) {
                if (!(ok = wait(&p_full[w][0], np & 1))) break;
                tc_fence_after();
                if (!(ok = values(j, vst))) break;
              } else if (lane == 0) {
                mbar_arrive(&kv_empty[vst]);
              }
            }
            __syncwarp();
          }
          it += 2 * nt;
        } else {
          // blocks in the order of the ring: K 0, V 0, K 1, V 1, ...; P V (block j) before S (block j + 1).  A
          // block that this tile does not need is handed back as it comes
          for (int j = -1; j < nt; ++j) {
            const uint32_t vst = it % kStages;
            if (j >= 0) {
              if (!(ok = wait(&kv_full[vst], (it / kStages) & 1))) break;
              ++it;
            }
            const uint32_t kst = it % kStages;
            if (j + 1 < nt) {
              if (!(ok = wait(&kv_full[kst], (it / kStages) & 1))) break;
              ++it;
            }
            const bool pv = j >= 0 && j < ntw, qk = j + 1 < ntw;
            if (pv && !(ok = wait(&p_full[w][0], np & 1))) break;
            // tile 0 starts; then each block's products of one tile, then of the other
            if (!(ok = wait(&turn[w], (nturn & 1) ^ (w ^ 1)))) break;
            ++nturn;
            tc_fence_after();
            if (pv) {
              if (!(ok = values(j, vst))) break;
            } else if (j >= 0 && lane == 0) {
              mbar_arrive(&kv_empty[vst]);
            }
            if (qk) {
              scores(j + 1, kst);
            } else {
              if (lane == 0) {
                mbar_arrive(&turn[w ^ 1]);
                if (j + 1 < nt) mbar_arrive(&kv_empty[kst]);
              }
              __syncwarp();
            }
          }
        }
      }
      if (*(volatile int*)&patience.gave_up) {
        // products in flight end before the tensor memory is freed
        if (elect_one()) tc_commit(&drained[w]);
        __syncwarp();
        for (int j = 0; j < 100000 && !mbar_try_wait(&drained[w], 0); ++j) {
        }
      }
    }
  } else {
    // -------------------------------------------------- softmax: one row per thread
    reg_inc();
    const int w = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's tensor-memory lanes (lane field, bits 16 up)
    const uint32_t ts = tmem + lanes + kSCol + w * 128, to = tmem + lanes + kOCol + w * D,
                   tp = tmem + lanes + kPCol + w * kPStep;
    const int tok_in = row / p.G, head = row % p.G;
    uint32_t ns = 0, no = 0, blk = 0;
    for (uint32_t i = 0;; ++i) {
      const int sst = i % kSegRing;
      if (!wait_phase(&seg_full[sst], (i / kSegRing) & 1, &patience)) break;
      const Segment& s = segs[sst];
      if (!s.valid) break;
      const int k0 = s.k0, nt = s.end[w] - k0;
      const int tok = s.t0 + w * p.tq + tok_in;  // in the request
      const bool mine = tok_in < p.tq && tok < s.n;
      const int lim = min(s.ctx + tok, s.ctx + s.n - 1);       // the last key this row sees
      const int jm = ((s.ctx + s.t0 + w * p.tq + 1) >> 7) - k0;  // the first block that the tile does not wholly see
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      const int fold_slot = s.slot >= 0 ? s.slot : 2 * (int)blockIdx.x + 1;
#pragma unroll 1
      for (int j = 0, stop = kFold; ok; stop += kFold) {
        for (; j < min(nt, stop); ++j) {
          if (!(ok = wait_phase(&s_full[w], ns & 1, &patience))) break;
          ++ns;
          tc_fence_after();
          const uint32_t miss = missing[(blk + j) & 7];
          if (j >= jm || miss) {
            // scores of keys that the row does not see become -inf where they lie, 32 columns at a time (a loop,
            // for the sake of the code's size)
            const int last = lim - (k0 + j) * 128;
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
          float x[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, x + c * 32);
          tmem_wait_ld();
          if constexpr (kApart) {  // the next scores may come
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free[w]);
          }
          float mx[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) mx[e] = fmaxf(x[e], x[e + 8]);
#pragma unroll
          for (int c = 16; c < 128; c += 16)
#pragma unroll
            for (int e = 0; e < 8; ++e) mx[e] = fmaxf(fmaxf(mx[e], x[c + e]), x[c + 8 + e]);
          const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                  fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * p.scale;
          if (j == 0) {
            m = top;
          } else {
            if constexpr (kApart) {  // the last block's product has read P, and O is whole
              if (!(ok = wait_phase(&o_done[w], no & 1, &patience))) break;
              ++no;
              tc_fence_after();
            }
            const bool far = top > m + 8.f;
            if (__any_sync(0xffffffffu, far)) {
              // (at D = 128 the barrier of this block's S covers every product into O)
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
          const uint64_t scale2 = pair_f32(p.scale, p.scale), mu2 = pair_f32(mu, mu);
          uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 y = unpair_f32(fma2(pair_f32(x[c * 32 + 2 * e], x[c * 32 + 2 * e + 1]), scale2, mu2));
              const float a = ex2(y.x), b = ex2(y.y);
              sum[e & 3] = add2(sum[e & 3], pair_f32(a, b));
              r[e] = pack_bf16(a, b);
            }
            tmem_st16(tp + c * 16, r);
            if (c & 1) {  // half of the keys: the product starts on them
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_full[w][c >> 1]);
            }
          }
          const float2 t = unpair_f32(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
          l += t.x + t.y;
        }
        if (!ok || j >= nt) break;
        // O is whole once the next scores are there (at D = 64, once its last product is done)
        if (!(ok = wait_phase(kApart ? &o_done[w] : &s_full[w], (kApart ? no : ns) & 1, &patience))) break;
        tc_fence_after();
        l = fold_results(p, D, fold_slot, w * 128 + row, to, m, l, mine, stop > kFold, false);
      }
      if (!ok) break;
      blk += s.k1 - k0;
      if (nt > 0) {
        if (!wait_phase(&o_done[w], no & 1, &patience)) break;
        ++no;
        tc_fence_after();
      }
      if (nt > kFold) l = fold_results(p, D, fold_slot, w * 128 + row, to, m, l, mine, true, true);
      const bool set_aside = nt > 0 && odd[sst];
      const float f = s.slot >= 0 ? 1.f : nt == 0 || l == 0.f ? 0.f : 1.0f / l;  // a row without keys is zero
      __nv_bfloat16* dst = p.out + ((int64_t)s.row0 + w * p.tq + tok_in) * p.ld_out + (int64_t)(s.g * p.G + head) * D;
      float4* rec = nullptr;
      if (s.slot >= 0) {
        rec = part_cols(p, D, s.slot, w * 128 + row, 0);
        if (mine) *reinterpret_cast<float2*>(part_ml(p, D, s.slot, w * 128 + row)) = make_float2(m, nt > 0 ? l : 0.f);
      }
      // (32-byte stores where a row allows it: lanes hold different rows, and each store takes a cycle per
      // lane: 16-byte ones took 4000 cycles of a part's end, these 2500)
      const bool wide = (p.ld_out & 15) == 0 && (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
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
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = f == 0.f ? 0.f : o[e] * f;
        if (mine && !rec) {
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
        } else if (mine && nt > 0) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            rec[(c + e) / 4 * kTileRows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      tc_fence_before();  // O is read before the next part's first P is handed over
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[sst]);
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
  static std::atomic<uint64_t> allowed{0};
  static std::atomic<int> regs{0};
  cudaError_t e = allow_smem(chunk_kernel<D>, Smem<D>::kBytes, &allowed);
  if (e != cudaSuccess) return e;
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes a;
    if ((e = cudaFuncGetAttributes(&a, chunk_kernel<D>)) != cudaSuccess) return e;
    regs.store(a.numRegs, std::memory_order_relaxed);
  }
  // the register shares add up to this allocation: with fewer a warpgroup would wait for registers for ever (build.py
  // checks the compiler's count, so that this is met by builds of another kind only)
  if (regs.load(std::memory_order_relaxed) != kLaunchRegs) return cudaErrorInvalidKernelImage;
  return launch_early(chunk_kernel<D>, dim3((unsigned)p.workers), dim3(kThreads), Smem<D>::kBytes, stream, p, qmap, kmap,
                      vmap);
}

}  // namespace

cudaError_t launch_chunk(const AttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, int D, cudaStream_t stream) {
  return D == 128 ? launch_chunk_t<128>(p, qmap, kmap, vmap, stream) : launch_chunk_t<64>(p, qmap, kmap, vmap, stream);
}

}  // namespace mk
