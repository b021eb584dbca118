// Paged attention of few query rows per request and key/value head (a decode
// step's one token of a group of up to eight heads), and the join of partial
// results.
//
// Every key and value is read once for a handful of rows, so HBM bounds it
// and the arithmetic only has to keep out of the way: at the SM's share of
// HBM (about 45 GB/s) 64 KB of keys and values land per SM every 1.5 us.  Each
// warp is a worker of its own, with its own part of the work line, its own
// ring of blocks filled by TMA (pages gathered into a 128-byte-swizzled tile),
// its own softmax state in registers: no warp waits for another.  The products
// run on m16n8k16 warp matrix instructions with the keys (and the columns of
// the values) along their 16 and the query rows along their 8, so a decode
// step's four rows fill half of one; a tcgen05 product has 128 rows, and would
// put two more round trips (through tensor memory) into each block's chain.
// With nine to 32 rows the chunk kernel is faster all the same (four requests
// of 32768 keys: 20 rows 93 us there, 113 us with three eights of rows here;
// 64 requests of 512 to 8192 keys and four rows 199 us there, 178 us here),
// so this one has a single eight.  Four warps with three blocks of 16 KB each:
// 183 us for those 64 requests; six with two 187, twelve with two of 8 KB 189,
// eight with three of 8 KB 193.  Since then 179 (6.5 TB/s at a copy's 6.8),
// with the next item's query rows read ahead and an item's fixed cost in the
// division at 96 keys (256 requests of 500 keys: 71 us with 64 and the rows not
// read ahead, 63 after; with 128 keys 65, with 160 67).
//
//   s = q k^T scale;  m' = max(m, max s);  p = 2^(s - m');
//   l = l 2^(m - m') + sum p;  o = o 2^(m - m') + p v
//
// The probabilities enter the second product as two bf16 parts (p and what
// its rounding leaves), which keeps them to 2^-16; the extra products cost
// nothing here.
#include "paged_attention.cuh"

namespace mk {
namespace {

using namespace ptx;

constexpr int kStages = 3;
static_assert(kMaxFewRows == 8, "the query tile is one eight of rows, a whole swizzle atom");
constexpr int kHalfBytes = kRowBlockBytes / 2;  // keys, or values, of a block
constexpr int kStageBytes = kRowBlockBytes;

template <int D>
constexpr int smem_bytes_rows() {
  return 1024 + kRowWarps * (kStages * kStageBytes + kMaxFewRows * D * 2);
}

// 16-byte chunk c of row r in a tile of 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t swz(uint32_t base, int r, int c) {
  return base + r * 128 + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ bool nonfinite_lo(uint32_t w) { return (w & 0x7F80u) == 0x7F80u; }
__device__ __forceinline__ bool nonfinite_hi(uint32_t w) { return (w & 0x7F800000u) == 0x7F800000u; }

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32, 1)
    rows_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
  constexpr int KU = Geometry<D, false>::kKeys;  // keys per block
  constexpr int NH = D / 64;                     // 128-byte column halves
  constexpr int NK = KU / 16;                    // key tiles of a block
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kRowWarps][kStages];
  __shared__ uint64_t live[kRowWarps][kStages];  // keys of a block that were loaded
  __shared__ Patience patience;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = base + warp * kStages * kStageBytes;
  const uint32_t qs = smem_addr(base + kRowWarps * kStages * kStageBytes + warp * kMaxFewRows * D * 2);
  if (threadIdx.x == 0) {
    patience.gave_up = 0;
    patience.limit = 1;  // (a block's copies)
    for (int i = 0; i < kRowWarps; ++i)
      for (int j = 0; j < kStages; ++j) mbar_init(&full[i][j], 1);
    fence_mbar_init();
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  __syncthreads();
  launch_dependents();
  wait_dependency();

  const int w = warp * gridDim.x + blockIdx.x;  // (few workers are spread over the SMs)
  const Line line = measure_line<D, false>(p, lane);
  if (line.bad && w == 0 && lane == 0) set_status(p.status, MK_DEV_BAD_INDEX);
  const int64_t x0 = line.border(w), x1 = line.border(w + 1);
  Note note = {0, 0, 0, 0};
  if (lane == 0) *note_of(p, D, w) = note;
  if (line.bad || x0 >= x1) return;
  const int pmask = (1 << p.page_shift) - 1;
  const int box = min(KU, pmask + 1);     // keys per TMA box
  const int npg = KU / box;               // pages a block touches

  Cursor<D, false> cons;
  cons.find(p, line, x0, lane);
  Cursor<D, false> prod = cons;
  int pk = 0, pke = 0;        // the producer's next block and the end of its item's part
  bool pdone = false;
  int win_b = -1, win0 = 0, win = -1;  // 32 entries of the block table, one per lane
  uint32_t issued = 0, done = 0;

  // first block and end of a cursor's item in this worker's part
  auto part_of = [&](const Cursor<D, false>& c, int& k0, int& k1) {
    const int nk = c.blocks(p);
    k0 = c.block_at(x0, nk);
    k1 = c.block_at(x1, nk);
  };
  auto next_part = [&](Cursor<D, false>& c, int& k0, int& k1) {
    for (;;) {
      c.next(p);
      if (c.b >= p.B || c.start >= x1) return false;
      part_of(c, k0, k1);
      if (k0 < k1) return true;
    }
  };
  // load the producer's next block into the ring
  auto issue = [&]() {
    if (pdone) return;
    const int st = issued % kStages;
    uint8_t* dst = ring + st * kStageBytes;
    const int key0 = pk * KU, j0 = key0 >> p.page_shift, L = prod.s.ctx + prod.s.n;
    if (prod.b != win_b || j0 < win0 || j0 >= win0 + 32) {
      win_b = prod.b;
      win0 = j0 & ~31;
      const int j = win0 + lane;
      win = (j < p.max_pages && ((int64_t)j << p.page_shift) < L) ? p.table[(size_t)prod.b * p.max_pages + j] : -1;
    }
    uint64_t keys = 0;
#pragma unroll
    for (int h = 0; h < (KU + 31) / 32; ++h) {
      const int key = key0 + h * 32 + lane;
      const int id = __shfl_sync(0xffffffffu, win, ((key >> p.page_shift) - win0) & 31);
      const bool in = key < L && h * 32 + lane < KU, ok = in && (unsigned)id < (unsigned)p.num_pages;
      keys |= (uint64_t)__ballot_sync(0xffffffffu, ok) << (32 * h);
      if (in && !ok) set_status(p.status, MK_DEV_BAD_INDEX);
    }
    // one box per page, column half, and keys or values
    const int pg = lane / (2 * NH), hv = lane % (2 * NH), half = hv % NH, is_v = hv / NH;
    const int id = __shfl_sync(0xffffffffu, win, (j0 + pg - win0) & 31);
    const bool mine = pg < npg && ((keys >> (pg * box)) & 1);
    const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
    if (lane == 0) {
      live[warp][st] = keys;
      mbar_arrive_expect_tx(&full[warp][st], boxes * box * 128);
    }
    __syncwarp();
    if (mine) {
      const int row = ((id * p.Hkv + prod.g) << p.page_shift) + (key0 & pmask);
      tma_load_2d(dst + is_v * kHalfBytes + half * (KU * 128) + pg * box * 128, is_v ? &vmap : &kmap, half * 64, row,
                  &full[warp][st]);
    }
    ++issued;
    if (++pk >= pke) pdone = !next_part(prod, pk, pke);
  };

  int ck = 0, cke = 0;
  part_of(cons, ck, cke);
  if (ck >= cke && !next_part(cons, ck, cke)) return;
  prod = cons;
  pk = ck;
  pke = cke;
#pragma unroll 1
  for (int i = 0; i < kStages; ++i) issue();

  // this lane's place in the 16 x 8 results: keys (columns of the values) g and g + 8, query rows c0, c0 + 1
  const int g = lane >> 2, c0 = (lane & 3) * 2;
  // this lane's pieces of an item's query rows (row r = token * G + head; rows past the last are zero), read while
  // the item before is worked on
  constexpr int QP = kMaxFewRows * (D / 8) / 32;
  uint4 qv[QP];
  auto load_q = [&](const Cursor<D, false>& c) {
    const __nv_bfloat16* qb = p.q + (int64_t)c.s.row0 * p.ld_q + (int64_t)c.g * p.G * D;
    const int nrows = c.s.n * p.G;
#pragma unroll
    for (int j = 0; j < QP; ++j) {
      const int r = (lane + j * 32) / (D / 8), col = (lane + j * 32) % (D / 8) * 8;
      qv[j] = make_uint4(0, 0, 0, 0);
      if (r < nrows) qv[j] = __ldg(reinterpret_cast<const uint4*>(qb + (int64_t)(r / p.G) * p.ld_q + (r % p.G) * D + col));
    }
  };
  load_q(cons);
  for (bool more = true; more;) {
    const int n = cons.s.n, ctx = cons.s.ctx, L = ctx + n, nrows = n * p.G;
    const int nk = cons.blocks(p), kb = ck;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < QP; ++j) {
      const int r = (lane + j * 32) / (D / 8), c = (lane + j * 32) % (D / 8);
      const uint32_t a = swz(qs + (c >> 3) * (kMaxFewRows * 128), r, c & 7);
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(qv[j].x), "r"(qv[j].y), "r"(qv[j].z),
                   "r"(qv[j].w)
                   : "memory");
    }
    __syncwarp();
    Cursor<D, false> coming = cons;
    int nk0 = 0, nk1 = 0;
    more = next_part(coming, nk0, nk1);
    if (more) load_q(coming);
    // the last key each of this lane's two rows sees
    int lim[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) lim[e] = c0 + e < nrows ? ctx + (c0 + e) / p.G : L - 1;
    uint32_t qf[D / 32][4];  // query operands of two 16-column steps each
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk) {
      const int c = kk * 4 + (lane >> 3);
      ldsm4(swz(qs + (c >> 3) * (kMaxFewRows * 128), lane & 7, c & 7), qf[kk]);
    }
    const int slot = 2 * w + (kb == 0 ? 1 : 0);  // of the part's record (free while a whole item is worked on)
    float o[D / 16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][e] = 0.f;

    constexpr int kFold = kFoldKeys / KU;
    float mfold[2] = {-INFINITY, -INFINITY}, lfold[2] = {0.f, 0.f};  // the maxima of folded results, and their sums
#pragma unroll 1
    for (int stop = kb + kFold;; stop += kFold) {
      for (; ck < min(cke, stop); ++ck) {
        const int st = done % kStages;
        if (!wait_phase(&full[warp][st], (done / kStages) & 1, &patience)) {
          if (lane == 0) set_status(p.status, MK_DEV_RING_TIMEOUT);
          // the copies in flight land in this CTA's memory: give them time before it goes
          for (uint32_t d = done; d < issued; ++d)
            for (int i = 0; i < 100000 && !mbar_try_wait(&full[warp][d % kStages], (d / kStages) & 1); ++i) {
            }
          return;
        }
        const uint32_t ks = smem_addr(ring + st * kStageBytes), vs = ks + kHalfBytes;
        const uint64_t keys = live[warp][st];
        const int key0 = ck * KU;
        constexpr uint64_t kAll = KU == 64 ? ~0ull : (1ull << (KU & 63)) - 1;
        const bool masked = keys != kAll || key0 + KU > ctx + 1;

        float s[NK][4];
#pragma unroll
        for (int t = 0; t < NK; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t a[NK][4];  // keys t * 16 .. + 15, columns kk * 16 .. + 15
          const int c = kk * 2 + (lane >> 4);
#pragma unroll
          for (int t = 0; t < NK; ++t) ldsm4(swz(ks + (c >> 3) * (KU * 128), t * 16 + (lane & 15), c & 7), a[t]);
#pragma unroll
          for (int t = 0; t < NK; ++t) mma_bf16(s[t], a[t], qf[kk >> 1][(kk & 1) * 2], qf[kk >> 1][(kk & 1) * 2 + 1]);
        }
        if (masked) {
#pragma unroll
          for (int t = 0; t < NK; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = t * 16 + g + (e >> 1) * 8;
              if (!((keys >> k) & 1) || key0 + k > lim[e & 1]) s[t][e] = -INFINITY;
            }
        }
        bool moved = false;
        float mnew[2], muse[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(s[0][e], s[0][e + 2]);
#pragma unroll
          for (int t = 1; t < NK; ++t) x = fmaxf(x, fmaxf(s[t][e], s[t][e + 2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          mnew[e] = fmaxf(m[e], x * p.scale);
          muse[e] = mnew[e] == -INFINITY ? 0.f : mnew[e];  // a row without any key so far
          moved |= mnew[e] != m[e];
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = ex2(m[e] - muse[e]);
            m[e] = mnew[e];
            l[e] *= f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
              o[t][e] *= f;
              o[t][e + 2] *= f;
            }
          }
        }
#pragma unroll
        for (int t = 0; t < NK; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = ex2(fmaf(s[t][e], p.scale, -muse[e & 1]));
            s[t][e] = x;
            l[e & 1] += x;
          }
        bool bad_v = false;  // a value that is not finite behind a mask
#pragma unroll
        for (int t = 0; t < NK; ++t) {
          // probabilities as operands: 16 keys by 8 rows, transposed, in two parts
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = s[t][2 * e], y = s[t][2 * e + 1];
            const uint32_t h = pack_bf16(x, y);
            hi[e] = movm_trans(h);
            lo[e] = movm_trans(pack_bf16(x - bf_lo(h), y - bf_hi(h)));
          }
          // this lane's four keys of the 16: c0, c0 + 1, c0 + 8, c0 + 9
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          if (masked) {
            const uint32_t k16 = (uint32_t)(keys >> (t * 16)) >> c0;
            keep0 = ((k16 & 1) ? 0xFFFFu : 0u) | ((k16 & 2) ? 0xFFFF0000u : 0u);
            keep1 = ((k16 & 0x100) ? 0xFFFFu : 0u) | ((k16 & 0x200) ? 0xFFFF0000u : 0u);
          }
#pragma unroll
          for (int d = 0; d < D / 16; d += 4) {
            uint32_t a[4][4];  // columns (d + q) * 16 .. + 15 of the values by the 16 keys
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int r = t * 16 + (lane >> 4) * 8 + (lane & 7), c = (d + q) * 2 + ((lane >> 3) & 1);
              ldsm4t(swz(vs + (c >> 3) * (KU * 128), r, c & 7), a[q]);
              if (masked) {
                // values that were not loaded are zero, whatever the memory held
                a[q][0] &= keep0; a[q][1] &= keep0; a[q][2] &= keep1; a[q][3] &= keep1;
                if (n > 1) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    if (nonfinite_lo(a[q][e])) { a[q][e] &= 0xFFFF0000u; bad_v = true; }
                    if (nonfinite_hi(a[q][e])) { a[q][e] &= 0xFFFFu; bad_v = true; }
                  }
                }
              }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) mma_bf16(o[d + q], a[q], hi[0], hi[1]);
#pragma unroll
            for (int q = 0; q < 4; ++q) mma_bf16(o[d + q], a[q], lo[0], lo[1]);
          }
        }
        if (masked && n > 1 && __any_sync(0xffffffffu, bad_v)) {
          // 0 * inf would reach the rows that do not see the key: such values were left
          // out above and go to the rows that see it only
#pragma unroll 1
          for (int k = 0; k < KU; ++k) {
            if (!((keys >> k) & 1)) continue;
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int col = d * 16 + q * 8 + g, c = col >> 3;
                const uint32_t w2 = lds32(swz(vs + (c >> 3) * (KU * 128), k, c & 7) + ((col & 7) >> 1) * 4);
                const uint32_t v = col & 1 ? w2 >> 16 : w2 & 0xFFFFu;
                if ((v & 0x7F80u) != 0x7F80u) continue;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (key0 + k <= lim[e]) o[d][2 * q + e] += bf_lo(v);
              }
          }
        }
        __syncwarp();  // every lane has read the block
        ++done;
        issue();
      }
      if (cke - kb <= kFold) break;
      // a long part: the results so far go to the place of its record, at its end what lies there is added to the rest
      const bool some = stop > kb + kFold, last = ck >= cke;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = c0 + e;
        if (r >= nrows) continue;
        float* dst = part_o(p, D, slot, r) + g;
        const float f = fold_weight(mfold[e], m[e]);
        mfold[e] = m[e];
        lfold[e] = lfold[e] * f + l[e];
        l[e] = last ? lfold[e] : 0.f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float* at = dst + d * 16 + q * 8;
            const float x = o[d][2 * q + e] + (some ? *at * f : 0.f);
            if (!last) *at = x;
            o[d][2 * q + e] = last ? x : 0.f;
          }
      }
      if (last) break;
    }

#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
    }
    const bool whole = kb == 0 && cke == nk;
    if (kb != 0 && cke == nk) note = {cons.first_worker(line), cons.s.row0, cons.g, n};
    __nv_bfloat16* ob = p.out + (int64_t)cons.s.row0 * p.ld_out + (int64_t)cons.g * p.G * D;
    if (whole) {
      const float f0 = l[0] == 0.f ? 0.f : 1.0f / l[0], f1 = l[1] == 0.f ? 0.f : 1.0f / l[1];
      // neighbouring columns sit in lanes g and g ^ 1: even g stores row c0, odd g row c0 + 1
      const int r = c0 + (g & 1);
      __nv_bfloat16* dst = ob + (int64_t)(r / p.G) * p.ld_out + (r % p.G) * D + (g & ~1);
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float x = o[d][2 * q] * f0, y = o[d][2 * q + 1] * f1;  // (a row without keys is zero)
          const float other = __shfl_xor_sync(0xffffffffu, g & 1 ? x : y, 4);
          const uint32_t two = g & 1 ? pack_bf16(other, y) : pack_bf16(x, other);
          if (r < nrows) *reinterpret_cast<uint32_t*>(dst + d * 16 + q * 8) = two;
        }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = c0 + e;
        if (r >= nrows) continue;
        float* dst = part_o(p, D, slot, r) + g;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          dst[d * 16] = o[d][e];
          dst[d * 16 + 8] = o[d][e + 2];
        }
        if (g == 0) *reinterpret_cast<float2*>(part_ml(p, D, slot, r)) = make_float2(m[e], l[e]);
      }
    }
    cons = coming;
    ck = nk0;
    cke = nk1;
  }
  if (lane == 0 && note.tokens) *note_of(p, D, w) = note;
}

// Join of the items that workers' borders cut.  The item that ends in worker
// w's part and began before it is worker w's to note; its partial records are
// the second slot of the worker it began with, then the first slots of the
// workers up to w, in order of keys.  A block looks at the notes of kRowWarps
// workers and deals their items' rows out to its warps; with few rows several
// warps share the records of one and meet in shared memory.  (A block per
// worker spent more on its 608 blocks than on the records: one request of 4096
// keys 14.2 us, 64 of 512 to 8192 keys 175.4; this way 13.2 and 173.8.)
constexpr int kJoinWarps = 16;

__device__ __forceinline__ Note read_note(const AttnParams& p, int D, int w) {
  const int4 n = __ldcg(reinterpret_cast<const int4*>(note_of(p, D, w)));
  return Note{n.x, n.y, n.z, n.w};
}
// the i-th partial record of a noted item
__device__ __forceinline__ int record(const Note& n, int i) { return i == 0 ? 2 * n.first + 1 : 2 * (n.first + i); }

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_rows_kernel(const __grid_constant__ AttnParams p) {
  constexpr int E = D / 32;
  __shared__ float so[kJoinWarps][D], sml[kJoinWarps][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  wait_dependency();
  Note notes[kRowWarps];
#pragma unroll
  for (int k = 0; k < kRowWarps; ++k) notes[k] = read_note(p, D, blockIdx.x + k * gridDim.x);
  int total = 0, most = 0;  // rows of the noted items; records of the longest
#pragma unroll
  for (int k = 0; k < kRowWarps; ++k) {
    if (notes[k].tokens == 0) continue;
    total += notes[k].tokens * p.G;
    most = max(most, (int)(blockIdx.x + k * gridDim.x) - notes[k].first + 1);
  }
  int shares = 1;
  while (shares * 2 * total <= kJoinWarps && shares * 4 < most) shares *= 2;
  const int at_once = kJoinWarps / shares, share = warp % shares;
  for (int r0 = 0; r0 < total; r0 += at_once) {
    // this warp's row: of which item, which token and head
    int row = r0 + warp / shares, w = 0;
    const bool on = row < total;
    Note note = {0, 0, 0, 0};
    bool found = false;
#pragma unroll
    for (int k = 0; k < kRowWarps; ++k) {
      const int rows = notes[k].tokens * p.G;
      if (on && !found) {
        if (row < rows) {
          found = true;
          note = notes[k];
          w = blockIdx.x + k * gridDim.x;
        } else {
          row -= rows;
        }
      }
    }
    const int count = on ? w - note.first + 1 : 0, tok = row / p.G, head = row % p.G;
    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    constexpr int U = 8;  // records in flight
    for (int i0 = share; i0 < count; i0 += U * shares) {
      float2 ml[U];
      float v[U][E];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * shares;
        ml[j] = make_float2(-INFINITY, 0.f);
        if (i < count) {
          const int slot = record(note, i);
          ml[j] = __ldcg(reinterpret_cast<const float2*>(part_ml(p, D, slot, row)));
          const float* src = part_o(p, D, slot, row) + lane * E;
          if constexpr (E == 4) {
            const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
            v[j][0] = t.x; v[j][1] = t.y; v[j][2] = t.z; v[j][3] = t.w;
          } else {
            const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
            v[j][0] = t.x; v[j][1] = t.y;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (ml[j].y == 0.f) continue;  // no key, or no record
        const float mn = fmaxf(m, ml[j].x), mu = mn == -INFINITY ? 0.f : mn;
        const float f0 = ex2(m - mu), f1 = ex2(ml[j].x - mu);
        l = l * f0 + ml[j].y * f1;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f0 + v[j][e] * f1;
        m = mn;
      }
    }
    if (shares > 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
      if (lane == 0) {
        sml[warp][0] = m;
        sml[warp][1] = l;
      }
      __syncthreads();
      if (share == 0) {
        for (int j = 1; j < shares; ++j) {
          const float m1 = sml[warp + j][0], l1 = sml[warp + j][1];
          if (l1 == 0.f) continue;
          const float mn = fmaxf(m, m1), mu = mn == -INFINITY ? 0.f : mn;
          const float f0 = ex2(m - mu), f1 = ex2(m1 - mu);
          l = l * f0 + l1 * f1;
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = o[e] * f0 + so[warp + j][lane * E + e] * f1;
          m = mn;
        }
      }
      __syncthreads();
    }
    if (on && share == 0) {
      const float f = l == 0.f ? 0.f : 1.0f / l;
      __nv_bfloat16* dst = p.out + ((int64_t)note.row0 + tok) * p.ld_out + (int64_t)(note.g * p.G + head) * D + lane * E;
      if constexpr (E == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f));
      else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16(o[0] * f, o[1] * f);
    }
  }
}

// The same of chunks: a thread per row of the item's two tiles, a block per eight columns.
constexpr int kJoinCols = 8;

template <int D>
__global__ void __launch_bounds__(kTileRows) join_chunk_kernel(const __grid_constant__ AttnParams p) {
  launch_dependents();
  wait_dependency();
  const Note note = read_note(p, D, blockIdx.x);
  if (note.tokens == 0) return;
  const int row = threadIdx.x, col0 = blockIdx.y * kJoinCols;
  const int t = (row & 127) / p.G, head = (row & 127) % p.G, tok = (row >> 7) * p.tq + t;
  if (t >= p.tq || tok >= note.tokens) return;
  const int count = blockIdx.x - note.first + 1;
  float m = -INFINITY, l = 0.f, o[kJoinCols];
#pragma unroll
  for (int e = 0; e < kJoinCols; ++e) o[e] = 0.f;
  constexpr int U = 4;  // records in flight
  for (int i0 = 0; i0 < count; i0 += U) {
    float2 ml[U];
    float v[U][kJoinCols];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      ml[j] = make_float2(-INFINITY, 0.f);
      if (i0 + j >= count) continue;
      const int slot = record(note, i0 + j);
      ml[j] = __ldcg(reinterpret_cast<const float2*>(part_ml(p, D, slot, row)));
      const float4* src = part_cols(p, D, slot, row, col0);
#pragma unroll
      for (int e = 0; e < kJoinCols; e += 4) {
        const float4 x = __ldcg(src + e / 4 * kTileRows);
        v[j][e] = x.x; v[j][e + 1] = x.y; v[j][e + 2] = x.z; v[j][e + 3] = x.w;
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (ml[j].y == 0.f) continue;  // no key, or no record
      const float mn = fmaxf(m, ml[j].x), mu = mn == -INFINITY ? 0.f : mn;
      const float f0 = ex2(m - mu), f1 = ex2(ml[j].x - mu);
      l = l * f0 + ml[j].y * f1;
#pragma unroll
      for (int e = 0; e < kJoinCols; ++e) o[e] = o[e] * f0 + v[j][e] * f1;
      m = mn;
    }
  }
  const float f = l == 0.f ? 0.f : 1.0f / l;
  __nv_bfloat16* dst = p.out + ((int64_t)note.row0 + tok) * p.ld_out + (int64_t)(note.g * p.G + head) * D + col0;
#pragma unroll
  for (int e = 0; e < kJoinCols; e += 8)
    *reinterpret_cast<uint4*>(dst + e) =
        make_uint4(pack_bf16(o[e] * f, o[e + 1] * f), pack_bf16(o[e + 2] * f, o[e + 3] * f),
                   pack_bf16(o[e + 4] * f, o[e + 5] * f), pack_bf16(o[e + 6] * f, o[e + 7] * f));
}

}  // namespace

cudaError_t launch_join(const AttnParams& p, int D, bool chunk, cudaStream_t stream) {
  if (p.workers < 2) return cudaSuccess;
  if (chunk)  // a block per worker and eight columns
    return launch_early(D == 128 ? join_chunk_kernel<128> : join_chunk_kernel<64>,
                        dim3((unsigned)p.workers, (unsigned)(D / kJoinCols)), dim3(kTileRows), 0, stream, p);
  return launch_early(D == 128 ? join_rows_kernel<128> : join_rows_kernel<64>, dim3((unsigned)(p.workers / kRowWarps)),
                      dim3(kJoinWarps * 32), 0, stream, p);
}

template <int D>
static cudaError_t launch_rows_d(const AttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 cudaStream_t stream) {
  constexpr int smem = smem_bytes_rows<D>();
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(rows_kernel<D>, smem, &allowed);
  if (e != cudaSuccess) return e;
  return launch_early(rows_kernel<D>, dim3((unsigned)(p.workers / kRowWarps)), dim3(kRowWarps * 32), smem, stream, p,
                      kmap, vmap);
}

cudaError_t launch_rows(const AttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int D,
                        cudaStream_t stream) {
  return D == 128 ? launch_rows_d<128>(p, kmap, vmap, stream) : launch_rows_d<64>(p, kmap, vmap, stream);
}

}  // namespace mk
