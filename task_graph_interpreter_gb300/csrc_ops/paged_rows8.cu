// Paged attention of few query rows over e4m3 pages: the division of the work,
// the rings of blocks and the join are those of bf16 pages (paged_rows.cu).
//
// HBM bounds it, and half the bytes arrive per key, so the arithmetic has half
// the time per key.  Codes become f16 in registers, which is exact, and the
// products are m16n8k16 of f16 with f32 sums:
//
//   queries   bf16 to f16 after a power of two per row that brings the row's
//             largest to [2^14, 2^15): exact but for elements 2^-28 below it
//   keys      four neighbouring codes of a row are one 32-bit piece of a
//             16-byte ldmatrix row; the order of a head's elements within the
//             product is free, so both pairs of the piece are used where they
//             lie, and the query's operand is read in the same order
//   values    a transposed ldmatrix of 16-bit units gives code pairs of two
//             columns for two keys; one byte permutation sorts them by column
//   scales    of keys: one factor per 16 keys (a page has at least 16), with
//             the row's and the softmax scale; of values: onto the
//             probabilities, relative to the power of two of the largest scale
//             so far, which the results carry (a tile more than 2^kFar below it is
//             added to results in a smaller unit, or its probabilities would
//             leave f16: a page that some rows do not see, or that has no
//             weight, takes nothing from the others)
//
// Probabilities are kept times 2^14, and rounded to f16 (2^-11) once the
// scale of the values is on them; what they are summed to is not rounded.  (Two
// parts, as over bf16 pages, would keep what codes of four bits do not have.)
//
// Eight warps of 8 KB blocks, three in flight: 64 requests of 512 to 8192 keys
// and four rows 101.5 us (5.7 TB/s; bf16 pages 178), four warps of 16 KB 126, for
// a block's chain of products, softmax and products has half the time that it
// has over bf16 pages; heads of 64 58 and 80.  What is left there is that chain
// and the join.  One request of 4096 keys 13.4 us: two launches and eight
// dependent round trips.  Up to two eights of rows run here (four requests of
// 32768 keys and 12 rows 66 us); with three eights registers leave no room.
#include <type_traits>

#include "paged_attention.cuh"

namespace mk {
namespace {

using namespace ptx;

constexpr float kBias = 14.f;                // probabilities are kept times 2^kBias
// A tile whose scale is more than 2^kFar below the unit is added apart: nearer ones keep 2^-11 of probabilities down to
// 2^-22, and 2^-33.  (4, 6 and 15 take the same time where pages' scales are some powers of two apart.)
constexpr int kFar = 6;
// The results' unit goes down by 2^kMostDown at most: they are under 2^41 in it (kFoldKeys keys of at most 2 * 448 times
// 2^kBias).
constexpr int kMostDown = 60;
constexpr int kStages8 = 3;
constexpr int kSmemBytes8 = 1024 + kRowWarps8 * kStages8 * kRowBlockBytes8;
static_assert(kSmemBytes8 <= 229376, "shared memory of a CTA, beside the static part");

// 16-byte chunk c of row r in a tile of D-byte rows: 128-byte or 64-byte swizzle
template <int D>
__device__ __forceinline__ uint32_t swz8(uint32_t base, int r, int c) {
  return base + r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4);
}

// Codes of four that are NaN, as bytes of ones.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

// 2^(d) for d <= 0 (zero where it is not a normal number)
__device__ __forceinline__ float exp2_down(int d) { return d < -126 ? 0.f : __uint_as_float((uint32_t)(127 + d) << 23); }

__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23 & 0xFF); }

template <int NR, int N>
__device__ __forceinline__ void times(float (&o)[NR][N][4], float f) {
#pragma unroll
  for (int h = 0; h < NR; ++h)
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[h][t][e] *= f;
}

// NR: eights of query rows
template <int D, int NR>
__global__ void __launch_bounds__(kRowWarps8 * 32, 1)
    rows8_kernel(const __grid_constant__ Attn8Params p, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  constexpr int KU = Geometry<D, false, true>::kKeys, NK = KU / 16;  // keys of a block, key tiles
  constexpr int kMostPages = KU / 16;                                // pages that a block touches
  constexpr int STAGES = kStages8, STAGE = kRowBlockBytes8, HALF = STAGE / 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kRowWarps8][STAGES];
  __shared__ uint64_t live[kRowWarps8][STAGES];                     // keys of a block that were loaded
  __shared__ float scales[kRowWarps8][STAGES][2][kMostPages];       // of its pages' keys and values
  __shared__ Patience patience;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = base + warp * STAGES * STAGE;
  if (threadIdx.x == 0) {
    patience.gave_up = 0;
    patience.limit = 1;  // (a block's copies)
    for (int i = 0; i < kRowWarps8; ++i)
      for (int j = 0; j < STAGES; ++j) mbar_init(&full[i][j], 1 + 32);
    fence_mbar_init();
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  __syncthreads();
  launch_dependents();
  wait_dependency();

  const int w = warp * gridDim.x + blockIdx.x;  // (few workers are spread over the SMs)
  const Line line = measure_line<D, false, true>(p, lane);
  if (line.bad && w == 0 && lane == 0) set_status(p.status, MK_DEV_BAD_INDEX);
  const int64_t x0 = line.border(w), x1 = line.border(w + 1);
  Note note = {0, 0, 0, 0};
  if (lane == 0) *note_of(p, D, w) = note;
  if (line.bad || x0 >= x1) return;
  const int pmask = (1 << p.page_shift) - 1;
  const int box = min(KU, pmask + 1);     // keys per TMA box
  const int npg = KU / box;               // pages a block touches

  using Place = Cursor<D, false, true>;
  Place cons;
  cons.find(p, line, x0, lane);
  Place prod = cons;
  int pk = 0, pke = 0;        // the producer's next block and the end of its item's part
  bool pdone = false;
  int win_b = -1, win0 = 0, win = -1;  // 32 entries of the block table, one per lane
  uint32_t issued = 0, done = 0;

  // first block and end of a cursor's item in this worker's part
  auto part_of = [&](const Place& c, int& k0, int& k1) {
    const int nk = c.blocks(p);
    k0 = c.block_at(x0, nk);
    k1 = c.block_at(x1, nk);
  };
  auto next_part = [&](Place& c, int& k0, int& k1) {
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
    const int st = issued % STAGES;
    uint8_t* dst = ring + st * STAGE;
    const int key0 = pk * KU, j0 = key0 >> p.page_shift, L = prod.s.ctx + prod.s.n;
    if (prod.b != win_b || j0 < win0 || j0 >= win0 + 32) {
      win_b = prod.b;
      win0 = j0 & ~31;
      const int j = win0 + lane;
      win = (j < p.max_pages && ((int64_t)j << p.page_shift) < L) ? p.table[(size_t)prod.b * p.max_pages + j] : -1;
    }
    uint64_t keys = 0;
#pragma unroll
    for (int h = 0; h < KU / 32; ++h) {
      const int key = key0 + h * 32 + lane;
      const int id = __shfl_sync(0xffffffffu, win, ((key >> p.page_shift) - win0) & 31);
      const bool in = key < L, ok = in && (unsigned)id < (unsigned)p.num_pages;
      keys |= (uint64_t)__ballot_sync(0xffffffffu, ok) << (32 * h);
      if (in && !ok) set_status(p.status, MK_DEV_BAD_INDEX);
    }
    // one box per page, of keys or values, and its scale
    const int pg = lane >> 1, is_v = lane & 1;
    const int id = __shfl_sync(0xffffffffu, win, (j0 + pg - win0) & 31);
    const bool mine = pg < npg && ((keys >> (pg * box)) & 1);
    const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
    if (lane == 0) {
      live[warp][st] = keys;
      mbar_arrive_expect_tx(&full[warp][st], boxes * box * D);
    }
    __syncwarp();
    if (mine) {
      const int row = ((id * p.Hkv + prod.g) << p.page_shift) + (key0 & pmask);
      tma_load_2d(dst + is_v * HALF + pg * box * D, is_v ? &vmap : &kmap, 0, row, &full[warp][st]);
      copy_async4(&scales[warp][st][is_v][pg], (is_v ? p.vscale : p.kscale) + (int64_t)id * p.Hkv + prod.g);
    } else if (pg < npg) {
      scales[warp][st][is_v][pg] = is_v ? 0.f : 1.f;  // (a page without keys)
    }
    mbar_arrive_copies(&full[warp][st]);
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
  for (int i = 0; i < STAGES; ++i) issue();

  // this lane's place in the products: row g of their eight or sixteen, elements (columns) c0, c0 + 1
  const int g = lane >> 2, c0 = (lane & 3) * 2;
  // row 8 h + g of an item's query rows (row r = token * G + head; rows past the last are zero), four elements of every
  // 16; with one eight of rows read while the item before is worked on
  uint2 qv[D / 16];
  auto load_q = [&](const Place& c, int h) {
    const int r = 8 * h + g;
    const bool in = r < c.s.n * p.G;
    const __nv_bfloat16* qr = p.q + (int64_t)(c.s.row0 + (in ? r / p.G : 0)) * p.ld_q +
                              ((int64_t)c.g * p.G + (in ? r % p.G : 0)) * D + 2 * c0;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
      qv[j] = in ? __ldg(reinterpret_cast<const uint2*>(qr + j * 16)) : make_uint2(0, 0);
  };
  if (NR == 1) load_q(cons, 0);
  for (bool more = true; more;) {
    const int n = cons.s.n, ctx = cons.s.ctx, L = ctx + n, nrows = n * p.G;
    const int nk = cons.blocks(p), kb = ck;
    float rs[NR][2];
    uint32_t qf[NR][D / 16][2];
#pragma unroll
    for (int h = 0; h < NR; ++h) {
      if (NR > 1) load_q(cons, h);
      // the row's largest element, as bf16 bits, to [2^14, 2^15)
      uint32_t big = 0;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) big = __vmaxu2(big, __vmaxu2(qv[j].x & 0x7FFF7FFFu, qv[j].y & 0x7FFF7FFFu));
      big = max(big & 0xFFFFu, big >> 16);
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      const int qe = min(max((int)(big >> 7), 15), 254);
      const float up = __uint_as_float((uint32_t)(141 + 127 - qe) << 23);       // 2^(14 - e)
      const float down = p.scale * __uint_as_float((uint32_t)(qe - 14) << 23);  // softmax scale 2^(e - 14)
#pragma unroll
      for (int e = 0; e < 2; ++e) rs[h][e] = __shfl_sync(0xffffffffu, down, (c0 + e) * 4);
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        qf[h][j][0] = pack_f16(bf_lo(qv[j].x) * up, bf_hi(qv[j].x) * up);
        qf[h][j][1] = pack_f16(bf_lo(qv[j].y) * up, bf_hi(qv[j].y) * up);
      }
    }
    Place coming = cons;
    int nk0 = 0, nk1 = 0;
    more = next_part(coming, nk0, nk1);
    if (NR == 1 && more) load_q(coming, 0);
    // the last key each of this lane's two rows of an eight sees
    const auto last_key = [&](int h, int e) {
      const int r = 8 * h + c0 + e;
      return r < nrows ? ctx + r / p.G : L - 1;
    };
    int lim[NR][2];
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) lim[h][e] = last_key(h, e);
    const int slot = 2 * w + (kb == 0 ? 1 : 0);  // of the part's record (free while a whole item is worked on)
    // results, in units of 2^(ve - 127): the power of two of the largest scale of values so far
    float o[NR][D / 16][4], m[NR][2], l[NR][2];
    int ve = 1;
    constexpr int kFold = kFoldKeys / KU;
    float mfold[NR][2], lfold[NR][2];  // the maxima of folded results, and their sums
#pragma unroll
    for (int h = 0; h < NR; ++h) {
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[h][t][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[h][e] = mfold[h][e] = -INFINITY;
        l[h][e] = lfold[h][e] = 0.f;
      }
    }
#pragma unroll 1
    for (int stop = kb + kFold;; stop += kFold) {
      for (; ck < min(cke, stop); ++ck) {
        const int st = done % STAGES;
        if (!wait_phase(&full[warp][st], (done / STAGES) & 1, &patience)) {
          if (lane == 0) set_status(p.status, MK_DEV_RING_TIMEOUT);
          // the copies in flight land in this CTA's memory: give them time before it goes
          for (uint32_t d = done; d < issued; ++d)
            for (int i = 0; i < 100000 && !mbar_try_wait(&full[warp][d % STAGES], (d / STAGES) & 1); ++i) {
            }
          return;
        }
        const uint32_t ks = smem_addr(ring + st * STAGE), vs = ks + HALF;
        const uint64_t keys = live[warp][st];
        const int key0 = ck * KU;
        constexpr uint64_t kAll = KU == 64 ? ~0ull : (1ull << (KU & 63)) - 1;
        const bool masked = keys != kAll || key0 + KU > ctx + 1;
        float ksc[NK], vsc[NK];  // scales, by tiles of 16 keys
#pragma unroll
        for (int t = 0; t < NK; ++t) {
          const int pg = t * 16 / box;
          ksc[t] = scales[warp][st][0][pg];
          vsc[t] = scales[warp][st][1][pg];
        }

        float s[NR][NK][4];
#pragma unroll
        for (int h = 0; h < NR; ++h)
#pragma unroll
          for (int t = 0; t < NK; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][t][e] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; j += 2) {
#pragma unroll
          for (int t = 0; t < NK; ++t) {
            // keys t * 16 .. + 15 by elements j * 16 .. + 31: codes of keys g and g + 8
            uint32_t k[4];
            ldsm4(swz8<D>(ks, t * 16 + (lane & 15), j + (lane >> 4)), k);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t a[4];
              widen_e4m3(k[2 * i], a[0], a[2]);
              widen_e4m3(k[2 * i + 1], a[1], a[3]);
#pragma unroll
              for (int h = 0; h < NR; ++h) mma_f16(s[h][t], a, qf[h][j + i][0], qf[h][j + i][1]);
            }
          }
        }
        if (masked) {
#pragma unroll
          for (int h = 0; h < NR; ++h)
#pragma unroll
            for (int t = 0; t < NK; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int k = t * 16 + g + (e >> 1) * 8;
                if (!((keys >> k) & 1) || key0 + k > lim[h][e & 1]) s[h][t][e] = -INFINITY;
              }
        }
        int vmax = ve, vmin = 254;
#pragma unroll
        for (int t = 0; t < NK; ++t) {
          const int e = exponent(vsc[t]);
          vmax = max(vmax, e);
          vmin = min(vmin, e == 0 ? 254 : e);  // (pages without keys have none)
        }
        vmax = min(vmax, 253);
        bool moved = vmax != ve;
        float mnew[NR][2];
        // what a score is worth in the exponent of two (a masked one times zero would be NaN)
        const auto worth = [&](int h, int t, int e) { return fmaxf(ksc[t] * rs[h][e], 0x1p-126f); };
#pragma unroll
        for (int h = 0; h < NR; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[h][0][e], s[h][0][e + 2]) * worth(h, 0, e);
#pragma unroll
            for (int t = 1; t < NK; ++t) x = fmaxf(x, fmaxf(s[h][t][e], s[h][t][e + 2]) * worth(h, t, e));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            mnew[h][e] = fmaxf(m[h][e], x);
            moved |= mnew[h][e] != m[h][e];
          }
        const auto from = [&](float mx) { return mx == -INFINITY ? 0.f : mx; };  // a row without any key so far
        if (__any_sync(0xffffffffu, moved)) {
          const float fv = exp2_down(ve - vmax);
          ve = vmax;
#pragma unroll
          for (int h = 0; h < NR; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float f = ex2(m[h][e] - from(mnew[h][e]));
              m[h][e] = mnew[h][e];
              l[h][e] *= f;
#pragma unroll
              for (int t = 0; t < D / 16; ++t) {
                o[h][t][e] *= f * fv;
                o[h][t][e + 2] *= f * fv;
              }
            }
        }
        const float vref = __uint_as_float((uint32_t)(254 - ve) << 23);  // 2^(127 - ve)
#pragma unroll
        for (int h = 0; h < NR; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mu = kBias - from(m[h][e]);
#pragma unroll
            for (int t = 0; t < NK; ++t) {
              const float f = worth(h, t, e);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float x = ex2(fmaf(s[h][t][e + 2 * i], f, mu));
                s[h][t][e + 2 * i] = x;
                l[h][e] += x;
              }
            }
          }
        bool bad_v = false;  // a value that is not finite behind a mask
        // (APART: a tile's scale lies far below the unit; code of its own, as a branch per tile cost heads of 64 5 %)
        const auto add_values = [&](auto APART) {
#pragma unroll
          for (int t = 0; t < NK; ++t) {
            // probabilities as operands: 16 keys by 8 rows, transposed
            float vf = vsc[t] * vref;
            const int down = min(ve - exponent(vsc[t]), kMostDown);
            if (APART.value) {
              const float up = __uint_as_float((uint32_t)(127 + down) << 23);
              vf *= up;
              times(o, up);
            }
            uint32_t pr[NR][2];
#pragma unroll
            for (int h = 0; h < NR; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                pr[h][e] = movm_trans(pack_f16(s[h][t][2 * e] * vf, s[h][t][2 * e + 1] * vf));
            // this lane's four keys of the 16: c0, c0 + 1, c0 + 8, c0 + 9
            uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
            if (masked) {
              const uint32_t k16 = (uint32_t)(keys >> (t * 16)) >> c0;
              keep0 = ((k16 & 1) ? 0xFFFFu : 0u) | ((k16 & 2) ? 0xFFFF0000u : 0u);
              keep1 = ((k16 & 0x100) ? 0xFFFFu : 0u) | ((k16 & 0x200) ? 0xFFFF0000u : 0u);
            }
#pragma unroll
            for (int d = 0; d < D / 16; d += 2) {
              // columns d * 16 .. + 31 of the 16 keys: columns 2 g and 2 g + 1 of each 16, of keys c0 and c0 + 1, then
              // c0 + 8 and c0 + 9
              uint32_t v[4];
              ldsm4t(swz8<D>(vs, t * 16 + (lane & 15), d + (lane >> 4)), v);
              if (masked) {
                // values that were not loaded are zero, whatever the memory held
                v[0] &= keep0; v[1] &= keep1; v[2] &= keep0; v[3] &= keep1;
                if (n > 1) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const uint32_t odd = nan_codes(v[e]);
                    bad_v |= odd != 0;
                    v[e] &= ~odd;
                  }
                }
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t a[4];
                widen_e4m3(__byte_perm(v[2 * i], 0, 0x3120), a[0], a[1]);
                widen_e4m3(__byte_perm(v[2 * i + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                for (int h = 0; h < NR; ++h) mma_f16(o[h][d + i], a, pr[h][0], pr[h][1]);
              }
            }
            if (APART.value) times(o, exp2_down(-down));
          }
        };
        if (vmin + kFar < ve) add_values(std::true_type());
        else add_values(std::false_type());
        if (masked && n > 1 && __any_sync(0xffffffffu, bad_v)) {
          // 0 * NaN would reach the rows that do not see the key: such values were left
          // out above and go to the rows that see it only
#pragma unroll 1
          for (int k = 0; k < KU; ++k) {
            if (!((keys >> k) & 1)) continue;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              const uint32_t two = lds32(swz8<D>(vs, k, d) + (g >> 1) * 4) >> (g & 1) * 16;
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                if ((two >> (8 * q) & 0x7Fu) != 0x7Fu) continue;
#pragma unroll
                for (int h = 0; h < NR; ++h)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    if (key0 + k <= lim[h][e]) o[h][d][2 * q + e] = __uint_as_float(0x7FC00000u);
              }
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
      const float unit = __uint_as_float((uint32_t)ve << 23);
#pragma unroll
      for (int h = 0; h < NR; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * h + c0 + e;
          if (r >= nrows) continue;
          const float f = fold_weight(mfold[h][e], m[h][e]);
          mfold[h][e] = m[h][e];
          lfold[h][e] = lfold[h][e] * f + l[h][e];
          l[h][e] = last ? lfold[h][e] : 0.f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            float2* at = reinterpret_cast<float2*>(part_o(p, D, slot, r) + d * 16 + 2 * g);
            const float2 was = some ? *at : make_float2(0.f, 0.f);
            const float2 x = make_float2(o[h][d][e] * unit + was.x * f, o[h][d][2 + e] * unit + was.y * f);
            if (!last) *at = x;
            o[h][d][e] = last ? x.x : 0.f;
            o[h][d][2 + e] = last ? x.y : 0.f;
          }
        }
      if (last) {
        ve = 127;
        break;
      }
      ve = 1;
    }

#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[h][e] += __shfl_xor_sync(0xffffffffu, l[h][e], 4);
        l[h][e] += __shfl_xor_sync(0xffffffffu, l[h][e], 8);
        l[h][e] += __shfl_xor_sync(0xffffffffu, l[h][e], 16);
      }
    const bool whole = kb == 0 && cke == nk;
    if (kb != 0 && cke == nk) note = {cons.first_worker(line), cons.s.row0, cons.g, n};
    __nv_bfloat16* ob = p.out + (int64_t)cons.s.row0 * p.ld_out + (int64_t)cons.g * p.G * D;
    const float unit = __uint_as_float((uint32_t)ve << 23);
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * h + c0 + e;
        if (r >= nrows) continue;
        if (whole) {
          const float f = l[h][e] == 0.f ? 0.f : 1.0f / l[h][e];  // (a row without keys is zero)
          __nv_bfloat16* dst = ob + (int64_t)(r / p.G) * p.ld_out + (r % p.G) * D + 2 * g;
#pragma unroll
          for (int d = 0; d < D / 16; ++d)
            *reinterpret_cast<uint32_t*>(dst + d * 16) = pack_bf16(o[h][d][e] * unit * f, o[h][d][2 + e] * unit * f);
        } else {
          float* dst = part_o(p, D, slot, r) + 2 * g;
#pragma unroll
          for (int d = 0; d < D / 16; ++d)
            *reinterpret_cast<float2*>(dst + d * 16) = make_float2(o[h][d][e] * unit, o[h][d][2 + e] * unit);
          if (g == 0) *reinterpret_cast<float2*>(part_ml(p, D, slot, r)) = make_float2(m[h][e], l[h][e]);
        }
      }
    cons = coming;
    ck = nk0;
    cke = nk1;
  }
  if (lane == 0 && note.tokens) *note_of(p, D, w) = note;
}

template <int D, int NR>
cudaError_t launch_rows8_t(const Attn8Params& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                           cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(rows8_kernel<D, NR>, kSmemBytes8, &allowed);
  if (e != cudaSuccess) return e;
  return launch_early(rows8_kernel<D, NR>, dim3((unsigned)(p.workers / kRowWarps8)), dim3(kRowWarps8 * 32), kSmemBytes8,
                      stream, p, kmap, vmap);
}
template <int D>
cudaError_t launch_rows8_d(const Attn8Params& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                           cudaStream_t stream) {
  static_assert(kMaxFewRows8 == 16, "two eights of rows at most");
  if (p.rows <= 8) return launch_rows8_t<D, 1>(p, kmap, vmap, stream);
  return launch_rows8_t<D, 2>(p, kmap, vmap, stream);
}

}  // namespace

cudaError_t launch_rows8(const Attn8Params& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int D,
                         cudaStream_t stream) {
  return D == 128 ? launch_rows8_d<128>(p, kmap, vmap, stream) : launch_rows8_d<64>(p, kmap, vmap, stream);
}

}  // namespace mk
