// Paged attention of few query rows per request and key/value head (single
// tokens, drafts: at most 32 rows), and the join of partial results.
//
// Every key and value is read once for a handful of rows, so HBM bounds it
// and the arithmetic only has to keep out of the way: at the SM's share of
// HBM (about 45 GB/s) a 16 KB block of keys and values lands per warp every
// 1.5 us.  Each warp is a worker of its own, with its own part of the work
// line, its own ring of three blocks filled by TMA (pages gathered into a
// 128-byte-swizzled tile), its own softmax state in registers: no warp waits
// for another.  The products run on m16n8k16 warp matrix instructions, which
// take 16 rows at a time; a tcgen05 product has 128 rows, of which a decode
// step would fill four, and would put two more round trips (through tensor
// memory) into each block's chain.
//
//   s = q k^T scale;  m' = max(m, max s);  p = 2^(s - m');
//   l = l 2^(m - m') + sum p;  o = o 2^(m - m') + p v
//
// The probabilities enter the second product as two bf16 parts (p and what
// its rounding leaves), which keeps them to 2^-17; the extra products cost
// nothing here.
#include "paged_attention.cuh"

namespace mk {
namespace {

using namespace ptx;

constexpr int kStages = 3;
constexpr int kHalfBytes = 8192;             // keys, or values, of a block
constexpr int kStageBytes = 2 * kHalfBytes;
constexpr int kThreads = kRowWarps * 32;

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

template <int D, int NM>
__global__ void __launch_bounds__(kThreads, 1)
    rows_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
  constexpr int KU = Geometry<D, false>::kKeys;  // keys per block
  constexpr int NH = D / 64;                     // 128-byte column halves
  constexpr int NT = KU / 8;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kRowWarps][kStages];
  __shared__ uint64_t live[kRowWarps][kStages];  // keys of a block that were loaded
  __shared__ int gave_up;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = base + warp * kStages * kStageBytes;
  const uint32_t qs = smem_addr(base + kRowWarps * kStages * kStageBytes + warp * kMaxFewRows * D * 2);
  if (threadIdx.x == 0) {
    gave_up = 0;
    for (int i = 0; i < kRowWarps; ++i)
      for (int j = 0; j < kStages; ++j) mbar_init(&full[i][j], 1);
    fence_mbar_init();
  }
  __syncthreads();
  launch_dependents();

  const int w = blockIdx.x * kRowWarps + warp;
  const Line line = measure_line<D, false>(p, lane);
  if (line.bad && w == 0 && lane == 0) set_status(p.status, MK_DEV_BAD_INDEX);
  const int64_t x0 = line.border(w), x1 = line.border(w + 1);
  int4 note = make_int4(0, 0, 0, 0);
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
    for (int h = 0; h < KU / 32; ++h) {
      const int key = key0 + h * 32 + lane;
      const int id = __shfl_sync(0xffffffffu, win, ((key >> p.page_shift) - win0) & 31);
      const bool in = key < L, ok = in && (unsigned)id < (unsigned)p.num_pages;
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
  bool more = ck < cke || next_part(cons, ck, cke);
  if (!more) return;
  prod = cons;
  pk = ck;
  pke = cke;
  for (int i = 0; i < kStages; ++i) issue();

  const int r0 = lane >> 2, c0 = (lane & 3) * 2;
  while (more) {
    const int n = cons.s.n, ctx = cons.s.ctx, L = ctx + n, nrows = n * p.G;
    const int nk = cons.blocks(p), kb = ck;
    // query rows, row r = token * G + head, into shared memory; rows past the last are zero
    const __nv_bfloat16* qb = p.q + (int64_t)p.cu[cons.b] * p.ld_q + (int64_t)cons.g * p.G * D;
    for (int i = lane; i < NM * 16 * (D / 8); i += 32) {
      const int r = i / (D / 8), c = i % (D / 8);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < nrows) v = __ldg(reinterpret_cast<const uint4*>(qb + (int64_t)(r / p.G) * p.ld_q + (r % p.G) * D + c * 8));
      const uint32_t a = swz(qs + (c >> 3) * (NM * 16 * 128), r, c & 7);
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                   : "memory");
    }
    __syncwarp();
    // the last key each of this lane's rows sees
    int lim[2 * NM];
#pragma unroll
    for (int i = 0; i < 2 * NM; ++i) {
      const int r = i * 8 + r0;
      lim[i] = r < nrows ? ctx + r / p.G : L - 1;
    }
    auto load_q = [&](int m, int kk, uint32_t (&a)[4]) {
      // matrices: rows 0-7 / 8-15 of the tile, then the same at the next 8 columns
      const int r = m * 16 + (lane & 15), c = kk * 2 + (lane >> 4);
      ldsm4(swz(qs + (c >> 3) * (NM * 16 * 128), r, c & 7), a);
    };
    uint32_t qf[NM == 1 ? D / 16 : 1][4];
    if constexpr (NM == 1) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) load_q(0, kk, qf[kk]);
    }
    float o[NM][D / 8][4], m[2 * NM], l[2 * NM];
#pragma unroll
    for (int i = 0; i < NM; ++i)
#pragma unroll
      for (int t = 0; t < D / 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][t][e] = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * NM; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }

    for (; ck < cke; ++ck) {
      const int st = done % kStages;
      if (!wait_phase(&full[warp][st], (done / kStages) & 1, &gave_up)) {
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

      float s[NM][NT][4];
#pragma unroll
      for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][t][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t a[NM][4];
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          if constexpr (NM == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[i][e] = qf[kk][e];
          } else {
            load_q(i, kk, a[i]);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
          uint32_t b[4];  // keys t*8.. and t*8+8.., columns kk*16.. and +8
          const int r = t * 8 + (lane >> 4) * 8 + (lane & 7), c = kk * 2 + ((lane >> 3) & 1);
          ldsm4(swz(ks + (c >> 3) * (KU * 128), r, c & 7), b);
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            mma_bf16(s[i][t], a[i], b[0], b[1]);
            mma_bf16(s[i][t + 1], a[i], b[2], b[3]);
          }
        }
      }
      if (masked) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = t * 8 + c0 + (e & 1);
            const bool there = (keys >> k) & 1;
#pragma unroll
            for (int i = 0; i < NM; ++i)
              if (!there || key0 + k > lim[2 * i + (e >> 1)]) s[i][t][e] = -INFINITY;
          }
      }
      bool moved = false;
      float mnew[2 * NM], muse[2 * NM];
#pragma unroll
      for (int i = 0; i < 2 * NM; ++i) {
        float x = -INFINITY;
#pragma unroll
        for (int t = 0; t < NT; ++t) x = fmaxf(x, fmaxf(s[i >> 1][t][(i & 1) * 2], s[i >> 1][t][(i & 1) * 2 + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        mnew[i] = fmaxf(m[i], x * p.scale);
        muse[i] = mnew[i] == -INFINITY ? 0.f : mnew[i];  // a row without any key so far
        moved |= mnew[i] != m[i];
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < 2 * NM; ++i) {
          const float f = ex2(m[i] - muse[i]);
          m[i] = mnew[i];
          l[i] *= f;
#pragma unroll
          for (int t = 0; t < D / 8; ++t) {
            o[i >> 1][t][(i & 1) * 2] *= f;
            o[i >> 1][t][(i & 1) * 2 + 1] *= f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = ex2(fmaf(s[i][t][e], p.scale, -muse[2 * i + (e >> 1)]));
            s[i][t][e] = x;
            l[2 * i + (e >> 1)] += x;
          }
      bool odd = false;  // a value that is not finite behind a mask
#pragma unroll
      for (int kk = 0; kk < KU / 16; ++kk) {
        uint32_t hi[NM][4], lo[NM][4];
#pragma unroll
        for (int i = 0; i < NM; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = s[i][2 * kk + (e >> 1)][(e & 1) * 2], y = s[i][2 * kk + (e >> 1)][(e & 1) * 2 + 1];
            const uint32_t h = pack_bf16(x, y);
            hi[i][e] = h;
            lo[i][e] = pack_bf16(x - bf_lo(h), y - bf_hi(h));
          }
        // this lane's four keys of the 16: c0, c0 + 1, c0 + 8, c0 + 9
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (masked) {
          const uint32_t kb16 = (uint32_t)(keys >> (kk * 16)) >> c0;
          keep0 = ((kb16 & 1) ? 0xFFFFu : 0u) | ((kb16 & 2) ? 0xFFFF0000u : 0u);
          keep1 = ((kb16 & 0x100) ? 0xFFFFu : 0u) | ((kb16 & 0x200) ? 0xFFFF0000u : 0u);
        }
#pragma unroll
        for (int t = 0; t < D / 8; t += 2) {
          uint32_t b[4];  // columns t*8.. (keys 0-7, 8-15), then the next 8 columns
          const int r = kk * 16 + (lane & 15), c = t + (lane >> 4);
          ldsm4t(swz(vs + (c >> 3) * (KU * 128), r, c & 7), b);
          if (masked) {
            // values that were not loaded are zero, whatever the memory held
            b[0] &= keep0; b[1] &= keep1; b[2] &= keep0; b[3] &= keep1;
            if (n > 1) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (nonfinite_lo(b[e])) { b[e] &= 0xFFFF0000u; odd = true; }
                if (nonfinite_hi(b[e])) { b[e] &= 0xFFFFu; odd = true; }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            mma_bf16(o[i][t], hi[i], b[0], b[1]);
            mma_bf16(o[i][t + 1], hi[i], b[2], b[3]);
            mma_bf16(o[i][t], lo[i], b[0], b[1]);
            mma_bf16(o[i][t + 1], lo[i], b[2], b[3]);
          }
        }
      }
      if (masked && n > 1 && __any_sync(0xffffffffu, odd)) {
        // 0 * inf would reach the rows that do not see the key: such values were left
        // out above and go to the rows that see it only
        for (int k = 0; k < KU; ++k) {
          if (!((keys >> k) & 1)) continue;
#pragma unroll
          for (int t = 0; t < D / 8; ++t) {
            const uint32_t v = lds32(swz(vs + (t >> 3) * (KU * 128), k, t & 7) + c0 * 2);
#pragma unroll
            for (int i = 0; i < 2 * NM; ++i) {
              if (key0 + k > lim[i]) continue;
              if (nonfinite_lo(v)) o[i >> 1][t][(i & 1) * 2] += bf_lo(v);
              if (nonfinite_hi(v)) o[i >> 1][t][(i & 1) * 2 + 1] += bf_hi(v);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the block
      ++done;
      issue();
    }

#pragma unroll
    for (int i = 0; i < 2 * NM; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    const bool whole = kb == 0 && cke == nk;
    const int slot = 2 * w + (kb == 0 ? 1 : 0);
    if (!whole) {
      note.x |= kb == 0 ? kGoesOn : cke == nk ? kCameIn | kEnded : kCameIn;
      if (kb != 0) {
        note.y = p.cu[cons.b];
        note.z = cons.g;
        note.w = n;
      }
    }
    __nv_bfloat16* ob = p.out + (int64_t)p.cu[cons.b] * p.ld_out + (int64_t)cons.g * p.G * D;
#pragma unroll
    for (int i = 0; i < 2 * NM; ++i) {
      const int r = i * 8 + r0;
      if (r >= nrows) continue;
      if (whole) {
        const float f = l[i] == 0.f ? 0.f : 1.0f / l[i];  // a row without keys is zero
        __nv_bfloat16* dst = ob + (int64_t)(r / p.G) * p.ld_out + (r % p.G) * D + c0;
#pragma unroll
        for (int t = 0; t < D / 8; ++t)
          *reinterpret_cast<uint32_t*>(dst + t * 8) =
              pack_bf16(o[i >> 1][t][(i & 1) * 2] * f, o[i >> 1][t][(i & 1) * 2 + 1] * f);
      } else {
        float* dst = part_o(p, D, slot, r) + c0;
#pragma unroll
        for (int t = 0; t < D / 8; ++t)
          *reinterpret_cast<float2*>(dst + t * 8) =
              make_float2(o[i >> 1][t][(i & 1) * 2], o[i >> 1][t][(i & 1) * 2 + 1]);
        if ((lane & 3) == 0) *reinterpret_cast<float2*>(part_ml(p, D, slot, r)) = make_float2(m[i], l[i]);
      }
    }
    more = next_part(cons, ck, cke);
  }
  if (lane == 0 && note.x) *note_of(p, D, w) = note;
}

// Join of the items that workers' borders cut: block w looks whether an item
// ends in worker w's part that began before it.  Its partial records are the
// second slot of the nearest worker before whose last item goes on, then the
// first slots of the workers from there to w, in order of keys.  A warp
// merges a share of a row's records; shares meet in shared memory.
constexpr int kJoinWarps = 16;

template <int D, bool CHUNK>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int E = D / 32;
  __shared__ float so[kJoinWarps][D], sml[kJoinWarps][2];
  __shared__ int slots[kMaxWorkers + 1];
  __shared__ int count_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = blockIdx.x;
  wait_dependency();
  const int4 note = *note_of(p, D, w);
  if (!(note.x & kEnded)) return;
  const int rows_all = note.w * p.G, per = (rows_all + gridDim.y - 1) / gridDim.y;
  const int row_base = blockIdx.y * per, rows = min(per, rows_all - row_base);
  if (rows <= 0) return;
  if (warp == 0) {
    // records from the last to the first (a worker whose part rounds to nothing left none)
    int n = 1;
    if (lane == 0) slots[0] = 2 * w;
    for (int c0 = w - 1; c0 >= 0; c0 -= 32) {
      const int c = c0 - lane, flags = c >= 0 ? note_of(p, D, c)->x : 0;
      const unsigned begin = __ballot_sync(0xffffffffu, flags & kGoesOn);
      const unsigned upto = begin ? (begin & -begin) - 1 : 0xffffffffu;  // workers after the one where it began
      const unsigned in = __ballot_sync(0xffffffffu, flags & kCameIn) & upto;
      const int at = n + __popc(in & ((1u << lane) - 1));
      if (((in >> lane) & 1)) slots[at] = 2 * c;
      n += __popc(in);
      if (begin) {
        if (lane == __ffs(begin) - 1) slots[n] = 2 * c + 1;
        ++n;
        break;
      }
    }
    if (lane == 0) count_s = n;
  }
  __syncthreads();
  const int count = count_s;
  int shares = 1;
  while (shares * 2 * rows <= kJoinWarps && shares * 4 < count) shares *= 2;
  const int rows_at_once = kJoinWarps / shares, share = warp % shares;
  for (int rr0 = 0; rr0 < rows; rr0 += rows_at_once) {
    const int rr = rr0 + warp / shares;
    const bool on = rr < rows;
    // row of the item -> token and head; row of a partial record
    const int row = row_base + (on ? rr : 0), tok = row / p.G, head = row % p.G;
    const int rec = CHUNK ? (tok / p.tq) * 128 + (tok % p.tq) * p.G + head : row;
    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    constexpr int U = 8;  // records in flight
    for (int i0 = share; on && i0 < count; i0 += U * shares) {
      float2 ml[U];
      float v[U][E];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * shares;
        ml[j] = make_float2(-INFINITY, 0.f);
        if (i < count) {
          const int slot = slots[count - 1 - i];
          ml[j] = __ldcg(reinterpret_cast<const float2*>(part_ml(p, D, slot, rec)));
          const float* src = part_o(p, D, slot, rec) + lane * E;
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
      __nv_bfloat16* dst = p.out + ((int64_t)note.y + tok) * p.ld_out + (int64_t)(note.z * p.G + head) * D + lane * E;
      if constexpr (E == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f));
      else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16(o[0] * f, o[1] * f);
    }
  }
}

}  // namespace

cudaError_t launch_join(const AttnParams& p, int D, bool chunk, cudaStream_t stream) {
  if (p.workers < 2) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.workers, chunk ? 8u : 1u);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (chunk) return D == 128 ? cudaLaunchKernelEx(&cfg, join_kernel<128, true>, p) : cudaLaunchKernelEx(&cfg, join_kernel<64, true>, p);
  return D == 128 ? cudaLaunchKernelEx(&cfg, join_kernel<128, false>, p) : cudaLaunchKernelEx(&cfg, join_kernel<64, false>, p);
}

template <int D, int NM>
static cudaError_t launch_rows_t(const AttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 cudaStream_t stream) {
  constexpr int smem = smem_bytes_rows<D>();
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(rows_kernel<D, NM>, smem, &allowed);
  if (e != cudaSuccess) return e;
  rows_kernel<D, NM><<<(unsigned)(p.workers / kRowWarps), kThreads, smem, stream>>>(p, kmap, vmap);
  return cudaGetLastError();
}

cudaError_t launch_rows(const AttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int D,
                        cudaStream_t stream) {
  if (p.rows <= 16) return D == 128 ? launch_rows_t<128, 1>(p, kmap, vmap, stream) : launch_rows_t<64, 1>(p, kmap, vmap, stream);
  return D == 128 ? launch_rows_t<128, 2>(p, kmap, vmap, stream) : launch_rows_t<64, 2>(p, kmap, vmap, stream);
}

}  // namespace mk
