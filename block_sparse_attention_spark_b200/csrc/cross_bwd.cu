// Gradient of cross attention on the sm_100a tensor cores (bf16).
//
//   D_i = dO_i . O_i,  P = exp(S - lse),  dV = P^T dO,  dS = P (dO V^T - D),
//   dQ = scale dS K,  dK = scale dS^T Q   (a key head sums over its query heads)
//
// Three launches: stat_kernel forms D and lse log2 e of the rows; main_kernel's
// first blocks (rows_body, dQ) hold a tile of 128 queries and stream the keys, its
// others (keys_body, dK and dV) hold a tile of 128 keys and stream the queries;
// sum_kernel joins the shares of dK and dV. A fourth, sum_rows_kernel, where there
// are so few query tiles that their keys are split too. S and dP are formed twice,
// seven products of 128x128xd a tile pair where five would do: adding dQ up over
// key tiles would take float32 atomics (Nk / 128 times Nq d of them, in an order
// that changes) or one CTA for all the keys. (With one key tile there is nothing
// to add up; a body for that case has not been built.)
//
// Both bodies: one persistent CTA per SM, eight warps on the elementwise part
// (each thread one row of the tile's TMEM lanes and half of its 128 columns),
// one warp on TMA, one on MMAs. P and dS are rounded to bf16, the operand type
// of the MMA, in TMEM, where they are the A operand of the second product of
// each chain. S and dP of whole tiles have N = 128 (in rows_body an item's last
// key tile is cut to the next multiple of 16 keys), the second products N = d;
// N = 64 runs at half the rate.
// Sums, P before rounding and all statistics are float32.
//
// Measured (72,576 queries of 40 heads over 256 keys, d = 128): 1,520 us (1,713 in
// a loop of 0.15 s): statistics 241 us = 6.2 TB/s; dK and dV 620 = 1.23 PFLOP/s of
// MMA work, 90% of what the card sustains in cuBLAS under its 1,000 W (1.37): power
// bounds them (SM clock 1.52 GHz), exponentials on the FMA pipe or fewer
// instructions in the elementwise warps changed nothing; dQ about 600 for three
// products instead of four, 0.95: what keeps it below the others is not known.
//
// Bounded waits as in the forward kernels.
#include "cross_pack.cuh"
#include "cross_tc.cuh"

namespace spark {
namespace cross {
namespace bwd {

using namespace tc;

constexpr int TILE = 128, EW_WARPS = 8, TMA_WARP = 8, MMA_WARP = 9, OUT_WARP0 = 12;
constexpr int THREADS = 512;               // warps past the ones named stay idle
static_assert(256 * 176 + 256 * 72 <= THREADS * 128, "registers the block owns");
constexpr int STAGES = 5;

struct Args {
  TensorMap q, k, v, dout, dqm;              // dqm: dq
  View o, dov, dq, dk, dv;                   // o: out; dov: dout
  const float* lse;
  const int32_t* key_len;                    // kept keys per item (after packing), or null
  const int32_t* place;                      // packed row of each key, or null
  int* status;
  int B, Hq, Hkv, G, Nq, Nk, NqP;            // NqP: Nq rounded up to 128
  int qtiles, ktiles;
  int ksplits, kper, kitems;                 // shares of a key tile's query tiles, tiles per share (unless dealt)
  int qsplits, qitems;                       // shares of a query tile's key tiles
  int dealt;                                 // lengths, and more than one item a CTA: deal_out says who does what
  int* deal;                                 // its shares of a key tile and (at 4) key tiles before each item of the batch
  float scale, sl2;
  float *lse2, *delta;                       // [B * Hq][NqP]
  float* part;                               // [key tiles (dealt: that have kept keys)][shares][2][128][d]: dV, dK
  float* qpart;                              // [qitems][128][d] shares of dQ
};

// ------------------------------------------------------------------ who does what
// Shares of a key tile's L query tiles for `units` key tiles: the fewest of
// those within 2% of the least time, in tiles: the rounds of items times the tiles
// of an item and four more (its 128 KB of sums, written and read again, take about
// that long), and 0.15 for each share that sum_kernel reads in turn.
constexpr int KSLOTS = 6 * SM_COUNT;         // most shares in all, unless every tile has one
__host__ __device__ inline int most_shares(int units, int L) {
  const int s = units > 0 ? KSLOTS / units : KSLOTS;
  return s < 1 ? 1 : s < L ? s : L;
}
__host__ __device__ inline float share_cost(int units, int L, int s) {
  return (float)((L + s - 1) / s + 4) * (float)((units * s + SM_COUNT - 1) / SM_COUNT) + 0.15f * (float)s;
}

// What a CTA does: its items of dK and dV are `block`, block + blocks, ... below
// kitems, those of dQ first, first + step, ... below end.
struct Deal {
  int ksplits, kper, kitems;
  int b, before;                             // item of the batch of the CTA's first key tile, key tiles a head before that
  int first, end, step;
  int stay;                                  // no more than two key tiles: K stays in shared memory
};

// With lengths, which only the device knows, by one warp: key tiles without a
// kept key are left out, so that the others are shared out evenly; query tiles go
// to the CTAs in runs of equal weight, 1 for a key tile and 2 for the rest of an
// item. 2 x 16,128 queries of 8 heads over 512 keys, of which 256 and 256 are kept:
// 154 us (every blocks-th item, empty ones too, and no K that stays: 211); 500 and
// 75: 202 (224 with weights 2 and 1; before 227). With one item a CTA at most there
// is nothing to deal, and this would take 4 us (3 x 777 queries: 26 against 22).
__device__ __forceinline__ void deal_out(const Args& a, bool rows, int block, int blocks, Deal* out) {
  const int lane = threadIdx.x;
  auto tiles = [&](int b) { return b < a.B ? (item_len(a.key_len, a.Nk, b, nullptr, false) + TILE - 1) / TILE : 0; };
  const int mine = tiles(lane);
  int sum = mine, top = mine;
  for (int b = lane + 32; b < a.B; b += 32) {
    sum += tiles(b);
    top = max(top, tiles(b));
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  top = __reduce_max_sync(0xffffffffu, top);
  Deal d = {};
  const int units = a.Hkv * sum, L = a.G * a.qtiles, most = most_shares(units, L);
  float least = INFINITY;
  for (int s = 1 + lane; s <= most; s += 32) least = fminf(least, share_cost(units, L, s));
  least = -warp_maxf(-least);
  int pick = most;
  for (int s = 1 + lane; s <= most; s += 32)
    if (share_cost(units, L, s) <= least * 1.02f) pick = min(pick, s);
  pick = __reduce_min_sync(0xffffffffu, pick);
  d.kper = (L + pick - 1) / pick;
  d.ksplits = (L + d.kper - 1) / d.kper;
  d.kitems = units * d.ksplits;
  d.stay = top <= 2 && a.qsplits == 1;
  d.first = block;                           // shares of a query tile: every blocks-th
  d.end = a.qitems;
  d.step = blocks;
  const int64_t per_item = (int64_t)a.Hq * a.qtiles, all = per_item * (sum + 2 * (int64_t)a.B);
  const int64_t lo = all * block / blocks, hi = all * (block + 1) / blocks;
  if (rows && a.qsplits == 1) {
    d.step = 1;
    d.first = a.qitems;
  }
  if (lane == 0) *out = d;
  if (!rows && block == 0 && lane == 0) a.deal[0] = d.ksplits;
  __syncwarp();
  int run = 0;                               // key tiles of the items before
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane, t = b0 == 0 ? mine : tiles(b);
    int inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const int before = run + inc - t;
    run += __shfl_sync(0xffffffffu, inc, 31);
    if (b >= a.B) continue;
    if (rows) {
      if (a.qsplits == 1) {
        const int64_t w = t + 2, from = per_item * (before + 2 * (int64_t)b), to = from + per_item * w;
        if (lo >= from && lo < to) out->first = (int)(b * per_item + (lo - from + w - 1) / w);
        if (hi >= from && hi < to) out->end = (int)(b * per_item + (hi - from + w - 1) / w);
      }
    } else {
      const int u = block / d.ksplits;
      if (u >= a.Hkv * before && u < a.Hkv * (before + t)) {
        out->b = b;
        out->before = before;
      }
      if (block == 0) a.deal[4 + b] = before;
    }
  }
}

// ------------------------------------------------------------------ D and lse
// 16 lanes (d = 128; 8 for 64) a row, four rows a lane in flight. Rows past Nq get
// lse = +inf (so P = 0) and D = 0. Bound by HBM: O and dO are read once.
// The blocks past `blocks` pack the kept keys of a masked call, which needs
// nothing of this and nothing here needs. Forming D inside rows_body instead (four
// warps beside its elementwise ones) was slower: their instructions are the
// scarce thing there.
template <int D>
__global__ void __launch_bounds__(256) stat_kernel(const __grid_constant__ Args a, const __grid_constant__ PackArgs pack,
                                                  int per_head, int blocks) {
  constexpr int LPR = D / 8, ROWS = 256 / LPR;
  let_next_start();
  if ((int)blockIdx.x >= blocks) {
    pack_block(pack, blockIdx.x - blocks);
    return;
  }
  const int bh = blockIdx.x / per_head, part = blockIdx.x % per_head, b = bh / a.Hq, h = bh % a.Hq, l = threadIdx.x % LPR;
  const int n0 = part * (4 * ROWS) + threadIdx.x / LPR;
  // (the lengths of a masked call are counts: pack_block has looked at the caller's)
  if (a.key_len != nullptr && pack.mask == nullptr && part == 0 && h == 0 && threadIdx.x == 0)
    item_len(a.key_len, a.Nk, b, a.status, true);
  const char* po = a.o.data + 2 * (b * a.o.b + h * a.o.h + 8 * l);
  const char* pd = a.dov.data + 2 * (b * a.dov.b + h * a.dov.h + 8 * l);
  uint4 x[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = min(n0 + i * ROWS, a.Nq - 1);
    x[i] = __ldcs(reinterpret_cast<const uint4*>(po + 2 * n * a.o.n));
    y[i] = *reinterpret_cast<const uint4*>(pd + 2 * n * a.dov.n);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ys[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      s = fmaf(bf_lo(xs[c]), bf_lo(ys[c]), s);
      s = fmaf(bf_hi(xs[c]), bf_hi(ys[c]), s);
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int n = n0 + i * ROWS;
    if (l == 0 && n < a.NqP) {
      const size_t at = (size_t)bh * a.NqP + n;
      a.delta[at] = n < a.Nq ? s : 0.f;
      // a row without weights (lse = -inf) has no gradient either
      const float lse = n < a.Nq ? a.lse[(size_t)bh * a.Nq + n] : INFINITY;
      a.lse2[at] = lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
    }
  }
}

template <int D>
struct Lay {
  static constexpr int ATOMS = D / 64;
  static constexpr int ATOM = TILE * 128;
  static constexpr int BYTES = ATOM * ATOMS;           // a tile of 128 rows
  static constexpr int OFF_ROW = (2 + STAGES) * BYTES; // two sets of lse and D of 128 queries
  static constexpr int OFF_BAR = OFF_ROW + 2048;
  static constexpr int OFF_DEAL = OFF_BAR + 448;
  static constexpr int SMEM = OFF_BAR + 512;
  static_assert(SMEM <= 232448, "shared memory of a block");
};
constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(TILE >> 4) << 24);

// D (TMEM) = A B^T for two tiles of 128 rows (K-major), n of B's rows.
template <int D>
__device__ __forceinline__ void product_nt(uint32_t e, uint32_t d, uint32_t sa, uint32_t sb, int n) {
  const uint64_t da = sdesc(sa, 16, 1024), db = sdesc(sb, 16, 1024);
  const uint32_t idesc = IDESC | ((uint32_t)(n >> 3) << 17);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint64_t o = (uint64_t)(((ks >> 2) * Lay<D>::ATOM + (ks & 3) * 32) >> 4);
    mma_f16_if(e, d, da + o, db + o, idesc, ks > 0 ? 1u : 0u);
  }
}
// D (TMEM, 128 x d) (+)= A (TMEM, bf16, 16 rows of B a step) B, B a tile of rows in shared memory.
// GAP: A's values of B's rows 64.. are GAP columns further on.
template <int D, int GAP>
__device__ __forceinline__ void product_ts(uint32_t e, uint32_t d, uint32_t ta, uint32_t sb, int steps, bool add) {
  const uint64_t db = sdesc(sb, Lay<D>::ATOM, 1024);
  const uint32_t idesc = IDESC | (1u << 16) | ((uint32_t)(D >> 3) << 17);
  if (steps == TILE / 16) {
#pragma unroll
    for (int kk = 0; kk < TILE / 16; ++kk)
      mma_ts_if(e, d, ta + 8u * kk + (kk >= 4 ? (uint32_t)GAP : 0u), db + (uint64_t)((kk * 2048) >> 4), idesc, (kk > 0 || add) ? 1u : 0u);
  } else {
    for (int kk = 0; kk < steps; ++kk)
      mma_ts_if(e, d, ta + 8u * kk + (kk >= 4 ? (uint32_t)GAP : 0u), db + (uint64_t)((kk * 2048) >> 4), idesc, (kk > 0 || add) ? 1u : 0u);
  }
}
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const TensorMap& m, int n, int h, int b, uint32_t bar) {
  mbar_arrive_tx(bar, Lay<D>::BYTES);
#pragma unroll
  for (int x = 0; x < Lay<D>::ATOMS; ++x)
    tma_load_4d(dst + x * Lay<D>::ATOM, &m.map, 64 * x, n, m.h_on ? h : 0, m.b_on ? b : 0, bar);
}

// Shared start and end of both bodies.
struct Block {
  uint32_t base, bar0, tmem;
  int warp, lane;
  volatile int* abort_flag;
};
template <int D>
__device__ __forceinline__ bool start(unsigned char* smem, int nbar, const unsigned* counts, int* status, Block& k) {
  k.lane = threadIdx.x & 31;
  k.warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  k.base = smem_u32(smem);
  if (k.base & 1023u) {                      // the swizzle needs it; the launch guarantees it
    if (threadIdx.x == 0) set_status(status, STATUS_BAD_INPUT);
    return false;
  }
  k.bar0 = k.base + Lay<D>::OFF_BAR;
  uint32_t* words = reinterpret_cast<uint32_t*>(smem + Lay<D>::OFF_BAR + 8 * nbar);
  k.abort_flag = reinterpret_cast<volatile int*>(words + 1);
  if (threadIdx.x == 0) {
    words[1] = words[2] = 0;             // abort; a wait of the elementwise warps gave up
    for (int i = 0; i < nbar; ++i) mbar_init(k.bar0 + 8u * i, counts[i]);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (k.warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(words)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  k.tmem = __shfl_sync(0xffffffffu, words[0], 0);
  wait_for_last();
  return true;
}
__device__ __forceinline__ void finish(const Block& k) {
  fence_before();
  __syncthreads();
  fence_after();
  if (k.warp == MMA_WARP)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(k.tmem), "r"(512u));
}

// ------------------------------------------------------------------ dK, dV
// TMEM: S^T 0, dP^T 128, dV 256, dK 384. Lanes are keys, columns queries. P and
// dS stand over their S and dP, the lower 64 columns' values at 0..31, the upper
// ones' at 64..95, so that neither half of the warps writes over what the other
// has yet to read. The chains S -> P -> dV and dP -> dS -> dK alternate: the
// tensor cores work on one while the warps work on the other.
// What stands in the rows of k and v past the kept ones only reaches their
// own lanes, which are not written.
template <int D>
__device__ __forceinline__ void keys_body(const Args& a, const Deal& deal, unsigned char* smem, int block, int blocks) {
  using L = Lay<D>;
  enum { FIXED_FULL, FIXED_EMPTY, S_FULL, P_FULL, DP_FULL, DS_FULL, ACC_FULL, ACC_EMPTY, ROW_FULL, ROW_READ = ROW_FULL + 2,
         FULL = ROW_READ + 2, EMPTY = FULL + STAGES, DRAIN = EMPTY + STAGES, NBAR };
  unsigned counts[NBAR];
#pragma unroll
  for (int i = 0; i < NBAR; ++i)
    counts[i] = (i == P_FULL || i == DS_FULL || i == ACC_EMPTY || i == ROW_READ || i == ROW_READ + 1) ? EW_WARPS : 1;
  Block k;
  if (!start<D>(smem, NBAR, counts, a.status, k)) return;
  const int ksplits = deal.ksplits, kper = deal.kper, kitems = deal.kitems;
  auto bar = [&](int i) { return k.bar0 + 8u * (uint32_t)i; };
  auto stage = [&](uint32_t i) { return k.base + (2u + i % STAGES) * L::BYTES; };
  const int L_all = a.G * a.qtiles;          // query tiles of a key head
  // query tiles of item it: none where the key tile has no kept key (dealt items have)
  auto share = [&](int it) -> int {
    if (!a.dealt && a.key_len != nullptr) {
      const int u = it / ksplits;
      if (u % a.ktiles * TILE >= item_len(a.key_len, a.Nk, u / (a.ktiles * a.Hkv), nullptr, false)) return 0;
    }
    return min(kper, L_all - it % ksplits * kper);
  };
  // item it: key tile kt of (b, hk), from query tile t0 on; b and the key tiles a head before it go on with it
  struct Walk { int b, before, count; };
  auto tiles_of = [&](int b) { return (item_len(a.key_len, a.Nk, b, nullptr, false) + TILE - 1) / TILE; };
  auto next = [&](Walk& w, int it, int& hk, int& kt, int& t0) {
    const int u = it / ksplits;
    if (!a.dealt) {
      w.b = u / (a.Hkv * a.ktiles);
      w.before = w.b * a.ktiles;
    } else {
      while (u >= a.Hkv * (w.before + w.count) && w.b + 1 < a.B) {
        w.before += w.count;
        w.count = tiles_of(++w.b);
      }
    }
    hk = (u - a.Hkv * w.before) / w.count;
    kt = (u - a.Hkv * w.before) % w.count;
    t0 = it % ksplits * kper;
  };

  if (k.warp < EW_WARPS) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (k.warp < EW_WARPS) {
    const int half = k.warp >> 2;
    const uint32_t tb = k.tmem + ((uint32_t)((k.warp & 3) * 32) << 16);
    const uint32_t sc = tb + 64u * (uint32_t)half, dc = tb + 128u + 64u * (uint32_t)half;
    uint32_t nt = 0, ni = 0;                 // tiles, items seen
    bool ok = true;
    auto wait = [&](int i, uint32_t parity) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(i), parity, a.status));
      fence_after();
      return ok;
    };
    auto arrive = [&](int i) {
      fence_before();
      __syncwarp();
      if (k.lane == 0) mbar_arrive(bar(i));
    };
    for (int it = block; ok && it < kitems; it += blocks) {
      const int tiles = share(it);
      if (tiles == 0) continue;
      for (int j = 0; j < tiles; ++j, ++nt) {
        // lse log2 e and D of the tile's queries: one value per column, read by all lanes at once
        const float4* lse4 = reinterpret_cast<const float4*>(smem + L::OFF_ROW + 1024 * (nt & 1)) + 16 * half;
        const float4* del4 = lse4 + 32;
        if (!wait(ROW_FULL + (nt & 1), (nt >> 1) & 1u) || !wait(S_FULL, nt & 1u)) break;
        uint32_t x[64], w[32];
        float p[64];
        tmem_ld32p(sc, x);
        tmem_ld32p(sc + 32u, x + 32);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 s = lse4[c];
          const uint64_t sl = f2(a.sl2, a.sl2);
          float u0, u1, u2, u3;
          unf2(ffma2(f2(__uint_as_float(x[4 * c]), __uint_as_float(x[4 * c + 1])), sl, f2(-s.x, -s.y)), u0, u1);
          unf2(ffma2(f2(__uint_as_float(x[4 * c + 2]), __uint_as_float(x[4 * c + 3])), sl, f2(-s.z, -s.w)), u2, u3);
          p[4 * c] = ex2(u0);
          p[4 * c + 1] = ex2(u1);
          p[4 * c + 2] = ex2(u2);
          p[4 * c + 3] = ex2(u3);
          w[2 * c] = pack2<false>(p[4 * c], p[4 * c + 1]);
          w[2 * c + 1] = pack2<false>(p[4 * c + 2], p[4 * c + 3]);
        }
        tmem_st32p(sc, w);
        tmem_st_wait();
        arrive(P_FULL);
        if (!wait(DP_FULL, nt & 1u)) break;
        tmem_ld32p(dc, x);
        tmem_ld32p(dc + 32u, x + 32);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 s = del4[c];
          const float d0 = p[4 * c] * (__uint_as_float(x[4 * c]) - s.x);
          const float d1 = p[4 * c + 1] * (__uint_as_float(x[4 * c + 1]) - s.y);
          const float d2 = p[4 * c + 2] * (__uint_as_float(x[4 * c + 2]) - s.z);
          const float d3 = p[4 * c + 3] * (__uint_as_float(x[4 * c + 3]) - s.w);
          w[2 * c] = pack2<false>(d0, d1);
          w[2 * c + 1] = pack2<false>(d2, d3);
        }
        tmem_st32p(dc, w);
        tmem_st_wait();
        arrive(DS_FULL);
        if (k.lane == 0) mbar_arrive(bar(ROW_READ + (nt & 1)));
      }
      // shares of dV (the first four warps) and dK
      if (!ok || !wait(ACC_FULL, ni++ & 1u)) break;
      float* dst = a.part + (((size_t)it * 2 + half) * TILE + (k.warp & 3) * 32 + k.lane) * D;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        tmem_ld32p(tb + 256u + 128u * (uint32_t)half + 32u * c, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 8) store32(dst + 32 * c + e, x + e);
      }
      arrive(ACC_EMPTY);
    }
    if (!ok) *k.abort_flag = 1;
  } else if (k.warp == TMA_WARP) {
    if (k.lane == 0) {
      uint32_t nf = 0, nk = 0, nr = 0;
      bool ok = true;
      Walk w = a.dealt ? Walk{deal.b, deal.before, tiles_of(deal.b)} : Walk{0, 0, a.ktiles};
      for (int it = block; ok && it < kitems; it += blocks) {
        const int tiles = share(it);
        if (tiles == 0) continue;
        int hk, kt, t0;
        next(w, it, hk, kt, t0);
        const int b = w.b;
        if (nf > 0) ok = mbar_wait(bar(FIXED_EMPTY), (nf - 1) & 1u, a.status);
        if (!ok || *k.abort_flag) { ok = false; break; }
        mbar_arrive_tx(bar(FIXED_FULL), 2 * L::BYTES);
#pragma unroll
        for (int x = 0; x < L::ATOMS; ++x) {
          tma_load_4d(k.base + x * L::ATOM, &a.k.map, 64 * x, kt * TILE, a.k.h_on ? hk : 0, a.k.b_on ? b : 0, bar(FIXED_FULL));
          tma_load_4d(k.base + L::BYTES + x * L::ATOM, &a.v.map, 64 * x, kt * TILE, a.v.h_on ? hk : 0, a.v.b_on ? b : 0, bar(FIXED_FULL));
        }
        ++nf;
        for (int j = 0; ok && j < 2 * tiles; ++j, ++nk) {
          // Q_0, dO_0, Q_1, dO_1, ...
          if (nk >= STAGES) ok = mbar_wait(bar(EMPTY + nk % STAGES), (nk / STAGES - 1) & 1u, a.status);
          if (!ok || *k.abort_flag) { ok = false; break; }
          const int t = t0 + (j >> 1), h = hk * a.G + t / a.qtiles, n = (t % a.qtiles) * TILE;
          load_tile<D>(stage(nk), (j & 1) ? a.dout : a.q, n, h, b, bar(FULL + nk % STAGES));
          if ((j & 1) == 0) {                // and the tile's lse and D
            const uint32_t i = nr & 1u, to = k.base + L::OFF_ROW + 1024u * i;
            if (nr >= 2) ok = mbar_wait(bar(ROW_READ + i), (nr / 2 - 1) & 1u, a.status);
            if (!ok) { ++nk; break; }
            const size_t at = ((size_t)b * a.Hq + h) * a.NqP + n;
            mbar_arrive_tx(bar(ROW_FULL + i), 1024);
            bulk_load(to, a.lse2 + at, 512, bar(ROW_FULL + i));
            bulk_load(to + 512, a.delta + at, 512, bar(ROW_FULL + i));
            ++nr;
          }
        }
      }
      if (nf > 0) mbar_wait(bar(FIXED_FULL), (nf - 1) & 1u, a.status);
      for (uint32_t x = nr > 2 ? nr - 2 : 0; x < nr; ++x) mbar_wait(bar(ROW_FULL + (x & 1u)), (x >> 1) & 1u, a.status);
      for (uint32_t x = nk > STAGES ? nk - STAGES : 0; x < nk; ++x) mbar_wait(bar(FULL + x % STAGES), (x / STAGES) & 1u, a.status);
      if (!ok) *k.abort_flag = 1;
    }
  } else if (k.warp == MMA_WARP) {
    uint32_t nk = 0, nt = 0, ni = 0;
    const uint32_t e = elect_one();
    bool ok = true;
    auto wait = [&](int i, uint32_t parity) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(i), parity, a.status));
      fence_after();
      return ok;
    };
    auto wait_stage = [&](uint32_t i) { return wait(FULL + i % STAGES, (i / STAGES) & 1u); };
    const uint32_t sK = k.base, sV = k.base + L::BYTES;
    for (int it = block; ok && it < kitems; it += blocks) {
      const int tiles = __shfl_sync(0xffffffffu, share(it), 0);
      if (tiles == 0) continue;
      if (!wait(FIXED_FULL, ni & 1u) || !wait_stage(nk)) break;
      product_nt<D>(e, k.tmem, sK, stage(nk), TILE);
      mma_commit_if(e, bar(S_FULL));
      if (!wait_stage(nk + 1)) break;
      product_nt<D>(e, k.tmem + 128u, sV, stage(nk + 1), TILE);
      mma_commit_if(e, bar(DP_FULL));
      for (int j = 0; j < tiles; ++j, ++nt, nk += 2) {
        const bool more = j + 1 < tiles;
        if (!wait(P_FULL, nt & 1u)) break;
        // the accumulators are this item's once the last item's have been read
        if (j == 0 && ni > 0 && !wait(ACC_EMPTY, (ni - 1) & 1u)) break;
        product_ts<D, 32>(e, k.tmem + 256u, k.tmem, stage(nk + 1), TILE / 16, j > 0);           // dV += P^T dO
        mma_commit_if(e, bar(EMPTY + (nk + 1) % STAGES));
        if (more) {
          if (!wait_stage(nk + 2)) break;
          product_nt<D>(e, k.tmem, sK, stage(nk + 2), TILE);
          mma_commit_if(e, bar(S_FULL));
        }
        if (!wait(DS_FULL, nt & 1u)) break;
        product_ts<D, 32>(e, k.tmem + 384u, k.tmem + 128u, stage(nk), TILE / 16, j > 0);        // dK += dS^T Q
        mma_commit_if(e, bar(EMPTY + nk % STAGES));
        if (more) {
          if (!wait_stage(nk + 3)) break;
          product_nt<D>(e, k.tmem + 128u, sV, stage(nk + 3), TILE);
          mma_commit_if(e, bar(DP_FULL));
        }
      }
      if (!ok) break;
      mma_commit_if(e, bar(FIXED_EMPTY));
      mma_commit_if(e, bar(ACC_FULL));
      ++ni;
    }
    if (!ok && k.lane == 0) *k.abort_flag = 1;
    mma_commit_if(e, bar(DRAIN));
    mbar_wait(bar(DRAIN), 0, a.status);
    __syncwarp();
  }
  finish(k);
}

// ------------------------------------------------------------------ dQ
// TMEM: S 0, dP 128, dS 256 and 320 (two tiles), dQ 384. Lanes are queries,
// columns keys. The warps take S and dP into registers and say so at once, and
// dS has columns of its own, so the tensor cores form the next tile's S and
// dP while the warps work on this one's; dQ of tile t is issued after S and dP
// of tile t + 1, across items too.
// Shared memory, seven tiles: one of dO, one of V, and
//  - more than two key tiles: two that hold an item's Q and then its dQ on the
//    way out (a TMA store: rows straight from registers, 256 bytes a lane, took
//    5,000 clocks a tile); three of K, in use from S to dQ (with two the next but
//    one's copy, which waits for dQ, was 1,300 clocks late);
//  - one or two key tiles (STAY): three of Q and dQ, because two made the next but
//    one's Q wait for the store, 2,000 clocks an item; two of K, copied when
//    the key head changes. A CTA's items then follow one another in a head.
// One TMA warp brings Q and dO (the next dO, which has to wait for its buffer, is
// asked into L2 meanwhile), one K and V. Four warps write dQ out.
template <int D, bool STAY>
__device__ __forceinline__ void rows_body(const Args& a, const Deal& deal, unsigned char* smem) {
  using L = Lay<D>;
  constexpr int ROW_TMA_WARP = 10;
  enum { Q_FULL = 0, Q_READ = 3, DS_FULL = 6, DO_FULL = 8, DO_READ, V_FULL, V_READ, S_FULL, S_READ, DP_FULL, DP_READ,
         ACC_FULL, ACC_READ, K_FULL, K_READ = K_FULL + 3, DRAIN = K_READ + 3, NBAR };
  unsigned counts[NBAR];
#pragma unroll
  for (int i = 0; i < NBAR; ++i)
    counts[i] = (i == S_READ || i == DP_READ || (i & ~1) == DS_FULL) ? EW_WARPS
                : i == ACC_READ ? 4
                : i >= Q_READ && i < Q_READ + 3 ? 2 : 1;       // Q: the MMAs and the store of dQ
  Block k;
  if (!start<D>(smem, NBAR, counts, a.status, k)) return;
  auto bar = [&](int i) { return k.bar0 + 8u * (uint32_t)i; };
  constexpr uint32_t NX = STAY ? 3 : 2, NK = STAY ? 2 : 3;
  auto sX = [&](uint32_t i) { return k.base + i % NX * L::BYTES; };
  const uint32_t sdO = k.base + NX * L::BYTES, sV = sdO + L::BYTES;
  // K of tile t of all, tile j of its item
  auto k_at = [&](uint32_t t, int j) { return STAY ? (uint32_t)j : t % NK; };
  auto sK = [&](uint32_t i) { return sV + (1u + i) * L::BYTES; };
  const int it0 = deal.first, step = deal.step, end = deal.end;
  // item: query tile qt of (b, h), key tiles [k0, k0 + tiles)
  auto item = [&](int it, int valid, int& b, int& h, int& qt, int& k0) -> int {
    const int split = it % a.qsplits, u = it / a.qsplits;
    qt = u % a.qtiles;
    h = u / a.qtiles % a.Hq;
    b = u / a.qtiles / a.Hq;
    const int all = (valid + TILE - 1) / TILE, per = (all + a.qsplits - 1) / a.qsplits;
    k0 = split * per;
    return max(0, min(per, all - k0));
  };
  auto kept = [&](int it) { return item_len(a.key_len, a.Nk, it / (a.qsplits * a.qtiles * a.Hq), nullptr, false); };
  // phase x of a barrier (of a pair of them: use x of the pair) as a whole warp
  bool ok = true;
  auto wait = [&](int i, uint32_t x) {
    ok = __all_sync(0xffffffffu, mbar_wait(bar(i), x & 1u, a.status));
    fence_after();
    return ok;
  };
  auto wait2 = [&](int i, uint32_t x) { return wait(i + (int)(x & 1u), x >> 1); };

  if (k.warp < EW_WARPS) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (k.warp < EW_WARPS) {
    const int half = k.warp >> 2, r = (k.warp & 3) * 32 + k.lane;
    const uint32_t tb = k.tmem + ((uint32_t)((k.warp & 3) * 32) << 16);
    const uint32_t sc = tb + 64u * (uint32_t)half, dc = sc + 128u;
    auto arrive = [&](int i) {
      fence_before();
      __syncwarp();
      if (k.lane == 0) mbar_arrive(bar(i));
    };
    uint32_t nt = 0;
    // lse log2 e and D of this thread's row, read an item ahead
    auto row = [&](int it) {
      if (it >= end) return make_float2(0.f, 0.f);
      const int u = it / a.qsplits;
      const size_t at = (size_t)u * TILE + r;            // item order is row order
      return make_float2(a.lse2[at], a.delta[at]);
    };
    float2 next = row(it0);
    for (int it = it0; ok && it < end; it += step) {
      int b, h, qt, k0;
      const int valid = kept(it);
      const int tiles = item(it, valid, b, h, qt, k0);
      const float lse = next.x, delta = next.y;
      next = row(it + step);
      for (int j = 0; j < tiles; ++j, ++nt) {
        const int left = valid - (k0 + j) * TILE - 64 * half;        // kept keys among this half's columns
        if (!wait(S_FULL, nt)) break;
        uint32_t x[64];
        tmem_ld32p(sc, x);
        tmem_ld32p(sc + 32u, x + 32);
        tmem_ld_wait();
        arrive(S_READ);
        float p[64];
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          unf2(ffma2(f2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), f2(a.sl2, a.sl2), f2(-lse, -lse)), p[c], p[c + 1]);
          p[c] = ex2(p[c]);
          p[c + 1] = ex2(p[c + 1]);
        }
        if (!wait(DP_FULL, nt)) break;
        tmem_ld32p(dc, x);
        tmem_ld32p(dc + 32u, x + 32);
        tmem_ld_wait();
        arrive(DP_READ);
#pragma unroll
        for (int c = 0; c < 64; ++c) p[c] *= __uint_as_float(x[c]) - delta;
        if (left < 64) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= left) p[c] = 0.f;
        }
        // dQ of tile nt - 2, the last reader of these columns, came before this dP
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) w[c] = pack2<false>(p[2 * c], p[2 * c + 1]);
        tmem_st32p(tb + 256u + 64u * (nt & 1u) + 32u * (uint32_t)half, w);
        tmem_st_wait();
        arrive(DS_FULL + (nt & 1));
      }
    }
  } else if (k.warp >= OUT_WARP0) {
    const int tid = threadIdx.x - 32 * OUT_WARP0;                    // this thread's row
    const uint32_t tb = k.tmem + ((uint32_t)((k.warp - OUT_WARP0) * 32) << 16);
    uint32_t ni = 0;
    for (int it = it0; it < end; it += step) {
      int b, h, qt, k0;
      const int tiles = item(it, kept(it), b, h, qt, k0);
      const int n = qt * TILE + tid;
      if (tiles == 0) {                                  // no keys, or an empty share of them
        if (a.qsplits > 1) {
          for (int c = 0; c < D; c += 4)
            *reinterpret_cast<float4*>(a.qpart + ((size_t)it * TILE + tid) * D + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        } else if (n < a.Nq) {
          for (int c = 0; c < D; c += 8)
            *reinterpret_cast<uint4*>(a.dq.data + 2 * (b * a.dq.b + h * a.dq.h + (int64_t)n * a.dq.n + c)) = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      if (ok) wait(ACC_FULL, ni);
      // the four warps go on together: they meet at a barrier
      if (!ok) k.abort_flag[1] = 1;
      asm volatile("bar.sync 2, 128;" ::: "memory");
      ok = k.abort_flag[1] == 0;
      if (!ok) break;
      const uint32_t to = sX(ni);                        // Q's tile: its last product is done
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        tmem_ld32p(tb + 384u + 32u * c, x);
        tmem_ld_wait();
        if (c == D / 32 - 1) {                           // dQ has been read
          fence_before();
          __syncwarp();
          if (k.lane == 0) mbar_arrive(bar(ACC_READ));
        }
        if (a.qsplits > 1) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) store32(a.qpart + ((size_t)it * TILE + tid) * D + 32 * c + e, x + e);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              w[y] = pack2<false>(__uint_as_float(x[8 * e + 2 * y]) * a.scale, __uint_as_float(x[8 * e + 2 * y + 1]) * a.scale);
            const int ch = 4 * c + e;
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                         ::"r"(to + (ch >> 3) * L::ATOM + tid * 128 + (((ch & 7) ^ (tid & 7)) << 4)), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
          }
        }
      }
      fence_proxy_async();
      asm volatile("bar.sync 2, 128;" ::: "memory");
      if (tid == 0) {
        if (a.qsplits == 1) {
#pragma unroll
          for (int x = 0; x < L::ATOMS; ++x)
            tma_store_4d(to + x * L::ATOM, &a.dqm.map, 64 * x, qt * TILE, a.dqm.h_on ? h : 0, a.dqm.b_on ? b : 0);
          tma_store_commit();
          tma_store_wait_read();
        }
        mbar_arrive(bar(Q_READ + ni % NX));
      }
      ++ni;
    }
  } else if (k.warp == TMA_WARP || k.warp == ROW_TMA_WARP) {
    if (k.lane == 0) {
      // the copy into a buffer, its use u, once use u - 1 has been read
      auto load = [&](int full, int read, uint32_t u, uint32_t dst, const TensorMap& m, int n, int h, int b) {
        if (u > 0) ok = mbar_wait(bar(read), (u - 1) & 1u, a.status);
        if (*k.abort_flag) ok = false;
        if (ok) load_tile<D>(dst, m, n, h, b, bar(full));
        return ok;
      };
      uint32_t x = 0, y = 0;                             // copies issued: Q and dO of items, or K and V of key tiles
      uint32_t k_uses[3] = {0, 0, 0};                    // uses of each K tile
      int last_head = -1;
      auto ahead = [&](int it) {
        if (it >= end) return;
        int b, h, qt, k0;
        if (item(it, kept(it), b, h, qt, k0) == 0) return;
#pragma unroll
        for (int c = 0; c < L::ATOMS; ++c)
          tma_prefetch_4d(&a.dout.map, 64 * c, qt * TILE, a.dout.h_on ? h : 0, a.dout.b_on ? b : 0);
      };
      for (int it = it0; ok && it < end; it += step) {
        int b, h, qt, k0;
        const int tiles = item(it, kept(it), b, h, qt, k0);
        if (tiles == 0) continue;
        if (k.warp == ROW_TMA_WARP) {
          ahead(it + step);
          if (!load(Q_FULL + x % NX, Q_READ + x % NX, x / NX, sX(x), a.q, qt * TILE, h, b)) break;
          ++x;
          if (!load(DO_FULL, DO_READ, y, sdO, a.dout, qt * TILE, h, b)) break;
          ++y;
        } else {
          const int head = b * a.Hkv + h / a.G;
          for (int j = 0; j < tiles; ++j) {
            if (!STAY || head != last_head) {
              const uint32_t i = k_at(x, j);
              if (!load(K_FULL + i, K_READ + i, k_uses[i], sK(i), a.k, (k0 + j) * TILE, h / a.G, b)) break;
              ++k_uses[i];
              ++x;
            }
            if (!load(V_FULL, V_READ, y, sV, a.v, (k0 + j) * TILE, h / a.G, b)) break;
            ++y;
          }
          last_head = head;
        }
      }
      // every copy has landed before this CTA's shared memory goes
      if (k.warp == ROW_TMA_WARP) {
        for (uint32_t u = x > NX ? x - NX : 0; u < x; ++u) mbar_wait(bar(Q_FULL + u % NX), (u / NX) & 1u, a.status);
        if (y > 0) mbar_wait(bar(DO_FULL), (y - 1) & 1u, a.status);
      } else {
        for (int i = 0; i < 3; ++i)
          if (k_uses[i] > 0) mbar_wait(bar(K_FULL + i), (k_uses[i] - 1) & 1u, a.status);
        if (y > 0) mbar_wait(bar(V_FULL), (y - 1) & 1u, a.status);
      }
    }
  } else if (k.warp == MMA_WARP) {
    uint32_t nt = 0, ns = 0, ni = 0;                     // tiles, items begun, items whose dQ is complete
    const uint32_t e = elect_one();
    // dQ += dS K of a tile
    struct Tile { uint32_t t, k; int steps; bool first, last; };
    auto issue_dq = [&](const Tile& p) {
      if (!wait2(DS_FULL, p.t)) return;
      // the accumulator is this item's once the last item's has been read
      if (p.first && ni > 0 && !wait(ACC_READ, ni - 1)) return;
      product_ts<D, 0>(e, k.tmem + 384u, k.tmem + 256u + 64u * (p.t & 1u), sK(p.k), p.steps, !p.first);
      if (!STAY) mma_commit_if(e, bar(K_READ + p.k));
      if (p.last) {
        mma_commit_if(e, bar(ACC_FULL));
        ++ni;
      }
    };
    Tile prev = {};
    bool have = false;
    uint32_t k_uses[2] = {0, 0};                         // copies of K that stay
    int last_head = -1, head_tiles = 0;
    for (int it = it0; ok && it < end; it += step) {
      int b, h, qt, k0;
      const int valid = __shfl_sync(0xffffffffu, kept(it), 0);
      const int tiles = item(it, valid, b, h, qt, k0);
      if (tiles == 0) continue;
      const int head = b * a.Hkv + h / a.G;
      const bool fresh = !STAY || head != last_head;     // K has been copied for this item
      if (STAY && fresh) {
        // the last head's K is done with once its last dQ is
        if (have) issue_dq(prev);
        if (!ok) break;
        have = false;
        for (int j = 0; j < head_tiles; ++j) mma_commit_if(e, bar(K_READ + j));
        head_tiles = tiles;
      }
      last_head = head;
      for (int j = 0; ok && j < tiles; ++j, ++nt) {
        const uint32_t ki = k_at(nt, j);
        const bool last = j == tiles - 1;
        const int keys = last ? valid - (k0 + j) * TILE : TILE;
        const int n = keys < TILE ? (keys + 15) & ~15 : TILE;
        if (j == 0 && !wait(Q_FULL + ns % NX, ns / NX)) break;
        if (fresh && !wait(K_FULL + ki, !STAY ? nt / NK : j == 0 ? k_uses[0]++ : k_uses[1]++)) break;
        if (fresh && n > keys) {
          // K's rows past the last kept key are zeroed, up to the K of dS K (0 * NaN is NaN)
          for (int x = k.lane; x < (n - keys) * (D / 8); x += 32) {
            const int row = keys + x / (D / 8), c = x % (D / 8);
            const uint32_t at = sK(ki) + (c >> 3) * L::ATOM + row * 128 + (((c & 7) ^ (row & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
          }
          fence_proxy_async();
          __syncwarp();
        }
        if (nt > 0 && !wait(S_READ, nt - 1)) break;
        product_nt<D>(e, k.tmem, sX(ns), sK(ki), n);
        mma_commit_if(e, bar(S_FULL));
        if (last) mma_commit_if(e, bar(Q_READ + ns % NX));
        if (j == 0 && !wait(DO_FULL, ns)) break;
        if (!wait(V_FULL, nt)) break;
        if (nt > 0 && !wait(DP_READ, nt - 1)) break;
        product_nt<D>(e, k.tmem + 128u, sdO, sV, n);
        mma_commit_if(e, bar(DP_FULL));
        mma_commit_if(e, bar(V_READ));
        if (last) mma_commit_if(e, bar(DO_READ));
        if (have) issue_dq(prev);
        prev = Tile{nt, ki, n / 16, j == 0, last};
        have = true;
      }
      ++ns;
    }
    if (ok && have) issue_dq(prev);
    mma_commit_if(e, bar(DRAIN));
    mbar_wait(bar(DRAIN), 0, a.status);
    __syncwarp();
  }
  if (!ok) *k.abort_flag = 1;
  finish(k);
}

// Blocks of dQ first, then of dK and dV: those begin as the first ones end.
template <int D>
__global__ void __launch_bounds__(THREADS, 1) main_kernel(const __grid_constant__ Args a, int row_blocks) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const bool rows = (int)blockIdx.x < row_blocks;
  const int block = rows ? blockIdx.x : blockIdx.x - row_blocks, blocks = rows ? row_blocks : gridDim.x - row_blocks;
  Deal deal;
  if (a.dealt) {
    Deal* dealt = reinterpret_cast<Deal*>(smem + Lay<D>::OFF_DEAL);
    wait_for_last();
    if (threadIdx.x < 32) deal_out(a, rows, block, blocks, dealt);
    __syncthreads();
    deal = *dealt;
  } else {
    const int per = (a.qitems + blocks - 1) / blocks;
    deal = Deal{a.ksplits, a.kper, a.kitems, 0, 0, block * per, min((block + 1) * per, a.qitems), 1, a.ktiles <= 2 && a.qsplits == 1};
  }
  if (!rows) keys_body<D>(a, deal, smem, block, blocks);
  else if (deal.stay) rows_body<D, true>(a, deal, smem);
  else rows_body<D, false>(a, deal, smem);
}

// ------------------------------------------------------------------ shares
// dK and dV: shares of a key added in order, eight values a thread; the lower
// 128 threads of a block dV, the upper ones dK. grid (keys / (1024 / d), Hkv, B).
template <int D>
__global__ void __launch_bounds__(256) sum_kernel(const __grid_constant__ Args a) {
  wait_for_last();
  let_next_start();
  const int hk = blockIdx.y, b = blockIdx.z, y = threadIdx.x >> 7, x = threadIdx.x & 127;
  const int n = blockIdx.x * (1024 / D) + x / (D / 8), c = 8 * (x % (D / 8));
  if (n >= a.Nk) return;
  int row = a.place ? a.place[(size_t)b * a.Nk + n] : n;
  const int len = item_len(a.key_len, a.Nk, b, nullptr, false);
  if (row >= len) row = -1;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (row >= 0) {
    const int before = a.dealt ? a.deal[4 + b] : b * a.ktiles, tiles = a.dealt ? (len + TILE - 1) / TILE : a.ktiles;
    const int splits = a.dealt ? a.deal[0] : a.ksplits;
    const size_t it = ((size_t)a.Hkv * before + (size_t)hk * tiles + row / TILE) * splits;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float4* src = reinterpret_cast<const float4*>(a.part + (((it + s) * 2 + y) * TILE + row % TILE) * D + c);
      const float4 u = src[0], w = src[1];
      v[0] += u.x; v[1] += u.y; v[2] += u.z; v[3] += u.w;
      v[4] += w.x; v[5] += w.y; v[6] += w.z; v[7] += w.w;
    }
  }
  const float f = y ? a.scale : 1.f;
  const View& o = y ? a.dk : a.dv;
  *reinterpret_cast<uint4*>(o.data + 2 * (b * o.b + hk * o.h + (int64_t)n * o.n + c)) =
      make_uint4(pack2<false>(v[0] * f, v[1] * f), pack2<false>(v[2] * f, v[3] * f), pack2<false>(v[4] * f, v[5] * f),
                 pack2<false>(v[6] * f, v[7] * f));
}

// dQ where a query tile's keys were split: four values a thread. grid (queries / (1024 / d), B * Hq).
template <int D>
__global__ void __launch_bounds__(256) sum_rows_kernel(const __grid_constant__ Args a) {
  wait_for_last();
  const int bh = blockIdx.y, b = bh / a.Hq, h = bh % a.Hq;
  const int n = blockIdx.x * (1024 / D) + threadIdx.x / (D / 4), c = 4 * (threadIdx.x % (D / 4));
  if (n >= a.Nq) return;
  const size_t it = ((size_t)bh * a.qtiles + n / TILE) * a.qsplits;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < a.qsplits; ++s) {
    const float4 u = *reinterpret_cast<const float4*>(a.qpart + ((it + s) * TILE + n % TILE) * D + c);
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  }
  *reinterpret_cast<uint2*>(a.dq.data + 2 * (b * a.dq.b + h * a.dq.h + (int64_t)n * a.dq.n + c)) =
      make_uint2(pack2<false>(v.x * a.scale, v.y * a.scale), pack2<false>(v.z * a.scale, v.w * a.scale));
}

struct Plan {
  size_t off_lse, off_delta, off_deal, off_part, off_qpart, bytes;
  int kslots;                                // shares of dK and dV there is room for
};

static Plan plan(const Problem& p, Args* a) {
  a->B = p.B; a->Hq = p.Hq; a->Hkv = p.Hkv; a->G = p.G; a->Nq = p.Nq; a->Nk = p.Nk;
  a->qtiles = (p.Nq + TILE - 1) / TILE;
  a->ktiles = (p.Nk + TILE - 1) / TILE;
  a->NqP = a->qtiles * TILE;
  const int units = p.B * p.Hkv * a->ktiles, L = p.G * a->qtiles, most = most_shares(units, L);
  float least = share_cost(units, L, 1);
  for (int x = 2; x <= most; ++x) least = std::min(least, share_cost(units, L, x));
  int ks = 1;
  while (share_cost(units, L, ks) > least * 1.02f) ++ks;
  a->kper = (L + ks - 1) / ks;
  a->ksplits = (L + a->kper - 1) / a->kper;
  a->kitems = units * a->ksplits;
  const int64_t rows = (int64_t)p.B * p.Hq * a->qtiles;
  a->qsplits = (int)std::max<int64_t>(1, std::min<int64_t>(a->ktiles, SM_COUNT / rows));
  a->qitems = (int)(rows * a->qsplits);
  Plan pl;
  size_t o = 0;
  auto take = [&](size_t n) { const size_t at = o; o = align_up(o + n); return at; };
  pl.off_lse = take((size_t)p.B * p.Hq * a->NqP * 4);
  pl.off_delta = take((size_t)p.B * p.Hq * a->NqP * 4);
  // (with lengths the kernel chooses the shares: as many as there may be)
  pl.kslots = (int)std::min<int64_t>(std::max(units, KSLOTS), (int64_t)units * L);
  pl.off_deal = take((4 + (size_t)p.B) * 4);
  pl.off_part = take((size_t)pl.kslots * 2 * TILE * p.d * 4);
  pl.off_qpart = take(a->qsplits > 1 ? (size_t)a->qitems * TILE * p.d * 4 : 0);
  pl.bytes = o;
  return pl;
}

template <int D>
static cudaError_t run(const Args& a, int key_blocks, const PackArgs& pack, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(main_kernel<D>, Lay<D>::SMEM, &done);
  if (e != cudaSuccess) return e;
  const int row_blocks = std::min(a.qitems, SM_COUNT);
  const int per_head = (a.NqP * (D / 64) + 127) / 128;
  const int64_t stat_blocks = (int64_t)per_head * a.B * a.Hq, all = stat_blocks + pack_blocks(pack);
  if (all > INT32_MAX) return cudaErrorInvalidValue;
  stat_kernel<D><<<(unsigned)all, 256, 0, s>>>(a, pack, per_head, (int)stat_blocks);
  cudaError_t l = cudaGetLastError();
  if (l == cudaSuccess)
    l = launch_behind(main_kernel<D>, dim3(row_blocks + key_blocks), THREADS, Lay<D>::SMEM, s, a, row_blocks);
  if (l == cudaSuccess) l = launch_behind(sum_kernel<D>, dim3((a.Nk * (D / 64) + 15) / 16, a.Hkv, a.B), 256, 0, s, a);
  if (l == cudaSuccess && a.qsplits > 1)
    l = launch_behind(sum_rows_kernel<D>, dim3((a.Nq * (D / 64) + 15) / 16, a.B * a.Hq), 256, 0, s, a);
  return l;
}

}  // namespace bwd

size_t bwd_workspace(const Problem& p) {
  bwd::Args a = {};
  return bwd::plan(p, &a).bytes;
}

cudaError_t launch_bwd(const Problem& p, const Gradients& g, const PackArgs& pack, void* ws, cudaStream_t s) {
  bwd::Args a = {};
  const bwd::Plan pl = bwd::plan(p, &a);
  if (!make_tensor_map(&a.q, p.q, p.B, p.Hq, p.Nq, p.d, false, bwd::TILE) ||
      !make_tensor_map(&a.k, p.k, p.B, p.Hkv, p.Nk, p.d, false, bwd::TILE) ||
      !make_tensor_map(&a.v, p.v, p.B, p.Hkv, p.Nk, p.d, false, bwd::TILE) ||
      !make_tensor_map(&a.dqm, g.dq, p.B, p.Hq, p.Nq, p.d, false, bwd::TILE) ||
      !make_tensor_map(&a.dout, g.dout, p.B, p.Hq, p.Nq, p.d, false, bwd::TILE))
    return cudaErrorInvalidValue;
  char* w = static_cast<char*>(ws);
  a.o = p.out; a.dov = g.dout; a.dq = g.dq; a.dk = g.dk; a.dv = g.dv;
  a.lse = g.lse;
  a.key_len = p.key_len;
  a.place = pack.mask ? pack.place : nullptr;
  a.status = p.status;
  a.scale = p.scale;
  a.sl2 = p.scale * 1.4426950408889634f;
  a.lse2 = reinterpret_cast<float*>(w + pl.off_lse);
  a.delta = reinterpret_cast<float*>(w + pl.off_delta);
  a.deal = reinterpret_cast<int*>(w + pl.off_deal);
  a.part = reinterpret_cast<float*>(w + pl.off_part);
  a.qpart = reinterpret_cast<float*>(w + pl.off_qpart);
  a.dealt = p.key_len != nullptr && (a.qitems > SM_COUNT || a.kitems > SM_COUNT);
  const int key_blocks = std::min(a.dealt ? pl.kslots : a.kitems, SM_COUNT);
  return p.d == 128 ? bwd::run<128>(a, key_blocks, pack, s) : bwd::run<64>(a, key_blocks, pack, s);
}

}  // namespace cross
}  // namespace spark
