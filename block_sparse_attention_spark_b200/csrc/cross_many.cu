// Cross attention of many query rows on the sm_100a tensor cores.
//
// One persistent CTA per SM. A work item is two tiles of 128 query rows of one
// key head (each tile's rows are tokens of one query head) against all the
// kept keys of that head, or against one share of them when there are fewer
// tiles than SMs (the shares are joined by join_kernel). K and V stream in
// tiles of 128 keys through one ring (four 32 KB stages at d = 128) that both
// row tiles read, which halves the L2 traffic of one tile alone (at 72,576
// queries by 512 keys one row tile per CTA would ask 13 TB/s of it).
//
// TMEM (512 columns): S of the two tiles at 0 and 128, O at 256 and 384; P
// (16 bits, two keys a column) overwrites the first half of its S. One warp
// issues, in turn for the two tiles, P_j V_j and then S_{j+1} = Q K_{j+1}^T:
// while the tensor cores work for one tile, the other tile's four warps (one
// thread per row) turn S into P and hand it over in two halves of 64 keys. MMAs
// of one thread complete in issue order, so S_{j+1} arriving says that P_j V_j
// is done: O may be rescaled, the next tile's first S may overwrite P, without
// further barriers. Four more warps write O out while the softmax is at the
// next item, whose Q (a third buffer) and K are already there.
//
// The softmax is online with a lazy reference: the row's reference maximum
// moves (and O is rescaled in TMEM) only when a logit passes it by 8 (fp16: 6)
// in powers of two. Sums and maxima are float32; P is rounded to the tensors'
// type, the operand type of the MMA. The last tile of an item runs with N (and for P V, K) cut to the
// next multiple of 16 of its keys; V rows between are zeroed in shared memory,
// whatever they hold, because 0 * NaN is NaN.
//
// Measured (bf16, d = 128): 9,472 queries of 8 heads over 2,048 keys 71 us =
// 1,120 TFLOP/s; 72,576 queries of 40 heads over 512 keys 727 us = 1,046 (850 us
// in a loop of 0.15 s); over 77 keys 331 us = 4.5 TB/s. What bounds it: the chain
// S -> P -> P V of a row tile (about 2,100 clocks of softmax and 1,000 to 1,300 of
// MMAs and hand-overs a tile, the other row tile beside it), and the 1,000 W power cap: the SMs
// run at 1.56 GHz under it. Leaving out every exponential gained 2%, so the
// exponentials are not worth moving to the FMA pipe (tried: 2 to 13% slower).
//
// Every wait is bounded (2 s): on expiry the status word is set, copies and
// MMAs in flight are waited for (bounded again), TMEM is freed, the kernel returns.
#include <cuda_fp16.h>

#include "common.cuh"
#include "cross.h"
#include "cross_tc.cuh"

namespace spark {
namespace cross {
namespace many {

using namespace tc;

constexpr int ROWS = 128, KEYS = 128, SLOTS = 2;
// warps: softmax of tile 0 and of tile 1 (four each), TMA, MMA, two idle, output (four)
constexpr int SM_WARPS = 4 * SLOTS, TMA_WARP = SM_WARPS, MMA_WARP = SM_WARPS + 1, OUT_WARP0 = SM_WARPS + 4;
constexpr int THREADS = 32 * (SM_WARPS + 8);
// A thread is launched with 128 registers; the softmax needs about 180, the
// others little: 256 * 184 + 256 * 72 = 512 * 128.
constexpr int LAUNCH_REGS = 128, SOFTMAX_REGS = 184, OTHER_REGS = 72;
static_assert(SM_WARPS * 32 * SOFTMAX_REGS + 256 * OTHER_REGS <= THREADS * LAUNCH_REGS, "registers the block owns");
constexpr int QBUFS = 3;                     // a row tile's Q can load while both current ones are in use
// Log2 units: how far a logit passes the largest one that the reference was taken
// from before the reference moves, and how far the reference lies below that one.
// fp16 ends at 2^16 and loses what is below 2^-25, so its weights are formed up to
// 2^15: those down to 2^-34 of the row's largest count in P V as they do in the sum.
template <bool H> constexpr float LAZY = H ? 6.0f : 8.0f;
template <bool H> constexpr float BELOW = H ? 9.0f : 0.0f;
// (not below it where the logit is so large that the difference would be rounded
// noticeably, and weights could pass 2^16)
template <bool H>
__device__ __forceinline__ float reference(float m) { return H && fabsf(m) < 1048576.f ? m - BELOW<H> : m; }
constexpr uint32_t O_COL = 256;

struct Args {
  TensorMap q, k, v;
  View out;
  const int32_t* key_len;
  float* lse;
  int* status;
  int B, Hq, Hkv, G, Nq, Nk;
  int tokens;                                // row tiles per head
  int pairs;                                 // work items per key head: ceil(G * tokens / 2)
  int splits;
  int items;                                 // B * Hkv * pairs * splits
  float sl2;                                 // scale * log2 e
  int wide;                                  // out rows take 32-byte stores
  float* part;                               // splits > 1: [items][2][128][d] unnormalised O
  float2* stat;                              // [items][2][128] (reference, sum)
};

template <int D>
struct Lay {
  static constexpr int ATOMS = D / 64;
  static constexpr int ATOM = 128 * 128;               // 128 rows x 64 values
  static constexpr int TILE = ATOM * ATOMS;            // Q tile = K tile = V tile
  static constexpr int STAGES = D == 128 ? 4 : 8;      // of K and V
  static constexpr int OFF_STAT = (QBUFS + STAGES) * TILE;   // (reference, sum) of both tiles' rows
  static constexpr int OFF_BAR = OFF_STAT + SLOTS * ROWS * 8;
  static constexpr int SMEM = OFF_BAR + 512;
  static_assert(SMEM <= 232448, "shared memory of a block");
};

// A work item: its key head, its share of the keys and the two row tiles.
struct Item {
  int b, hk, pair, k0, valid, tiles;         // first key tile, kept keys of the item, key tiles of the share
};
__device__ __forceinline__ int item_batch(const Args& a, int it) { return it / (a.splits * a.pairs * a.Hkv); }
__device__ __forceinline__ Item item_of(const Args& a, int it, int valid) {
  Item w;
  const int split = it % a.splits, u = it / a.splits;
  w.pair = u % a.pairs;
  const int bk = u / a.pairs;
  w.b = bk / a.Hkv;
  w.hk = bk % a.Hkv;
  w.valid = valid;
  const int all = (w.valid + KEYS - 1) / KEYS, per = (all + a.splits - 1) / a.splits;
  w.k0 = split * per;
  w.tiles = max(0, min(per, all - w.k0));
  return w;
}

__device__ __forceinline__ int kept(const Args& a, int it) {
  return item_len(a.key_len, a.Nk, item_batch(a, it), nullptr, false);
}

template <int D, bool H>
__global__ void __launch_bounds__(THREADS, 1) kernel(const __grid_constant__ Args a) {
  using L = Lay<D>;
  enum { S_FULL = 0, P_FULL = 2, O_FULL = 6, O_EMPTY = 8, L_FULL = 10, L_EMPTY = 12, Q_FULL = 14, Q_EMPTY = Q_FULL + QBUFS,
         FULL = Q_EMPTY + QBUFS, EMPTY = FULL + L::STAGES, DRAIN = EMPTY + L::STAGES, NBAR };
  constexpr uint32_t FMT = H ? 0u : 1u;
  constexpr uint32_t IDESC = (1u << 4) | (FMT << 7) | (FMT << 10) | ((uint32_t)(ROWS >> 4) << 24);
  constexpr uint32_t IDESC_O = IDESC | (1u << 16) | ((uint32_t)(D >> 3) << 17);
  static_assert(8 * NBAR + 8 <= 512, "barriers");
  extern __shared__ __align__(1024) unsigned char smem[];
  float2* stat_sh = reinterpret_cast<float2*>(smem + L::OFF_STAT);       // [SLOTS][ROWS]
  uint32_t* tmem_sh = reinterpret_cast<uint32_t*>(smem + L::OFF_BAR + 8 * NBAR);
  int& abort_sh = *reinterpret_cast<int*>(tmem_sh + 1);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);     // uniform
  const uint32_t base = smem_u32(smem), bar0 = base + L::OFF_BAR;
  if (base & 1023u) {                        // the swizzle needs it; the launch guarantees it
    if (tid == 0) set_status(a.status, STATUS_BAD_INPUT);
    return;
  }
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  // O has barriers of its own: the next item's first S may arrive before this one's
  // O has been looked at, and a parity wait must not fall two phases behind
  auto s_full = [&](int s) { return bar(S_FULL + s); };
  auto p_full = [&](int s, int half) { return bar(P_FULL + 2 * s + half); };   // P of the lower, the upper 64 keys
  auto o_full = [&](int s) { return bar(O_FULL + s); };
  auto o_empty = [&](int s) { return bar(O_EMPTY + s); };
  auto l_full = [&](int s) { return bar(L_FULL + s); };
  auto l_empty = [&](int s) { return bar(L_EMPTY + s); };
  auto q_full = [&](uint32_t x) { return bar(Q_FULL + x % QBUFS); };
  auto q_empty = [&](uint32_t x) { return bar(Q_EMPTY + x % QBUFS); };
  auto full = [&](uint32_t x) { return bar(FULL + x % L::STAGES); };
  auto empty = [&](uint32_t x) { return bar(EMPTY + x % L::STAGES); };
  auto sQ = [&](uint32_t x) { return base + (x % QBUFS) * L::TILE; };
  auto sKV = [&](uint32_t x) { return base + (QBUFS + x % L::STAGES) * L::TILE; };

  if (tid == 0) {
    abort_sh = 0;
    for (int i = 0; i < NBAR; ++i) mbar_init(bar(i), (i >= P_FULL && i < O_FULL) || (i >= O_EMPTY && i < Q_FULL) ? 4 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_sh)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  wait_for_last();
  let_next_start();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_sh, 0);
  const int row_tiles = a.G * a.tokens;

  if (warp < SM_WARPS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
  if (warp < SM_WARPS) {
    // ------------------------------------------------ softmax and output, one thread per row
    const int s = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t tb = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t sc = tb + 128u * (uint32_t)s, oc = tb + O_COL + 128u * (uint32_t)s;
    const uint64_t sc2 = f2(a.sl2, a.sl2);
    uint32_t ns = 0, ni = 0;                 // S tiles, items seen
    bool ok = true;
    if (a.key_len != nullptr && blockIdx.x == 0 && s == 0)
      for (int b = r; b < a.B; b += ROWS) item_len(a.key_len, a.Nk, b, a.status, true);
    for (int it = blockIdx.x; ok && it < a.items; it += gridDim.x) {
      const Item w = item_of(a, it, kept(a, it));
      if (w.tiles == 0 || 2 * w.pair + s >= row_tiles) continue;
      float m = -INFINITY, limit = -INFINITY, l = 0.f;      // reference, the logit that moves it, sum
      for (int j = 0; ok && j < w.tiles; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(s_full(s), ns & 1u, a.status));
        ++ns;
        if (!ok) break;
        fence_after();
        // moves the row's reference to mt, and its O and sum with it, if it has none or mt passes it
        auto move = [&](float mt) {
          float corr = 1.f;
          if (m == -INFINITY) {
            m = reference<H>(mt);
            limit = mt + LAZY<H>;
          } else if (mt > limit) {
            limit = mt + LAZY<H>;
            mt = reference<H>(mt);
            corr = ex2(m - mt);
            l *= corr;
            m = mt;
          }
          if (__any_sync(0xffffffffu, corr != 1.f)) {
            // P_{j-1} V_{j-1} is done (S_j came after it), P_j V_j not issued yet
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              tmem_ld32p(oc + 32u * cc, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              tmem_st32p(oc + 32u * cc, o);
            }
          }
        };
        auto hand_over = [&](int hf) {
          tmem_st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(s, hf));   // the MMAs of these 64 keys need not wait for the others
        };
        const int valid = w.valid - (w.k0 + j) * KEYS;
        if (valid < KEYS) {
          // an item's last tile: 32 keys at a time, only as far as the MMAs go (two passes
          // over S; P of keys 32 c.. goes to columns 16 c.., whose S has been read)
          const int chunks = (((valid + 15) & ~15) + 31) / 32;
          float mt = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            uint32_t x[32];
            tmem_ld32p(sc + 32u * c, x);
            tmem_ld_wait();
            const int left = valid - 32 * c;
            if (left >= 32) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) mt = max3(mt, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e < left) mt = fmaxf(mt, __uint_as_float(x[e]));
            }
          }
          move(mt * a.sl2);
          const float ref = m == -INFINITY ? 0.f : m;        // logits all -inf: exp2(-inf - 0) = 0
          float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            uint32_t x[32], pw[16];
            tmem_ld32p(sc + 32u * c, x);
            tmem_ld_wait();
            const int left = valid - 32 * c;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float u = ex2(fmaf(__uint_as_float(x[e]), a.sl2, -ref));
              if (e >= left) u = 0.f;
              x[e] = __float_as_uint(u);
              rs[e & 3] += u;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) pw[e] = pack2<H>(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
            tmem_st16p(sc + 16u * c, pw);
          }
          l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
          hand_over(0);
          if (lane == 0) mbar_arrive(p_full(s, 1));
          continue;
        }
        uint32_t sv[KEYS];
#pragma unroll
        for (int c = 0; c < KEYS / 32; ++c) tmem_ld32p(sc + 32u * c, sv + 32 * c);
        tmem_ld_wait();
        float mc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mc[i] = fmaxf(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
#pragma unroll
        for (int c = 16; c < KEYS; c += 16)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mc[i] = max3(mc[i], __uint_as_float(sv[c + 2 * i]), __uint_as_float(sv[c + 2 * i + 1]));
        move(fmaxf(fmaxf(max3(mc[0], mc[1], mc[2]), max3(mc[3], mc[4], mc[5])), fmaxf(mc[6], mc[7])) * a.sl2);
        // (no branch on a row's reference: the stores are collective, and rows of a warp may differ in it)
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t nm2 = f2(-ref, -ref);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pw[32];
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float u0, u1;
            unf2(ffma2(f2(__uint_as_float(sv[64 * hf + c]), __uint_as_float(sv[64 * hf + c + 1])), sc2, nm2), u0, u1);
            u0 = ex2(u0);
            u1 = ex2(u1);
            acc[(c >> 1) & 3] = fadd2(acc[(c >> 1) & 3], f2(u0, u1));
            pw[c >> 1] = pack2<H>(u0, u1);
          }
          tmem_st32p(sc + 32u * hf, pw);
          hand_over(hf);
        }
        float r0, r1, r2, r3;
        unf2(fadd2(acc[0], acc[1]), r0, r1);
        unf2(fadd2(acc[2], acc[3]), r2, r3);
        l += (r0 + r2) + (r1 + r3);
      }
      if (!ok) break;
      // for the output warps, once they have the last item's
      if (ni > 0) ok = __all_sync(0xffffffffu, mbar_wait(l_empty(s), (ni - 1) & 1u, a.status));
      if (!ok) break;
      stat_sh[s * ROWS + r] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(l_full(s));
      ++ni;
    }
    if (!ok) atomicExch(&abort_sh, 1);
  } else if (warp >= OUT_WARP0) {
    // ------------------------------------------------ output: O of each row tile while the softmax is at the next item
    const int r = (warp - OUT_WARP0) * 32 + lane;
    const uint32_t tb = tmem + ((uint32_t)((warp - OUT_WARP0) * 32) << 16);
    uint32_t ni[SLOTS] = {0, 0};
    bool ok = true;
    for (int it = blockIdx.x; ok && it < a.items; it += gridDim.x) {
      const Item w = item_of(a, it, kept(a, it));
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        const int t = 2 * w.pair + s;
        if (!ok || t >= row_tiles) break;
        float m = -INFINITY, l = 0.f;
        if (w.tiles > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(l_full(s), ni[s] & 1u, a.status) && mbar_wait(o_full(s), ni[s] & 1u, a.status));
          if (!ok) break;
          fence_after();
          const float2 st = stat_sh[s * ROWS + r];
          m = st.x;
          l = st.y;
          __syncwarp();
          if (lane == 0) mbar_arrive(l_empty(s));
          ++ni[s];
        }
        const uint32_t oc = tb + O_COL + 128u * (uint32_t)s;
        const int g = t / a.tokens, n = (t % a.tokens) * ROWS + r, h = w.hk * a.G + g;
        const bool live = n < a.Nq;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float* part = a.part + ((size_t)it * SLOTS + s) * ROWS * D + (size_t)r * D;
        char* dst = a.out.data + 2 * (w.b * a.out.b + h * a.out.h + (int64_t)n * a.out.n);
        uint64_t squares = 0;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          if (w.tiles > 0) {
            tmem_ld32p(oc + 32u * cc, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (cc == D / 32 - 1 && w.tiles > 0) {           // O has been read
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty(s));
          }
          if (a.splits > 1) {
            if (live) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) store32(part + 32 * cc + e, o + e);
            }
          } else if (live) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint64_t x = f2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
              if constexpr (H) {
                squares = ffma2(x, x, squares);
                float lo, hi;
                unf2(fmul2(x, f2(inv, inv)), lo, hi);
                pk[e] = pack2<H>(lo, hi);
              } else {
                pk[e] = pack2<H>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
              }
            }
            if (a.wide) {
              store32(dst + 64 * cc, pk);
              store32(dst + 64 * cc + 32, pk + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint4*>(dst + 64 * cc + 16 * e) = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
            }
          }
        }
        if constexpr (H) {
          // in_range for the row as it was written, where its squares (infinite if a value is)
          // add up to more than the largest one's 65504^2. In pairs on the FMA pipe: 77 keys of
          // 72,576 queries 333 us (327 without); maxima of all values instead 351, clamping them 375
          float s0, s1;
          unf2(squares, s0, s1);
          const float all = (s0 + s1) * inv * inv;
          if (live && a.splits == 1 && all > 4.29e9f && all < INFINITY) {
#pragma unroll 1
            for (int c = 0; c < D; ++c) {
              uint16_t& x = reinterpret_cast<uint16_t*>(dst)[c];
              if ((x & 0x7fffu) == 0x7c00u) x -= 1;      // infinity: the type's largest value
            }
          }
        }
        if (live && a.splits > 1) a.stat[((size_t)it * SLOTS + s) * ROWS + r] = make_float2(m, l);
        if (live && a.splits == 1 && a.lse != nullptr)
          a.lse[((size_t)w.b * a.Hq + h) * a.Nq + n] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      }
    }
    if (!ok) atomicExch(&abort_sh, 1);
  } else if (warp == TMA_WARP) {
    // ------------------------------------------------ loads: Q of tile 0, K_0, Q of tile 1, V_0, K_1, V_1, ...
    if (lane == 0) {
      uint32_t nk = 0, nq = 0;               // tiles issued
      bool ok = true;
      auto load = [&](uint32_t dst, const TensorMap& m, int n, int h, int b, uint32_t full_bar, uint32_t empty_bar,
                      bool used, uint32_t parity) {
        if (used) ok = mbar_wait(empty_bar, parity, a.status);
        if (!ok || *(volatile int*)&abort_sh) { ok = false; return; }
        mbar_arrive_tx(full_bar, L::TILE);
#pragma unroll
        for (int x = 0; x < L::ATOMS; ++x)
          tma_load_4d(dst + x * L::ATOM, &m.map, 64 * x, n, m.h_on ? h : 0, m.b_on ? b : 0, full_bar);
      };
      for (int it = blockIdx.x; ok && it < a.items; it += gridDim.x) {
        const Item w = item_of(a, it, kept(a, it));
        for (int j = 0; ok && j < 2 * w.tiles; ++j) {
          if (j < SLOTS && 2 * w.pair + j < row_tiles) {
            const int t = 2 * w.pair + j;
            load(sQ(nq), a.q, (t % a.tokens) * ROWS, w.hk * a.G + t / a.tokens, w.b, q_full(nq), q_empty(nq),
                 nq >= QBUFS, (nq / QBUFS - 1) & 1u);
            if (!ok) break;
            ++nq;
          }
          load(sKV(nk), (j & 1) ? a.v : a.k, (w.k0 + (j >> 1)) * KEYS, w.hk, w.b, full(nk), empty(nk), nk >= L::STAGES,
               (nk / L::STAGES - 1) & 1u);
          if (!ok) break;
          ++nk;
        }
      }
      // every copy has landed before this CTA's shared memory goes
      for (uint32_t x = nq > QBUFS ? nq - QBUFS : 0; x < nq; ++x) mbar_wait(q_full(x), (x / QBUFS) & 1u, a.status);
      for (uint32_t x = nk > L::STAGES ? nk - L::STAGES : 0; x < nk; ++x) mbar_wait(full(x), (x / L::STAGES) & 1u, a.status);
      if (!ok) atomicExch(&abort_sh, 1);
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------ MMAs (warp-uniform, one lane's predicate on)
    uint32_t nk = 0, nq = 0, np[SLOTS] = {0, 0}, no[SLOTS] = {0, 0};
    const uint32_t e = elect_one();
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, a.status));
      fence_after();
      return ok;
    };
    // S of a slot from K in stage x, n keys (a multiple of 16)
    auto issue_s = [&](int s, uint32_t q, uint32_t x, int n) {
      const uint64_t dq = sdesc(sQ(q), 16, 1024), dk = sdesc(sKV(x), 16, 1024);
      const uint32_t idesc = IDESC | ((uint32_t)(n >> 3) << 17);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint64_t o = (uint64_t)(((ks >> 2) * L::ATOM + (ks & 3) * 32) >> 4);
        mma_f16_if(e, tmem + 128u * (uint32_t)s, dq + o, dk + o, idesc, ks > 0 ? 1u : 0u);
      }
      mma_commit_if(e, s_full(s));
    };
    for (int it = blockIdx.x; ok && it < a.items; it += gridDim.x) {
      const Item w = item_of(a, it, __shfl_sync(0xffffffffu, kept(a, it), 0));
      if (w.tiles == 0) continue;
      const int slots = 2 * w.pair + 1 < row_tiles ? 2 : 1;
      const int last = w.valid - (w.k0 + w.tiles - 1) * KEYS;       // keys of the last tile
      auto n16 = [&](int j) { return j == w.tiles - 1 && last < KEYS ? (last + 15) & ~15 : KEYS; };
      for (int s = 0; ok && s < slots; ++s) {
        if (!wait(q_full(nq + s), ((nq + s) / QBUFS) & 1u)) break;
        if (s == 0 && !wait(full(nk), (nk / L::STAGES) & 1u)) break;
        issue_s(s, nq + s, nk, n16(0));
        if (w.tiles == 1) mma_commit_if(e, q_empty(nq + s));
        if (s == slots - 1) mma_commit_if(e, empty(nk));
      }
      ++nk;
      for (int j = 0; ok && j < w.tiles; ++j) {
        // V_j in stage nk, K_{j+1} in the next one
        const bool more = j + 1 < w.tiles;
        if (!wait(full(nk), (nk / L::STAGES) & 1u)) break;
        const int n = n16(j);
        if (!more && (last & 15) != 0) {
          // rows of V past the last kept key, up to the MMA's K
          for (int x = lane; x < (n - last) * (D / 8); x += 32) {
            const int row = last + x / (D / 8), c = x % (D / 8);
            const uint32_t at = sKV(nk) + (c >> 3) * L::ATOM + row * 128 + (((c & 7) ^ (row & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
          }
          fence_proxy_async();
          __syncwarp();
        }
        if (more && !wait(full(nk + 1), ((nk + 1) / L::STAGES) & 1u)) break;
        for (int s = 0; ok && s < slots; ++s) {
          // O is this item's once the last one's has been read
          if (j == 0 && no[s]++ > 0 && !wait(o_empty(s), no[s] & 1u)) break;
          const uint64_t dv = sdesc(sKV(nk), L::ATOM, 1024);
          const uint32_t pa = tmem + 128u * (uint32_t)s, od = tmem + O_COL + 128u * (uint32_t)s;
          if (!wait(p_full(s, 0), np[s] & 1u)) break;
          if (n == KEYS) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts_if(e, od, pa + 8u * kk, dv + (uint64_t)((kk * 2048) >> 4), IDESC_O, (kk > 0 || j > 0) ? 1u : 0u);
            if (!wait(p_full(s, 1), np[s] & 1u)) break;
#pragma unroll
            for (int kk = 4; kk < 8; ++kk)
              mma_ts_if(e, od, pa + 8u * kk, dv + (uint64_t)((kk * 2048) >> 4), IDESC_O, 1u);
          } else {
            if (!wait(p_full(s, 1), np[s] & 1u)) break;
            for (int kk = 0; kk < n / 16; ++kk)
              mma_ts_if(e, od, pa + 8u * kk, dv + (uint64_t)((kk * 2048) >> 4), IDESC_O, (kk > 0 || j > 0) ? 1u : 0u);
          }
          ++np[s];
          if (s == slots - 1) mma_commit_if(e, empty(nk));
          if (!more) {
            mma_commit_if(e, o_full(s));
          } else {
            issue_s(s, nq + s, nk + 1, n16(j + 1));
            if (j + 2 == w.tiles) mma_commit_if(e, q_empty(nq + s));
            if (s == slots - 1) mma_commit_if(e, empty(nk + 1));
          }
        }
        nk += more ? 2 : 1;
      }
      nq += slots;
    }
    if (!ok && lane == 0) atomicExch(&abort_sh, 1);
    // one more commit: its arrival means that every MMA has completed
    mma_commit_if(e, bar(DRAIN));
    mbar_wait(bar(DRAIN), 0, a.status);
    __syncwarp();
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == MMA_WARP)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

// Joins the shares of a row: WARPS warps a row, 8 / WARPS rows a block, grid (row
// tiles * 128 rows, B * Hkv). Eight warps where there are more than 32 shares, or more
// than 4 of so few rows that the blocks run at once: 16,384 keys of 4 heads in 74
// shares 16.6 us (one warp a row 29.5), 8 heads' 64 rows over 8,192 keys 18.3 (18.9);
// 256 rows of the same 26.6 (25.1).
template <int D, bool H, int WARPS>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a) {
  constexpr int PER = 8 / WARPS, BLOCKS = ROWS / PER, V = D / 32;
  __shared__ float stat[8];
  __shared__ float sum[8][D];
  wait_for_last();
  const int t = blockIdx.x / BLOCKS, bk = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = bk / a.Hkv, hk = bk % a.Hkv;
  const int g = t / a.tokens, h = hk * a.G + g;
  const size_t first = ((size_t)bk * a.pairs + t / 2) * a.splits;    // item of share 0
  const int r = (blockIdx.x % BLOCKS) * PER + warp / WARPS, n = (t % a.tokens) * ROWS + r;
  if (n >= a.Nq) return;                     // (with several warps a row, the whole block)
  auto row = [&](int s) { return ((first + s) * SLOTS + (t & 1)) * ROWS + r; };
  float m = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) m = fmaxf(m, a.stat[row(s)].x);
  m = warp_maxf(m);
  float l = 0.f, o[V];
#pragma unroll
  for (int e = 0; e < V; ++e) o[e] = 0.f;
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 4
  for (int s = warp % WARPS; s < a.splits; s += WARPS) {
    const float2 st = a.stat[row(s)];
    const float f = exp2f(st.x - ref);
    l += f * st.y;
    const float* src = a.part + row(s) * D + lane * V;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = fmaf(f, src[e], o[e]);
  }
  if constexpr (WARPS > 1) {
    stat[warp] = l;
#pragma unroll
    for (int e = 0; e < V; ++e) sum[warp][lane * V + e] = o[e];
    __syncthreads();
    if (warp % WARPS != 0) return;
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      l += stat[warp + w];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] += sum[warp + w][lane * V + e];
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  char* dst = a.out.data + 2 * (b * a.out.b + h * a.out.h + (int64_t)n * a.out.n) + lane * (D / 16);
#pragma unroll
  for (int e = 0; e < D / 64; ++e)
    *reinterpret_cast<uint32_t*>(dst + 4 * e) = pack2<H>(in_range<H>(o[2 * e] * inv), in_range<H>(o[2 * e + 1] * inv));
  if (lane == 0 && a.lse != nullptr)
    a.lse[((size_t)b * a.Hq + h) * a.Nq + n] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

static void plan(const Problem& p, Args* a) {
  a->B = p.B; a->Hq = p.Hq; a->Hkv = p.Hkv; a->G = p.G; a->Nq = p.Nq; a->Nk = p.Nk;
  a->tokens = (p.Nq + ROWS - 1) / ROWS;
  a->pairs = (p.G * a->tokens + 1) / 2;
  const int64_t units = (int64_t)p.B * p.Hkv * a->pairs;
  const int tiles = (p.Nk + KEYS - 1) / KEYS;
  // shares of the keys: only while that many items still run at once
  int splits = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, SM_COUNT / std::max<int64_t>(units, 1)));
  a->splits = splits;
  a->items = (int)(units * splits);
}

static size_t workspace(const Problem& p, const Args& a) {
  return a.splits > 1 ? (size_t)a.items * SLOTS * ROWS * (p.d * sizeof(float) + sizeof(float2)) : 0;
}

template <int D, bool H>
static cudaError_t run(const Args& a, bool packed, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(kernel<D, H>, Lay<D>::SMEM, &done);
  if (e != cudaSuccess) return e;
  const int blocks = std::min(a.items, SM_COUNT);
  cudaError_t l;
  if (packed) {                              // behind this call's packing; else what came before is not known
    l = launch_behind(kernel<D, H>, dim3(blocks), THREADS, Lay<D>::SMEM, s, a);
  } else {
    kernel<D, H><<<blocks, THREADS, Lay<D>::SMEM, s>>>(a);
    l = cudaGetLastError();
  }
  if (l != cudaSuccess || a.splits == 1) return l;
  const int64_t rows = (int64_t)a.B * a.Hq * a.Nq;
  if (a.splits > 32 || (a.splits > 4 && rows <= 8 * SM_COUNT)) 
    return launch_behind(join_kernel<D, H, 8>, dim3(a.G * a.tokens * ROWS, a.B * a.Hkv), 256, 0, s, a);
  return launch_behind(join_kernel<D, H, 1>, dim3(a.G * a.tokens * (ROWS / 8), a.B * a.Hkv), 256, 0, s, a);
}

}  // namespace many

size_t many_workspace(const Problem& p) {
  many::Args a = {};
  many::plan(p, &a);
  return many::workspace(p, a);
}

void many_keys(const Problem& p, int64_t* keys, int* shares) {
  many::Args a = {};
  many::plan(p, &a);
  const int tiles = (p.Nk + many::KEYS - 1) / many::KEYS;
  *keys = (int64_t)((a.items + SM_COUNT - 1) / SM_COUNT) * ((tiles + a.splits - 1) / a.splits) * many::KEYS;
  *shares = a.splits;
}

cudaError_t launch_many(const Problem& p, bool packed, void* ws, cudaStream_t s) {
  many::Args a = {};
  many::plan(p, &a);
  if (!make_tensor_map(&a.q, p.q, p.B, p.Hq, p.Nq, p.d, p.fp16, many::ROWS) ||
      !make_tensor_map(&a.k, p.k, p.B, p.Hkv, p.Nk, p.d, p.fp16, many::KEYS) ||
      !make_tensor_map(&a.v, p.v, p.B, p.Hkv, p.Nk, p.d, p.fp16, many::KEYS))
    return cudaErrorInvalidValue;
  a.out = p.out;
  a.key_len = p.key_len;
  a.lse = p.lse;
  a.status = p.status;
  a.sl2 = p.scale * 1.4426950408889634f;
  a.wide = ((uintptr_t)p.out.data % 32 == 0 && p.out.b % 16 == 0 && p.out.h % 16 == 0 && p.out.n % 16 == 0);
  a.part = static_cast<float*>(ws);
  a.stat = reinterpret_cast<float2*>(a.part + (size_t)a.items * many::SLOTS * many::ROWS * p.d);
  if (p.d == 128) return p.fp16 ? many::run<128, true>(a, packed, s) : many::run<128, false>(a, packed, s);
  return p.fp16 ? many::run<64, true>(a, packed, s) : many::run<64, false>(a, packed, s);
}

}  // namespace cross
}  // namespace spark
