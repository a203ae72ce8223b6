// Cross attention of few query rows (one token, a handful of latents).
//
// The rows of one key head are its G query heads times Nq tokens; a tile is 16
// of them, the M of one mma.sync.m16n8k16. With so few rows the work is
// reading K and V once, so the keys are split over blocks (until every SM has
// one) and, inside a block, over four warps that each stream 32 keys at a time
// through a ring of their own in shared memory (cp.async, no block barrier in
// the loop): 16 KB per step at d = 128, two steps in flight per warp. Each warp keeps
// the running maximum, sum and O of its keys; warps are joined in shared
// memory. Up to eight blocks of a tile form a cluster, if all of those fit on the
// GPU at once, and join over its shared memory, each a part of the rows' values;
// more blocks leave their shares in the workspace for join_kernel. Keys that are
// not kept are not read at all: cp.async fills their rows with zeros and their
// logits are -inf.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "cross.h"

namespace spark {
namespace cross {
namespace few {

constexpr int WARPS = 4, THREADS = 32 * WARPS;
constexpr int ROWS = 16, KEYS = 32, STAGES = 3;
constexpr int MIN_KEYS = WARPS * KEYS;       // fewest keys worth a block of their own
constexpr int CLUSTER = 8;                   // most blocks of a tile that join among themselves
// Weights are 2^(logit - reference). fp16 ends at 2^16 and loses what is below 2^-25,
// so its reference lies 7 below the maximum: weights down to 2^-32 of the largest
// one a warp has seen count in P V as they do in the sum. However large the maximum,
// its difference to a 7 is never rounded to more than 8 (15 would become 16).
template <bool H> constexpr float BELOW = H ? 7.f : 0.f;

struct Args {
  Problem p;
  int rows;                // G * Nq
  int tiles, splits;
  int stages;              // STAGES, or 1 where a warp has one step at most
  int cluster;             // the splits of a tile are a cluster, which joins them
  int per_split;           // keys per split, a multiple of KEYS
  float* part;             // [tiles * B * Hkv][splits][16][d], then the (max, sum) pairs
  float2* stat;
};

template <int D>
struct Lay {
  static constexpr int ROW = 2 * D;                       // bytes of a row
  static constexpr int Q = ROWS * ROW;
  static constexpr int TILE = KEYS * ROW;                 // of K or V
  static constexpr int smem(int stages) { return Q + WARPS * stages * 2 * TILE; }
};

// byte offset of 16-byte chunk c of row r: chunks XORed by the row, so that
// the eight rows an ldmatrix phase reads fall in eight bank groups
template <int D>
__device__ __forceinline__ uint32_t at(int r, int c) {
  return (uint32_t)(r * 2 * D + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool H>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (H)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool H>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  if constexpr (H) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool H>
__device__ __forceinline__ void put4(char* dst, const float4& v) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack<H>(in_range<H>(v.x), in_range<H>(v.y)),
                                            pack<H>(in_range<H>(v.z), in_range<H>(v.w)));
}
// v += f * x
__device__ __forceinline__ void add4(float4& v, float f, const float4& x) {
  v.x = fmaf(f, x.x, v.x);
  v.y = fmaf(f, x.y, v.y);
  v.z = fmaf(f, x.z, v.z);
  v.w = fmaf(f, x.w, v.w);
}
__device__ __forceinline__ float4 times(const float4& v, float f) { return make_float4(v.x * f, v.y * f, v.z * f, v.w * f); }

template <int D, bool H>
__global__ void __launch_bounds__(THREADS) kernel(const __grid_constant__ Args a) {
  using L = Lay<D>;
  constexpr int CH = D / 8;                  // 16-byte chunks of a row
  let_next_start();
  extern __shared__ __align__(128) unsigned char smem[];
  const Problem& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = blockIdx.x, split = blockIdx.y, bk = blockIdx.z;
  const int b = bk / p.Hkv, hk = bk % p.Hkv;
  const uint32_t sq = smem_u32(smem), ring = sq + L::Q + warp * a.stages * 2 * L::TILE;
  const int len = item_len(p.key_len, p.Nk, b, p.status, tid == 0 && tile == 0 && split == 0 && hk == 0);
  const int k_end = min(len, (split + 1) * a.per_split);

  // Q rows, zeros past the last
  for (int i = tid; i < ROWS * CH; i += THREADS) {
    const int r = i / CH, c = i % CH;
    const int row = tile * ROWS + r;
    const bool ok = row < a.rows;
    const int g = ok ? row / p.Nq : 0, n = ok ? row % p.Nq : 0;
    copy16(sq + at<D>(r, c), p.q.data + 2 * (b * p.q.b + (int64_t)(hk * p.G + g) * p.q.h + n * p.q.n + 8 * c), ok);
  }
  cp_async_commit();

  const char* kp = p.k.data + 2 * (b * p.k.b + hk * p.k.h);
  const char* vp = p.v.data + 2 * (b * p.v.b + hk * p.v.h);
  const uint8_t* mask = p.key_mask ? p.key_mask + (size_t)b * p.Nk : nullptr;
  // this warp's steps: keys first + i * MIN_KEYS .. + 32
  const int first = split * a.per_split + warp * KEYS;
  const int steps = k_end > first ? (k_end - first + MIN_KEYS - 1) / MIN_KEYS : 0;
  // issues the copies of step i; the bits of its kept keys
  auto stage_of = [&](int i) { return a.stages == STAGES ? i % STAGES : 0; };
  auto issue = [&](int i) -> uint32_t {
    uint32_t kept = 0;
    if (i < steps) {
      const int k0 = first + i * MIN_KEYS;
      const int j = k0 + lane;
      const bool take = j < k_end && (mask == nullptr || mask[j] != 0);
      kept = __ballot_sync(0xffffffffu, take);
      const uint32_t st = ring + stage_of(i) * 2 * L::TILE;
#pragma unroll
      for (int x = 0; x < CH; ++x) {
        const int e = x * 32 + lane, r = e / CH, c = e % CH;
        const bool ok = (kept >> r) & 1u;
        const int64_t key = ok ? k0 + r : 0;
        copy16(st + at<D>(r, c), kp + 2 * (key * p.k.n + 8 * c), ok);
        copy16(st + L::TILE + at<D>(r, c), vp + 2 * (key * p.v.n + 8 * c), ok);
      }
    }
    cp_async_commit();
    return kept;
  };
  uint32_t kept0 = issue(0), kept1 = issue(1);

  // Q fragments (the Q copies are the oldest group)
  cp_async_wait<2>();
  __syncthreads();
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k) ldsm4(qf[k], sq + at<D>(lane & 15, 2 * k + (lane >> 4)));

  const float sl2 = p.scale * 1.4426950408889634f;
  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};               // reference, sum

  for (int i = 0; i < steps; ++i) {
    const uint32_t kept2 = issue(i + 2);
    cp_async_wait<2>();
    __syncwarp();
    const uint32_t st = ring + stage_of(i) * 2 * L::TILE;
    float s[KEYS / 8][4];
#pragma unroll
    for (int n = 0; n < KEYS / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
      for (int n2 = 0; n2 < KEYS / 16; ++n2) {
        uint32_t kb[4];
        ldsm4(kb, st + at<D>(16 * n2 + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
        mma<H>(s[2 * n2], qf[k], kb[0], kb[1]);
        mma<H>(s[2 * n2 + 1], qf[k], kb[2], kb[3]);
      }
    }
    // running softmax; rows lane / 4 and lane / 4 + 8
    float mx[2] = {H ? -INFINITY : m[0], H ? -INFINITY : m[1]};
#pragma unroll
    for (int n = 0; n < KEYS / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = 8 * n + 2 * (lane & 3) + (e & 1);
        s[n][e] = ((kept0 >> key) & 1u) ? s[n][e] * sl2 : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      if constexpr (H) mx[r] = fmaxf(m[r], mx[r] - BELOW<H>);
      const float c = mx[r] == -INFINITY ? 1.f : exp2f(m[r] - mx[r]);
      m[r] = mx[r];
      l[r] *= c;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][2 * r] *= c;
        o[n][2 * r + 1] *= c;
      }
    }
    // (logits all -inf so far: exp2(-inf - 0) = 0; NaN stays NaN and reaches sum and O)
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int n = 0; n < KEYS / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = exp2f(s[n][e] - ref[e >> 1]);
        l[e >> 1] += s[n][e];
      }
#pragma unroll
    for (int k = 0; k < KEYS / 16; ++k) {
      const uint32_t pa[4] = {pack<H>(s[2 * k][0], s[2 * k][1]), pack<H>(s[2 * k][2], s[2 * k][3]),
                              pack<H>(s[2 * k + 1][0], s[2 * k + 1][1]), pack<H>(s[2 * k + 1][2], s[2 * k + 1][3])};
#pragma unroll
      for (int n2 = 0; n2 < D / 16; ++n2) {
        uint32_t vb[4];
        ldsm4t(vb, st + L::TILE + at<D>(16 * k + (lane & 15), 2 * n2 + (lane >> 4)));
        mma<H>(o[2 * n2], pa, vb[0], vb[1]);
        mma<H>(o[2 * n2 + 1], pa, vb[2], vb[3]);
      }
    }
    __syncwarp();                            // the stage is refilled by the next issue
    kept0 = kept1;
    kept1 = kept2;
  }
  cp_async_wait<0>();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  // join the warps: O and statistics in shared memory, over the rings
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);                           // [WARPS][ROWS][D]
  float2* ss = reinterpret_cast<float2*>(smem + WARPS * ROWS * D * 4);  // [WARPS][ROWS]
  const int r0 = lane >> 2;
  const int live = min(ROWS, a.rows - tile * ROWS);                     // rows of this tile
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    const int c = 8 * n + 2 * (lane & 3);
    if (r0 < live) *reinterpret_cast<float2*>(so + ((warp * ROWS + r0) * D + c)) = make_float2(o[n][0], o[n][1]);
    if (r0 + 8 < live) *reinterpret_cast<float2*>(so + ((warp * ROWS + r0 + 8) * D + c)) = make_float2(o[n][2], o[n][3]);
  }
  if ((lane & 3) == 0) {
    ss[warp * ROWS + r0] = make_float2(m[0], l[0]);
    ss[warp * ROWS + r0 + 8] = make_float2(m[1], l[1]);
  }
  __syncthreads();
  float* wf = so + WARPS * ROWS * D + 2 * WARPS * ROWS;                 // [WARPS][ROWS] weights of the join
  float2* js = reinterpret_cast<float2*>(wf + WARPS * ROWS);          // [ROWS] the block's statistics
  float* jo = reinterpret_cast<float*>(js + ROWS);                      // [ROWS][D] its O, for its cluster
  const size_t part = ((size_t)bk * a.tiles + tile) * a.splits + split;
  // output row r of the tile
  auto out_row = [&](int r, int& h, int& n) {
    const int row = tile * ROWS + r, g = row / p.Nq;
    n = row - g * p.Nq;
    h = hk * p.G + g;
  };
  auto write_lse = [&](int r, float m_, float l_) {
    int h, n;
    out_row(r, h, n);
    if (p.lse != nullptr)
      p.lse[((size_t)b * p.Hq + h) * p.Nq + n] = l_ == 0.f ? -INFINITY : (m_ + log2f(l_)) * 0.6931471805599453f;
  };
  if (tid < live) {
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, ss[w * ROWS + tid].x);
    float f[WARPS];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      f[w] = mm == -INFINITY ? 0.f : exp2f(ss[w * ROWS + tid].x - mm);
      ll += f[w] * ss[w * ROWS + tid].y;
    }
    const float norm = a.splits > 1 ? 1.f : (ll == 0.f ? 0.f : 1.f / ll);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) wf[w * ROWS + tid] = f[w] * norm;
    js[tid] = make_float2(mm, ll);
    if (a.splits > 1 && !a.cluster) a.stat[part * ROWS + tid] = make_float2(mm, ll);
    if (a.splits == 1) write_lse(tid, mm, ll);
  }
  __syncthreads();
  // four values a thread at a time
#pragma unroll 4
  for (int i = 4 * tid; i < live * D; i += 4 * THREADS) {
    const int r = i / D, c = i % D;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) add4(v, wf[w * ROWS + r], *reinterpret_cast<const float4*>(so + (w * ROWS + r) * D + c));
    if (a.cluster) {
      *reinterpret_cast<float4*>(jo + i) = v;
    } else if (a.splits > 1) {
      *reinterpret_cast<float4*>(a.part + part * ROWS * D + i) = v;
    } else {
      int h, n;
      out_row(r, h, n);
      put4<H>(p.out.data + 2 * (b * p.out.b + h * p.out.h + n * p.out.n + c), v);
    }
  }
  if (a.cluster) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();       // (1, splits, 1): rank = split
    cluster.sync();
    for (int i = 4 * (split * THREADS + tid); i < live * D; i += 4 * a.splits * THREADS) {
      const int r = i / D, c = i % D;
      float2 st[CLUSTER];
      float4 x[CLUSTER], v = make_float4(0.f, 0.f, 0.f, 0.f);
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int k = 0; k < CLUSTER; ++k) {                 // all on their way at once
        st[k] = k < a.splits ? *cluster.map_shared_rank(js + r, k) : make_float2(-INFINITY, 0.f);
        x[k] = k < a.splits ? *cluster.map_shared_rank(reinterpret_cast<float4*>(jo + i), k) : v;
      }
#pragma unroll
      for (int k = 0; k < CLUSTER; ++k) mm = fmaxf(mm, st[k].x);
#pragma unroll
      for (int k = 0; k < CLUSTER; ++k) {
        const float f = st[k].x == -INFINITY ? 0.f : exp2f(st[k].x - mm);
        ll += f * st[k].y;
        add4(v, f, x[k]);
      }
      int h, n;
      out_row(r, h, n);
      put4<H>(p.out.data + 2 * (b * p.out.b + h * p.out.h + n * p.out.n + c), times(v, ll == 0.f ? 0.f : 1.f / ll));
      if (c == 0) write_lse(r, mm, ll);
    }
    cluster.sync();                                       // no block leaves while another reads its shared memory
  }
}

// Joins the splits of a row: grid (rows, B * Hkv). D / 4 threads have the row's
// values, 4 groups (d = 64: 8) of them a share each of the splits, added in
// shared memory in order.
template <int D, bool H>
__global__ void __launch_bounds__(THREADS) join_kernel(const __grid_constant__ Args a) {
  constexpr int LANES = D / 4, GROUPS = THREADS / LANES;
  __shared__ float4 sum[GROUPS][LANES];
  __shared__ float den[GROUPS];
  wait_for_last();
  const Problem& p = a.p;
  const int row = blockIdx.x, bk = blockIdx.y, x = threadIdx.x % LANES, y = threadIdx.x / LANES, c = 4 * x;
  const int b = bk / p.Hkv, hk = bk % p.Hkv;
  const size_t unit = (size_t)bk * a.tiles + row / ROWS;
  const int r = row % ROWS;
  float mm = -INFINITY, ll = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = x; s < a.splits; s += LANES) mm = fmaxf(mm, a.stat[(unit * a.splits + s) * ROWS + r].x);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
  for (int s = y; s < a.splits; s += GROUPS) {
    const float2 st = a.stat[(unit * a.splits + s) * ROWS + r];
    const float f = exp2f(st.x - ref);
    ll += f * st.y;
    add4(v, f, *reinterpret_cast<const float4*>(a.part + ((unit * a.splits + s) * ROWS + r) * D + c));
  }
  sum[y][x] = v;
  if (x == 0) den[y] = ll;
  __syncthreads();
  if (y != 0) return;
#pragma unroll
  for (int i = 1; i < GROUPS; ++i) {
    add4(v, 1.f, sum[i][x]);
    ll += den[i];
  }
  const int g = row / p.Nq, n = row % p.Nq, h = hk * p.G + g;
  put4<H>(p.out.data + 2 * (b * p.out.b + h * p.out.h + n * p.out.n + c), times(v, ll == 0.f ? 0.f : 1.f / ll));
  if (c == 0 && p.lse != nullptr)
    p.lse[((size_t)b * p.Hq + h) * p.Nq + n] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
}

static Args plan(const Problem& p, void* ws) {
  Args a;
  a.p = p;
  a.rows = p.G * p.Nq;
  a.tiles = (a.rows + ROWS - 1) / ROWS;
  const int64_t units = (int64_t)a.tiles * p.B * p.Hkv;
  // split the keys until every SM has a block (its rings fill an SM's shared
  // memory); or, where that many clusters of blocks fit at two an SM, down to one step
  // a warp, which needs no ring (one token over 512 keys, 64 heads: 4 blocks a head)
  const int64_t most = (p.Nk + MIN_KEYS - 1) / MIN_KEYS;
  const bool short_keys = most <= CLUSTER && units * most <= ((most & (most - 1)) == 0 ? 2 : 1) * SM_COUNT;
  const int64_t want = short_keys ? most : std::max<int64_t>(1, std::min<int64_t>(most, SM_COUNT / units));
  a.per_split = (int)((most + want - 1) / want) * MIN_KEYS;
  a.splits = (p.Nk + a.per_split - 1) / a.per_split;
  a.stages = a.per_split == MIN_KEYS ? 1 : STAGES;
  // Clusters that do not fit in one round (16 of eight blocks: 37 us where the first
  // round takes 15; sizes between leave SMs of a GPC empty) are no clusters
  a.cluster = a.splits > 1 && a.splits <= CLUSTER &&
              (short_keys || a.splits == 2 || units * a.splits <= (a.splits > 4 ? 64 : 128));
  a.part = static_cast<float*>(ws);
  a.stat = reinterpret_cast<float2*>(a.part + units * a.splits * ROWS * p.d);
  return a;
}

template <int D, bool H>
static cudaError_t run(const Args& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(kernel<D, H>, Lay<D>::smem(STAGES), &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.tiles, a.splits, a.p.B * a.p.Hkv);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = Lay<D>::smem(a.stages);
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = attr.val.clusterDim.z = 1;
  attr.val.clusterDim.y = a.splits;
  cfg.attrs = &attr;
  cfg.numAttrs = a.cluster;
  const cudaError_t l = cudaLaunchKernelEx(&cfg, kernel<D, H>, a);
  if (l != cudaSuccess) return l;
  if (a.splits == 1 || a.cluster) return cudaSuccess;
  return launch_behind(join_kernel<D, H>, dim3(a.rows, a.p.B * a.p.Hkv), THREADS, 0, s, a);
}

}  // namespace few

size_t few_workspace(const Problem& p) {
  const few::Args a = few::plan(p, nullptr);
  return a.splits > 1 && !a.cluster ? (size_t)a.tiles * p.B * p.Hkv * a.splits * few::ROWS * (p.d * sizeof(float) + sizeof(float2)) : 0;
}

void few_keys(const Problem& p, int64_t* keys) {
  const few::Args a = few::plan(p, nullptr);
  const int at_once = (p.d == 128 ? 1 : 2) + (a.stages == 1);       // blocks an SM holds
  const int64_t blocks = (int64_t)a.tiles * p.B * p.Hkv * a.splits, wave = (int64_t)at_once * SM_COUNT;
  *keys = (blocks + wave - 1) / wave * (a.per_split + 256);
}

cudaError_t launch_few(const Problem& p, void* ws, cudaStream_t s) {
  const few::Args a = few::plan(p, ws);
  if (p.d == 128) return p.fp16 ? few::run<128, true>(a, s) : few::run<128, false>(a, s);
  return p.fp16 ? few::run<64, true>(a, s) : few::run<64, false>(a, s);
}

}  // namespace cross
}  // namespace spark
