// Rotary positions with several axes, the per-head RMS norm before them, and
// their gradient.
//
//   n_i = x_i r w_i, r = 1 / sqrt(mean x^2 + eps);  (u, v) of each pair becomes
//   (u cos - v sin, u sin + v cos) with the angle of its axis' position.
//   Gradient: dn = R^T dy, g = dn w, dx = r (g - x r^2 mean(x g)),
//   dw = sum over rows of dn x r.
//
// A few operations per value read and written: bound by HBM. One pass: a
// thread owns eight values (four pairs) of one token's row, forms their four
// cosines and sines once (turns in 64 bits: position times frequency, reduced
// to [-1/2, 1/2], then 32-bit sincospi), and walks heads of q or of k with
// them in registers, four rows (some gradients: two) in flight. A warp's 32 lanes hold
// two (d = 128) or four (d = 64) rows, so the mean of squares is a shuffle over
// 16 or 8 lanes. A block holds 256 / (d / 8) tokens of one tensor; heads are
// split over blocks when tokens alone do not fill the GPU.
//
// What counts is how many warps are resident: the forward kernel held to 64
// registers (four blocks an SM) reads and writes 72,576 tokens of 80 heads
// (bf16, d = 128) in 461 us = 6.4 TB/s, with 80 registers in 510; a software
// pipeline of the loads (more in flight a thread, fewer warps) took 508 to 750.
// Heads a block: as many as leave three blocks an SM in all (2 x 3,555 tokens of
// 24 + 8 heads, fp16: 26.4 us; for six blocks 29.1, for 24, where the angles are
// formed for four heads at a time, 41; 3 x 1,517 tokens of 24 heads 11.0 against
// 14.5 for six). The gradient's blocks with partial sums, 888: 87 us, 444: 88, 2,664: 90.
// 16-bit values are converted in pairs: value by value those took 31 us, in pairs 29.
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "views.h"

namespace spark {
namespace rotary {

constexpr int THREADS = 256;
constexpr int ROWS = 4;                    // rows in flight per thread (heads are shared out in fours)
constexpr int BWD_BLOCKS = SM_COUNT * 6;   // blocks of the gradient where it has partial sums of dw

struct Tensor {
  View in, x, out;                     // forward: rows, -, results; gradient: of the results, rows, of the rows
  const void* weight;
  int H, splits, per_split;            // heads, their shares, heads per share
  int items;                           // token tiles * splits
};
struct Args {
  Tensor t[2];                         // q, k
  const float* pos;                    // [B, N, axes] or null
  float* part;                         // [blocks][d] partial sums of dw
  int blocks_q;                        // blocks of q; the others are k's
  int N, axes;
  int npairs;                          // R / 2
  int tiles;                           // token tiles per batch item
  int grid[3];
  float eps;
  double start[3], scale[3];
  double freq[64];                     // turns per unit of position, by pair
  unsigned char axis[64];
};

// where a lane's eight values stand in the row: pair j of the lane is values
// 2j, 2j+1 of the register array
enum { CONTIG = 0, SPLIT4 = 1, SINGLES = 2 };

// Two 16-bit values of a word.
template <typename T>
__device__ __forceinline__ void unpack(uint32_t w, float& lo, float& hi) {
  if constexpr (sizeof(T) == 2 && !std::is_same<T, __half>::value) {
    lo = bf_lo(w);
    hi = bf_hi(w);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  }
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t w;
  if constexpr (std::is_same<T, __half>::value) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// A lane's eight values of a row as they come: four words of two (16-bit types)
// or eight. Value order: pair j of the lane is values 2j, 2j+1 of get and put;
// with SPLIT4 the first half of the words holds the pairs' first values.
template <typename T, int MODE>
struct Row {
  static constexpr int WORDS = 2 * sizeof(T);          // 4 or 8
  uint32_t w[WORDS];
  __device__ __forceinline__ static const T* first(const T* row, int l, int npairs) {
    return row + (MODE == SPLIT4 && 4 * l < npairs ? 4 * l : 8 * l);
  }
  __device__ __forceinline__ static const T* second(const T* row, int l, int npairs) {
    return row + (MODE == SPLIT4 && 4 * l < npairs ? npairs + 4 * l : 8 * l + 4);
  }
  __device__ __forceinline__ void load(const T* row, int l, int npairs) {
    if constexpr (MODE == SINGLES) {
      T v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = row[at(l, j, npairs)];
#pragma unroll
      for (int j = 0; j < WORDS; ++j) w[j] = reinterpret_cast<const uint32_t*>(v)[j];
    } else if constexpr (MODE == CONTIG) {
#pragma unroll
      for (int j = 0; j < WORDS; j += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(row + 8 * l) + j);
        w[j] = x.x; w[j + 1] = x.y; w[j + 2] = x.z; w[j + 3] = x.w;
      }
    } else if constexpr (WORDS == 4) {
      const uint2 x = *reinterpret_cast<const uint2*>(first(row, l, npairs));
      const uint2 y = *reinterpret_cast<const uint2*>(second(row, l, npairs));
      w[0] = x.x; w[1] = x.y; w[2] = y.x; w[3] = y.y;
    } else {
      const uint4 x = *reinterpret_cast<const uint4*>(first(row, l, npairs));
      const uint4 y = *reinterpret_cast<const uint4*>(second(row, l, npairs));
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
      w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
    }
  }
  __device__ __forceinline__ void store(T* row, int l, int npairs) const {
    if constexpr (MODE == SINGLES) {
      T v[8];
#pragma unroll
      for (int j = 0; j < WORDS; ++j) reinterpret_cast<uint32_t*>(v)[j] = w[j];
#pragma unroll
      for (int j = 0; j < 8; ++j) row[at(l, j, npairs)] = v[j];
    } else if constexpr (MODE == CONTIG) {
#pragma unroll
      for (int j = 0; j < WORDS; j += 4)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(row + 8 * l) + j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
    } else if constexpr (WORDS == 4) {
      *reinterpret_cast<uint2*>(const_cast<T*>(first(row, l, npairs))) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(const_cast<T*>(second(row, l, npairs))) = make_uint2(w[2], w[3]);
    } else {
      *reinterpret_cast<uint4*>(const_cast<T*>(first(row, l, npairs))) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(const_cast<T*>(second(row, l, npairs))) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < WORDS; ++j) w[j] = 0u;
  }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (WORDS == 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[MODE == SPLIT4 ? 2 * (j & 3) + (j >> 2) : j] = __uint_as_float(w[j]);
    } else if constexpr (MODE == SPLIT4) {
      unpack<T>(w[0], f[0], f[2]);
      unpack<T>(w[1], f[4], f[6]);
      unpack<T>(w[2], f[1], f[3]);
      unpack<T>(w[3], f[5], f[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) unpack<T>(w[j], f[2 * j], f[2 * j + 1]);
    }
  }
  __device__ __forceinline__ void put(const float* f) {
    if constexpr (WORDS == 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(f[MODE == SPLIT4 ? 2 * (j & 3) + (j >> 2) : j]);
    } else if constexpr (MODE == SPLIT4) {
      w[0] = pack<T>(f[0], f[2]);
      w[1] = pack<T>(f[4], f[6]);
      w[2] = pack<T>(f[1], f[3]);
      w[3] = pack<T>(f[5], f[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack<T>(f[2 * j], f[2 * j + 1]);
    }
  }
  // index in the row of value j
  __device__ __forceinline__ static int at(int l, int j, int npairs) {
    if constexpr (MODE == CONTIG) return 8 * l + j;
    if constexpr (MODE == SPLIT4)
      return 4 * l < npairs ? ((j & 1) ? npairs : 0) + 4 * l + (j >> 1) : 8 * l + ((j & 1) ? 4 : 0) + (j >> 1);
    const int i = 4 * l + (j >> 1);      // pairs past R / 2 are the kept values in turn
    return i < npairs ? i + ((j & 1) ? npairs : 0) : 2 * i + (j & 1);
  }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Turns the lane's pairs; sign -1: backwards. A pair past R / 2 is kept (not
// multiplied by 1 and 0: its values may be infinite).
template <int SIGN>
__device__ __forceinline__ void turn(float* f, const float* c, const float* s, unsigned live) {
  if (live == 15u) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float u = f[2 * j], v = f[2 * j + 1], sj = SIGN * s[j];
      f[2 * j] = fmaf(u, c[j], -v * sj);
      f[2 * j + 1] = fmaf(u, sj, v * c[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float u = f[2 * j], v = f[2 * j + 1], sj = SIGN * s[j];
      if ((live >> j) & 1u) {
        f[2 * j] = fmaf(u, c[j], -v * sj);
        f[2 * j + 1] = fmaf(u, sj, v * c[j]);
      }
    }
  }
}

template <typename T, int D, int MODE, bool NORM>
__device__ __forceinline__ void forward_row(Row<T, MODE>& x, const float* c, const float* s, const float* w,
                                            unsigned live, float eps) {
  float f[8];
  x.get(f);
  if constexpr (NORM) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
    const float r = rsqrtf(row_sum<D / 8>(ss) * (1.f / D) + eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= r * w[j];
  }
  turn<1>(f, c, s, live);
  x.put(f);
}

// y: gradient of the row's result, becomes the gradient of the row x.
template <typename T, int D, int MODE, bool NORM>
__device__ __forceinline__ void backward_row(Row<T, MODE>& y, const Row<T, MODE>& x, const float* c, const float* s,
                                             const float* w, unsigned live, float eps, float* dw) {
  float f[8];
  y.get(f);
  turn<-1>(f, c, s, live);
  if constexpr (NORM) {
    float xs[8], ss = 0.f, xg = 0.f;
    x.get(xs);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ss = fmaf(xs[j], xs[j], ss);
      xg = fmaf(xs[j], f[j] * w[j], xg);
    }
    ss = row_sum<D / 8>(ss);
    xg = row_sum<D / 8>(xg);
    const float r = rsqrtf(ss * (1.f / D) + eps);
    const float t = r * r * xg * (1.f / D);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[j] = fmaf(f[j], xs[j] * r, dw[j]);
      f[j] = fmaf(r * w[j], f[j], -(xs[j] * (r * t)));
    }
  }
  y.put(f);
}

// The heads [h0, h1) of a tensor at one token.
template <typename T, int D, int MODE, bool BWD, bool NORM>
__device__ __forceinline__ void heads(const Tensor& t, int b, int n, int h0, int h1, int l, int npairs, float eps,
                                      const float* c, const float* s, unsigned live, bool active, float* dw) {
  // gradient: two rows of 32-bit values, or of scattered ones, fill the registers;
  // with four of 16 bits instead of two 87 against 91 us (16 heads of 32,256,
  // norm) and 227 against 250 (80 heads of 36,288, none: 6.5 TB/s)
  constexpr int UNROLL = BWD && (sizeof(T) == 4 || MODE == SINGLES) ? 2 : ROWS;
  float w[8];
  if constexpr (NORM) {
    Row<T, MODE> wr;
    wr.load(static_cast<const T*>(t.weight), l, npairs);
    wr.get(w);
  }
  const T* pi = reinterpret_cast<const T*>(t.in.data) + b * t.in.b + n * t.in.n;
  const T* px = BWD && NORM ? reinterpret_cast<const T*>(t.x.data) + b * t.x.b + n * t.x.n : nullptr;
  T* po = reinterpret_cast<T*>(t.out.data) + b * t.out.b + n * t.out.n;
  int h = h0;
  for (; h + UNROLL <= h1; h += UNROLL) {
    Row<T, MODE> r[UNROLL], rx[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      r[u].load(pi + (h + u) * t.in.h, l, npairs);
      if constexpr (BWD && NORM) rx[u].load(px + (h + u) * t.x.h, l, npairs);
    }
    // idle lanes add zeros to dw: in place, the row they follow may be its gradient already.
    // (Cleared words cost nothing, a predicate on each sum 3 to 9%: 87 -> 89, 149 -> 164 us value by value)
    if (BWD && NORM && !active) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) r[u].clear();
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if constexpr (BWD) backward_row<T, D, MODE, NORM>(r[u], rx[u], c, s, w, live, eps, dw);
      else forward_row<T, D, MODE, NORM>(r[u], c, s, w, live, eps);
      if (active) r[u].store(po + (h + u) * t.out.h, l, npairs);
    }
  }
  for (; h < h1; ++h) {
    Row<T, MODE> r, rx;
    r.load(pi + h * t.in.h, l, npairs);
    if constexpr (BWD && NORM) rx.load(px + h * t.x.h, l, npairs);
    if (BWD && NORM && !active) r.clear();
    if constexpr (BWD) backward_row<T, D, MODE, NORM>(r, rx, c, s, w, live, eps, dw);
    else forward_row<T, D, MODE, NORM>(r, c, s, w, live, eps);
    if (active) r.store(po + h * t.out.h, l, npairs);
  }
}

// NORMED: some tensor has a weight. Blocks an SM: the gradient without a norm at
// four (64 registers), with one at three (at four some forms spill: 98 against
// 91 us for 16 heads of 32,256 in bf16, 167 against 143 for 36,288 in fp32).
// SINGLES is for being right, not fast: 2-byte accesses, and with a norm it spills
// (forward 88 to 156 bytes a thread, gradient 56 to 100). 72,576 tokens of 80 heads,
// norm, bf16: 1,076 us for R = 126 where R = 128 takes 468, gradient 1,274 (773);
// fp32, 40 heads: 799 (446).
template <typename T, int D, int MODE, bool BWD, bool NORMED>
__global__ void __launch_bounds__(THREADS, BWD && NORMED ? 3 : 4) kernel(const __grid_constant__ Args a) {
  constexpr int LPR = D / 8, TOK = THREADS / LPR;
  __shared__ double freq[64];
  __shared__ unsigned char axis[64];
  const int tid = threadIdx.x, l = tid % LPR;
  if (tid < 64) {
    freq[tid] = a.freq[tid];
    axis[tid] = a.axis[tid];
  }
  __syncthreads();
  const bool second = (int)blockIdx.x >= a.blocks_q;
  const Tensor& t = a.t[second];
  const int first = blockIdx.x - (second ? a.blocks_q : 0), step = second ? gridDim.x - a.blocks_q : a.blocks_q;
  float dw[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = 0.f;
  for (int it = first; it < t.items; it += step) {
    const int split = it % t.splits, tile = it / t.splits;
    const int b = tile / a.tiles, tok = (tile % a.tiles) * TOK + tid / LPR;
    const bool active = tok < a.N;
    const int n = active ? tok : a.N - 1;              // idle lanes follow the last token, unwritten
    // this lane's four angles
    double p[3] = {0.0, 0.0, 0.0};
    if (a.pos != nullptr) {
      const float* pp = a.pos + ((size_t)b * a.N + n) * a.axes;
#pragma unroll
      for (int x = 0; x < 3; ++x)
        if (x < a.axes) p[x] = (double)pp[x];
    } else {
      int rest = n;                                    // axes past the last have extent 1
#pragma unroll
      for (int x = 2; x >= 0; --x) {
        p[x] = (double)(rest % a.grid[x]);
        rest /= a.grid[x];
      }
    }
#pragma unroll
    for (int x = 0; x < 3; ++x) p[x] = a.start[x] + a.scale[x] * p[x];
    float c[4], s[4];
    unsigned live = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = 4 * l + j;
      c[j] = 1.f;
      s[j] = 0.f;
      if (i < a.npairs) {
        live |= 1u << j;
        const int ax = axis[i];
        double t = (ax == 0 ? p[0] : ax == 1 ? p[1] : p[2]) * freq[i];
        t -= rint(t);
        sincospif((float)(2.0 * t), &s[j], &c[j]);
      }
    }
    const int h0 = split * t.per_split, h1 = min(h0 + t.per_split, t.H);
    if (NORMED && t.weight != nullptr)
      heads<T, D, MODE, BWD, NORMED>(t, b, n, h0, h1, l, a.npairs, a.eps, c, s, live, active, dw);
    else
      heads<T, D, MODE, BWD, false>(t, b, n, h0, h1, l, a.npairs, a.eps, c, s, live, active, dw);
  }
  if constexpr (BWD && NORMED) {
    let_next_start();
    // this block's sums of dw: tokens of a warp by shuffles, warps in shared memory, a fixed order
    if (t.weight == nullptr) return;
    __shared__ float sh[THREADS / 32][D];
    const int warp = tid >> 5, lane = tid & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], o);
      if (lane < LPR) sh[warp][Row<T, MODE>::at(l, j, a.npairs)] = dw[j];
    }
    __syncthreads();
    if (tid < D) {
      float v = 0.f;
#pragma unroll
      for (int x = 0; x < THREADS / 32; ++x) v += sh[x][tid];
      a.part[(size_t)blockIdx.x * D + tid] = v;
    }
  }
}

// dw of q (blockIdx.y 0) and of k: the blocks' partial sums, eight columns a
// block, in 64 bits and a fixed order.
__global__ void __launch_bounds__(256) sum_kernel(const float* __restrict__ part, int blocks_q, int blocks, int d,
                                                  float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ double sh[32][9];
  wait_for_last();
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int col = blockIdx.x * 8 + x;
  float* dst = blockIdx.y ? dwk : dwq;
  if (dst == nullptr) return;
  const int b0 = blockIdx.y ? blocks_q : 0, b1 = blockIdx.y ? blocks : blocks_q;
  double v = 0.0;
#pragma unroll 8
  for (int i = b0 + y; i < b1; i += 32) v += (double)part[(size_t)i * d + col];
  sh[y][x] = v;
  __syncthreads();
  if (y == 0) {
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sh[i][x];
    dst[col] = (float)t;
  }
}

static int elem(const spark_rotary_params* p) { return p->dtype == SPARK_FP32 ? 4 : 2; }

static spark_status validate(const spark_rotary_params* p) {
  if (p == nullptr || p->B < 1 || p->Hq < 1 || p->Hk < 0 || p->N < 1 || p->d < 1) return SPARK_ERR_INVALID_ARG;
  if (p->dtype < SPARK_BF16 || p->dtype > SPARK_FP32) return SPARK_ERR_INVALID_ARG;
  if (p->axes < 1 || p->axes > 3) return SPARK_ERR_INVALID_ARG;
  if (p->pairing != SPARK_ROTARY_INTERLEAVED && p->pairing != SPARK_ROTARY_HALVES) return SPARK_ERR_INVALID_ARG;
  if (p->spectrum != SPARK_ROTARY_PER_AXIS && p->spectrum != SPARK_ROTARY_SHARED) return SPARK_ERR_INVALID_ARG;
  if (!(p->theta > 0.0) || !isfinite(p->theta) || !(p->eps >= 0.0) || !isfinite((float)p->eps)) return SPARK_ERR_INVALID_ARG;
  int64_t R = 0;
  for (int a = 0; a < p->axes; ++a) {
    if (p->dims[a] < 0 || p->dims[a] % 2 != 0) return SPARK_ERR_INVALID_ARG;
    if (!isfinite(p->start[a]) || !isfinite(p->scale[a])) return SPARK_ERR_INVALID_ARG;
    R += p->dims[a];
  }
  if (R > p->d) return SPARK_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return SPARK_ERR_UNSUPPORTED;
  if ((int64_t)p->B * ((int64_t)p->Hq + p->Hk) > 65535 || p->N > SPARK_CROSS_MAX_TOKENS) return SPARK_ERR_UNSUPPORTED;
  return SPARK_OK;
}

static bool grid_fits(const spark_rotary_params* p) {
  int64_t n = 1;
  for (int a = 0; a < p->axes; ++a) {
    if (p->grid[a] < 1 || p->grid[a] > p->N) return false;
    n *= p->grid[a];
    if (n > p->N) return false;
  }
  return n == p->N;
}

// Frequencies and the split of the work; the pointers are filled in by the calls.
static Args plan(const spark_rotary_params* p, const float* pos) {
  Args a = {};
  a.N = p->N;
  a.axes = p->axes;
  a.pos = pos;
  a.eps = (float)p->eps;
  int R = 0;
  for (int x = 0; x < p->axes; ++x) R += p->dims[x];
  a.npairs = R / 2;
  a.grid[0] = a.grid[1] = a.grid[2] = 1;
  double f = 1.0 / 6.283185307179586476925;
  for (int x = 0, i = 0; x < p->axes; ++x) {
    if (pos == nullptr) a.grid[x] = p->grid[x];
    a.start[x] = p->start[x];
    a.scale[x] = p->scale[x];
    // theta^(-2j / n) by steps of theta^(-2 / n): j roundings of 2^-53, and j times the
    // step's own error (pow's, up to 2^-52): below 2^-45 in all
    const double step = p->dims[x] > 0 ? pow(p->theta, -2.0 / (p->spectrum == SPARK_ROTARY_PER_AXIS ? p->dims[x] : R)) : 1.0;
    if (p->spectrum == SPARK_ROTARY_PER_AXIS) f = 1.0 / 6.283185307179586476925;
    for (int j = 0; j < p->dims[x] / 2; ++j, ++i, f *= step) {
      a.freq[i] = f;
      a.axis[i] = (unsigned char)x;
    }
  }
  // heads per block: they share a token's angles, so as many as still give every
  // SM a few blocks
  const int tok = THREADS / (p->d / 8);
  a.tiles = (p->N + tok - 1) / tok;
  const int64_t tiles = (int64_t)a.tiles * p->B, want = SM_COUNT * 3;
  const int heads = p->Hq + p->Hk;
  const int64_t share = std::max<int64_t>(1, tiles * heads / want);      // heads a block, for `want` blocks in all
  for (int x = 0; x < 2; ++x) {
    Tensor& t = a.t[x];
    t.H = x ? p->Hk : p->Hq;
    if (t.H == 0) continue;
    t.per_split = (int)std::min<int64_t>(t.H, (share + ROWS - 1) / ROWS * ROWS);
    t.splits = (t.H + t.per_split - 1) / t.per_split;
    t.per_split = (t.H + t.splits - 1) / t.splits;
    t.items = (int)std::min<int64_t>(tiles * t.splits, INT32_MAX);
  }
  return a;
}

template <typename T, int D, bool BWD, bool NORMED>
static void launch_mode(int mode, int blocks, const Args& a, cudaStream_t s) {
  if (mode == CONTIG) kernel<T, D, CONTIG, BWD, NORMED><<<blocks, THREADS, 0, s>>>(a);
  else if (mode == SPLIT4) kernel<T, D, SPLIT4, BWD, NORMED><<<blocks, THREADS, 0, s>>>(a);
  else kernel<T, D, SINGLES, BWD, NORMED><<<blocks, THREADS, 0, s>>>(a);
}

template <typename T, bool BWD, bool NORMED>
static void launch_size(const spark_rotary_params* p, int blocks, const Args& a, cudaStream_t s) {
  // half-split pairs: four of them per lane as two 4-value copies when R is a
  // multiple of 8, else value by value
  const int mode = p->pairing == SPARK_ROTARY_INTERLEAVED ? CONTIG : (a.npairs % 4 == 0 ? SPLIT4 : SINGLES);
  if (p->d == 128) launch_mode<T, 128, BWD, NORMED>(mode, blocks, a, s);
  else launch_mode<T, 64, BWD, NORMED>(mode, blocks, a, s);
}

template <bool BWD, bool NORMED>
static spark_status launch(const spark_rotary_params* p, int blocks, const Args& a, cudaStream_t s) {
  if (p->dtype == SPARK_BF16) launch_size<__nv_bfloat16, BWD, NORMED>(p, blocks, a, s);
  else if (p->dtype == SPARK_FP16) launch_size<__half, BWD, NORMED>(p, blocks, a, s);
  else launch_size<float, BWD, NORMED>(p, blocks, a, s);
  return cudaGetLastError() == cudaSuccess ? SPARK_OK : SPARK_ERR_CUDA;
}

}  // namespace rotary
}  // namespace spark

using namespace spark;

extern "C" {

spark_status spark_rotary_validate(const spark_rotary_params* p) { return rotary::validate(p); }

size_t spark_rotary_workspace_size(const spark_rotary_params* p) {
  return rotary::validate(p) == SPARK_OK ? (size_t)rotary::BWD_BLOCKS * p->d * sizeof(float) : 0;
}

spark_status spark_rotary(const spark_rotary_params* p, const spark_view* q, const spark_view* k,
                          const float* positions, const void* q_weight, const void* k_weight,
                          const spark_view* q_out, const spark_view* k_out, cudaStream_t stream) {
  const spark_status v = rotary::validate(p);
  if (v != SPARK_OK) return v;
  if (positions == nullptr && !rotary::grid_fits(p)) return SPARK_ERR_INVALID_ARG;
  rotary::Args a = rotary::plan(p, positions);
  const int es = rotary::elem(p);
  if (!make_view(q, p->B, p->Hq, p->N, p->d, es, false, &a.t[0].in) ||
      !make_view(q_out, p->B, p->Hq, p->N, p->d, es, true, &a.t[0].out))
    return SPARK_ERR_INVALID_ARG;
  if (p->Hk > 0 && (!make_view(k, p->B, p->Hk, p->N, p->d, es, false, &a.t[1].in) ||
                    !make_view(k_out, p->B, p->Hk, p->N, p->d, es, true, &a.t[1].out)))
    return SPARK_ERR_INVALID_ARG;
  if (!aligned(q_weight) || !aligned(k_weight) || ((uintptr_t)positions & 3u) != 0) return SPARK_ERR_INVALID_ARG;
  const int64_t blocks = (int64_t)a.t[0].items + a.t[1].items;
  if (blocks >= INT32_MAX) return SPARK_ERR_UNSUPPORTED;
  a.blocks_q = a.t[0].items;
  a.t[0].weight = q_weight;
  a.t[1].weight = k_weight;
  return rotary::launch<false, true>(p, (int)blocks, a, stream);
}

spark_status spark_rotary_bwd(const spark_rotary_params* p, const spark_view* dq_out, const spark_view* dk_out,
                              const spark_view* q, const spark_view* k, const float* positions,
                              const void* q_weight, const void* k_weight, const spark_view* dq,
                              const spark_view* dk, float* dq_weight, float* dk_weight, void* ws,
                              size_t ws_bytes, cudaStream_t stream) {
  const spark_status v = rotary::validate(p);
  if (v != SPARK_OK) return v;
  if (positions == nullptr && !rotary::grid_fits(p)) return SPARK_ERR_INVALID_ARG;
  rotary::Args a = rotary::plan(p, positions);
  const int es = rotary::elem(p);
  const spark_view* views[2][3] = {{dq_out, q, dq}, {dk_out, k, dk}};
  const void* weights[2] = {q_weight, p->Hk > 0 ? k_weight : nullptr};
  for (int x = 0; x < (p->Hk > 0 ? 2 : 1); ++x) {
    rotary::Tensor& t = a.t[x];
    t.weight = weights[x];
    if (!make_view(views[x][0], p->B, t.H, p->N, p->d, es, false, &t.in) ||
        !make_view(views[x][2], p->B, t.H, p->N, p->d, es, true, &t.out) ||
        (t.weight != nullptr && !make_view(views[x][1], p->B, t.H, p->N, p->d, es, false, &t.x)))
      return SPARK_ERR_INVALID_ARG;
  }
  if (!aligned(q_weight) || !aligned(k_weight) || ((uintptr_t)positions & 3u) != 0) return SPARK_ERR_INVALID_ARG;
  if ((weights[0] != nullptr && dq_weight == nullptr) || (weights[1] != nullptr && dk_weight == nullptr))
    return SPARK_ERR_INVALID_ARG;
  const bool norm = weights[0] != nullptr || weights[1] != nullptr;
  int64_t blocks = (int64_t)a.t[0].items + a.t[1].items;
  if (blocks >= INT32_MAX) return SPARK_ERR_UNSUPPORTED;
  a.blocks_q = a.t[0].items;
  if (norm) {
    if (ws == nullptr || !aligned(ws)) return SPARK_ERR_INVALID_ARG;
    if (ws_bytes < spark_rotary_workspace_size(p)) return SPARK_ERR_WORKSPACE;
    a.part = static_cast<float*>(ws);
    // blocks in proportion to the tensors' work: a row with a norm reads its x too
    if (blocks > rotary::BWD_BLOCKS) {
      blocks = rotary::BWD_BLOCKS;
      const double wq = a.t[0].H * (weights[0] ? 3.0 : 2.0), wk = a.t[1].H * (weights[1] ? 3.0 : 2.0);
      a.blocks_q = std::min(a.t[0].items, std::max(1, (int)(blocks * wq / (wq + wk) + 0.5)));
      if (p->Hk > 0) a.blocks_q = std::min<int>(a.blocks_q, (int)blocks - 1);
      else a.blocks_q = (int)blocks;
    }
  }
  const spark_status e = norm ? rotary::launch<true, true>(p, (int)blocks, a, stream)
                              : rotary::launch<true, false>(p, (int)blocks, a, stream);
  if (e != SPARK_OK || !norm) return e;
  const cudaError_t l = launch_behind(rotary::sum_kernel, dim3(p->d / 8, 2), 256, 0, stream, a.part, a.blocks_q, (int)blocks,
                                      p->d, weights[0] ? dq_weight : nullptr, weights[1] ? dk_weight : nullptr);
  return l == cudaSuccess ? SPARK_OK : SPARK_ERR_CUDA;
}

size_t spark_forward_rotary_workspace_size(const spark_params* p) {
  const size_t base = spark_workspace_size(p);
  return base == 0 ? 0 : (base + 255) / 256 * 256 + 3 * (size_t)p->B * p->H * p->N * p->d * 2;
}

spark_status spark_forward_rotary(const spark_params* p, const spark_rotary_params* r, const spark_view* q,
                                  const spark_view* k, const spark_view* v, const float* positions,
                                  const void* q_weight, const void* k_weight, void* out, float* lse, void* ws,
                                  size_t ws_bytes, cudaStream_t stream) {
  const spark_status vp = spark_validate(p);
  if (vp != SPARK_OK) return vp;
  const spark_status vr = rotary::validate(r);
  if (vr != SPARK_OK) return vr;
  if (r->B != p->B || r->Hq != p->H || r->Hk != p->H || r->N != p->N || r->d != p->d || r->dtype != SPARK_BF16)
    return SPARK_ERR_INVALID_ARG;
  if (positions == nullptr && !rotary::grid_fits(r)) return SPARK_ERR_INVALID_ARG;
  View seen[3];
  const spark_view* in[3] = {q, k, v};
  for (int x = 0; x < 3; ++x)
    if (!make_view(in[x], p->B, p->H, p->N, p->d, 2, false, &seen[x])) return SPARK_ERR_INVALID_ARG;
  if (out == nullptr || !aligned(out) || !aligned(q_weight) || !aligned(k_weight) || ((uintptr_t)positions & 3u) != 0)
    return SPARK_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws)) return SPARK_ERR_INVALID_ARG;
  if (ws_bytes < spark_forward_rotary_workspace_size(p)) return SPARK_ERR_WORKSPACE;
  const size_t base = (spark_workspace_size(p) + 255) / 256 * 256, bytes = (size_t)p->B * p->H * p->N * p->d * 2;
  const int64_t head = (int64_t)p->N * p->d;
  spark_view to[3];
  for (int x = 0; x < 3; ++x) to[x] = spark_view{static_cast<char*>(ws) + base + x * bytes, p->H * head, head, p->d};
  spark_status e = spark_rotary(r, q, k, positions, q_weight, k_weight, &to[0], &to[1], stream);
  if (e != SPARK_OK) return e;
  const bool contiguous = (p->B == 1 || seen[2].b == p->H * head) && (p->H == 1 || seen[2].h == head) && seen[2].n == p->d;
  if (!contiguous) {
    // the same kernel with no rotated values: a change of layout
    spark_rotary_params copy = *r;
    copy.Hk = 0;
    copy.axes = 1;
    copy.dims[0] = 0;
    copy.grid[0] = p->N;
    e = spark_rotary(&copy, v, nullptr, nullptr, nullptr, nullptr, &to[2], nullptr, stream);
    if (e != SPARK_OK) return e;
  }
  return spark_forward(p, to[0].data, to[1].data, contiguous ? v->data : to[2].data, out, lse, nullptr, nullptr, ws,
                       spark_workspace_size(p), stream);
}

}  // extern "C"
