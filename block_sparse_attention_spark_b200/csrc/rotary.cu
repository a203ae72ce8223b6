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
// to [-1/2, 1/2], then 32-bit sincospi), and walks the heads of q and of k
// with them in registers, four rows in flight. A warp's 32 lanes hold two
// (d = 128) or four (d = 64) rows, so the mean of squares is a shuffle over 16
// or 8 lanes. A block holds 256 / (d / 8) tokens; heads are split over blocks
// when tokens alone do not fill the GPU.
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "views.h"

namespace spark {
namespace rotary {

constexpr int THREADS = 256;
constexpr int UNROLL = 4;              // rows in flight per thread
constexpr int BWD_BLOCKS = SM_COUNT * 4;   // most blocks of the gradient (partial sums of dw)

struct Args {
  View q, k, qo, ko, dq, dk;           // bwd: q, k inputs; qo, ko gradients of the outputs; dq, dk written
  const float* pos;                    // [B, N, axes] or null
  const void *wq, *wk;
  float* part;                         // [blocks][2][d] partial sums of dw
  int B, Hq, Hk, N, axes;
  int npairs;                          // R / 2
  int tiles, splits, per_split;        // token tiles per item, head splits, heads per split
  long items;
  int grid[3];
  float eps;
  double start[3], scale[3];
  double freq[64];                     // turns per unit of position, by pair
  unsigned char axis[64];
};

// where a lane's eight values stand in the row: pair j of the lane is values
// 2j, 2j+1 of the register array
enum { CONTIG = 0, SPLIT4 = 1, SINGLES = 2 };

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f(float v) { return v; }

template <typename T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Pack {
  T v[N];
};

// A lane's eight values of a row (raw, converted on use).
template <typename T, int MODE>
struct Row {
  T v[8];
  __device__ __forceinline__ void load(const T* row, int l, int npairs) {
    if constexpr (MODE == CONTIG) {
      *reinterpret_cast<Pack<T, 8>*>(v) = *reinterpret_cast<const Pack<T, 8>*>(row + 8 * l);
    } else if constexpr (MODE == SPLIT4) {
      // the lanes before R / 8 hold four pairs, the others eight kept values
      const bool pairs = 4 * l < npairs;
      const Pack<T, 4> a = *reinterpret_cast<const Pack<T, 4>*>(row + (pairs ? 4 * l : 8 * l));
      const Pack<T, 4> b = *reinterpret_cast<const Pack<T, 4>*>(row + (pairs ? npairs + 4 * l : 8 * l + 4));
#pragma unroll
      for (int j = 0; j < 4; ++j) { v[2 * j] = a.v[j]; v[2 * j + 1] = b.v[j]; }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = row[at(l, j, npairs)];
    }
  }
  __device__ __forceinline__ void store(T* row, int l, int npairs) const {
    if constexpr (MODE == CONTIG) {
      *reinterpret_cast<Pack<T, 8>*>(row + 8 * l) = *reinterpret_cast<const Pack<T, 8>*>(v);
    } else if constexpr (MODE == SPLIT4) {
      const bool pairs = 4 * l < npairs;
      Pack<T, 4> a, b;
#pragma unroll
      for (int j = 0; j < 4; ++j) { a.v[j] = v[2 * j]; b.v[j] = v[2 * j + 1]; }
      *reinterpret_cast<Pack<T, 4>*>(row + (pairs ? 4 * l : 8 * l)) = a;
      *reinterpret_cast<Pack<T, 4>*>(row + (pairs ? npairs + 4 * l : 8 * l + 4)) = b;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) row[at(l, j, npairs)] = v[j];
    }
  }
  // index in the row of register value j
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

template <typename T, int D, int MODE, bool NORM>
__device__ __forceinline__ void forward_row(Row<T, MODE>& x, const float* c, const float* s, const float* w,
                                            unsigned live, float eps) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = to_f(x.v[j]);
  if constexpr (NORM) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
    const float r = 1.f / sqrtf(row_sum<D / 8>(ss) * (1.f / D) + eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= r * w[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float u = f[2 * j], v = f[2 * j + 1];
    if ((live >> j) & 1u) {
      f[2 * j] = fmaf(u, c[j], -v * s[j]);
      f[2 * j + 1] = fmaf(u, s[j], v * c[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) x.v[j] = from_f<T>(f[j]);
}

// y: gradient of the row's result, becomes the gradient of the row x.
template <typename T, int D, int MODE, bool NORM>
__device__ __forceinline__ void backward_row(Row<T, MODE>& y, const Row<T, MODE>& x, const float* c, const float* s,
                                             const float* w, unsigned live, float eps, bool active, float* dw) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = to_f(y.v[j]);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float u = f[2 * j], v = f[2 * j + 1];
    if ((live >> j) & 1u) {
      f[2 * j] = fmaf(u, c[j], v * s[j]);
      f[2 * j + 1] = fmaf(v, c[j], -u * s[j]);
    }
  }
  if constexpr (NORM) {
    float xs[8], ss = 0.f, xg = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      xs[j] = to_f(x.v[j]);
      ss = fmaf(xs[j], xs[j], ss);
      xg = fmaf(xs[j], f[j] * w[j], xg);
    }
    ss = row_sum<D / 8>(ss);
    xg = row_sum<D / 8>(xg);
    const float r = 1.f / sqrtf(ss * (1.f / D) + eps);
    const float t = r * r * xg * (1.f / D);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (active) dw[j] = fmaf(f[j], xs[j] * r, dw[j]);
      f[j] = r * (f[j] * w[j] - xs[j] * t);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) y.v[j] = from_f<T>(f[j]);
}

// The heads [h0, h1) of one tensor at one token.
template <typename T, int D, int MODE, bool BWD, bool NORM>
__device__ __forceinline__ void heads(const View& in, const View& x, const View& out, const void* weight, int b, int n,
                                      int h0, int h1, int l, const Args& a, const float* c, const float* s,
                                      unsigned live, bool active, float* dw) {
  float w[8];
  if constexpr (NORM) {
    Row<T, MODE> wr;
    wr.load(static_cast<const T*>(weight), l, a.npairs);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = to_f(wr.v[j]);
  }
  const T* pi = reinterpret_cast<const T*>(in.data) + b * in.b + n * in.n;
  const T* px = BWD && NORM ? reinterpret_cast<const T*>(x.data) + b * x.b + n * x.n : nullptr;
  T* po = reinterpret_cast<T*>(out.data) + b * out.b + n * out.n;
  int h = h0;
  for (; h + UNROLL <= h1; h += UNROLL) {
    Row<T, MODE> r[UNROLL], rx[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      r[u].load(pi + (h + u) * in.h, l, a.npairs);
      if constexpr (BWD && NORM) rx[u].load(px + (h + u) * x.h, l, a.npairs);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if constexpr (BWD) backward_row<T, D, MODE, NORM>(r[u], rx[u], c, s, w, live, a.eps, active, dw);
      else forward_row<T, D, MODE, NORM>(r[u], c, s, w, live, a.eps);
      if (active) r[u].store(po + (h + u) * out.h, l, a.npairs);
    }
  }
  for (; h < h1; ++h) {
    Row<T, MODE> r, rx;
    r.load(pi + h * in.h, l, a.npairs);
    if constexpr (BWD && NORM) rx.load(px + h * x.h, l, a.npairs);
    if constexpr (BWD) backward_row<T, D, MODE, NORM>(r, rx, c, s, w, live, a.eps, active, dw);
    else forward_row<T, D, MODE, NORM>(r, c, s, w, live, a.eps);
    if (active) r.store(po + h * out.h, l, a.npairs);
  }
}

template <typename T, int D, int MODE, bool BWD>
__global__ void __launch_bounds__(THREADS) kernel(const __grid_constant__ Args a) {
  constexpr int LPR = D / 8, TOK = THREADS / LPR;
  __shared__ double freq[64];
  __shared__ unsigned char axis[64];
  const int tid = threadIdx.x, l = tid % LPR;
  if (tid < 64) {
    freq[tid] = a.freq[tid];
    axis[tid] = a.axis[tid];
  }
  __syncthreads();
  float dwq[8], dwk[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dwq[j] = dwk[j] = 0.f;
  for (long it = blockIdx.x; it < a.items; it += gridDim.x) {
    const int split = (int)(it % a.splits);
    const long tile = it / a.splits;
    const int b = (int)(tile / a.tiles);
    const int tok = (int)(tile % a.tiles) * TOK + tid / LPR;
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
    const int h0 = split * a.per_split, h1 = min(h0 + a.per_split, a.Hq + a.Hk);
    if (h0 < a.Hq) {
      if (a.wq != nullptr)
        heads<T, D, MODE, BWD, true>(BWD ? a.qo : a.q, a.q, BWD ? a.dq : a.qo, a.wq, b, n, h0, min(h1, a.Hq), l, a, c,
                                     s, live, active, dwq);
      else
        heads<T, D, MODE, BWD, false>(BWD ? a.qo : a.q, a.q, BWD ? a.dq : a.qo, nullptr, b, n, h0, min(h1, a.Hq), l, a,
                                      c, s, live, active, dwq);
    }
    if (h1 > a.Hq) {
      if (a.wk != nullptr)
        heads<T, D, MODE, BWD, true>(BWD ? a.ko : a.k, a.k, BWD ? a.dk : a.ko, a.wk, b, n, max(h0, a.Hq) - a.Hq,
                                     h1 - a.Hq, l, a, c, s, live, active, dwk);
      else
        heads<T, D, MODE, BWD, false>(BWD ? a.ko : a.k, a.k, BWD ? a.dk : a.ko, nullptr, b, n, max(h0, a.Hq) - a.Hq,
                                      h1 - a.Hq, l, a, c, s, live, active, dwk);
    }
  }
  if constexpr (BWD) {
    // this block's sums of dw: tokens of a warp by shuffles, warps in shared memory, a fixed order
    if (a.wq == nullptr && a.wk == nullptr) return;
    __shared__ float sh[2][THREADS / 32][D];
    const int warp = tid >> 5, lane = tid & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        dwq[j] += __shfl_xor_sync(0xffffffffu, dwq[j], o);
        dwk[j] += __shfl_xor_sync(0xffffffffu, dwk[j], o);
      }
      if (lane < LPR) {
        const int i = Row<T, MODE>::at(l, j, a.npairs);
        sh[0][warp][i] = dwq[j];
        sh[1][warp][i] = dwk[j];
      }
    }
    __syncthreads();
    for (int i = tid; i < 2 * D; i += THREADS) {
      float v = 0.f;
#pragma unroll
      for (int x = 0; x < THREADS / 32; ++x) v += sh[i / D][x][i % D];
      a.part[(size_t)blockIdx.x * 2 * D + i] = v;
    }
  }
}

// dw of both tensors: the blocks' partial sums, 32 columns per block, in 64 bits.
__global__ void __launch_bounds__(1024) sum_kernel(const float* __restrict__ part, int blocks, int d,
                                                   float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ double sh[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + x;
  double v = 0.0;
  for (int i = y; i < blocks; i += 32) v += (double)part[(size_t)i * 2 * d + col];
  sh[y][x] = v;
  __syncthreads();
  if (y == 0) {
    double t = 0.0;
    for (int i = 0; i < 32; ++i) t += sh[i][x];
    float* dst = col < d ? dwq : dwk;
    if (dst != nullptr) dst[col < d ? col : col - d] = (float)t;
  }
}

static int elem(const spark_rotary_params* p) { return p->dtype == SPARK_FP32 ? 4 : 2; }

static spark_status validate(const spark_rotary_params* p) {
  if (p == nullptr || p->B < 1 || p->Hq < 1 || p->Hk < 0 || p->N < 1 || p->d < 1) return SPARK_ERR_INVALID_ARG;
  if (p->dtype < SPARK_BF16 || p->dtype > SPARK_FP32) return SPARK_ERR_INVALID_ARG;
  if (p->axes < 1 || p->axes > 3) return SPARK_ERR_INVALID_ARG;
  if (p->pairing != SPARK_ROTARY_INTERLEAVED && p->pairing != SPARK_ROTARY_HALVES) return SPARK_ERR_INVALID_ARG;
  if (p->spectrum != SPARK_ROTARY_PER_AXIS && p->spectrum != SPARK_ROTARY_SHARED) return SPARK_ERR_INVALID_ARG;
  if (!(p->theta > 0.0) || !isfinite(p->theta) || !(p->eps >= 0.0) || !isfinite(p->eps)) return SPARK_ERR_INVALID_ARG;
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
  a.B = p->B; a.Hq = p->Hq; a.Hk = p->Hk; a.N = p->N; a.axes = p->axes;
  a.pos = pos;
  a.eps = (float)p->eps;
  int R = 0;
  for (int x = 0; x < p->axes; ++x) R += p->dims[x];
  a.npairs = R / 2;
  a.grid[0] = a.grid[1] = a.grid[2] = 1;
  for (int x = 0, i = 0; x < p->axes; ++x) {
    if (pos == nullptr) a.grid[x] = p->grid[x];
    a.start[x] = p->start[x];
    a.scale[x] = p->scale[x];
    for (int j = 0; j < p->dims[x] / 2; ++j, ++i) {
      const double e = p->spectrum == SPARK_ROTARY_PER_AXIS ? 2.0 * j / p->dims[x] : 2.0 * i / R;
      a.freq[i] = pow(p->theta, -e) / 6.283185307179586476925;
      a.axis[i] = (unsigned char)x;
    }
  }
  const int tok = THREADS / (p->d / 8), heads = p->Hq + p->Hk;
  a.tiles = (p->N + tok - 1) / tok;
  // heads per block: all of them share a token's angles, so as many as still
  // give every SM several blocks
  const long tiles = (long)a.tiles * p->B;
  const long want = (long)SM_COUNT * 24;
  int splits = (int)std::min<long>((heads + UNROLL - 1) / UNROLL, std::max<long>(1, (want + tiles - 1) / tiles));
  a.per_split = ((heads + splits - 1) / splits + UNROLL - 1) / UNROLL * UNROLL;
  a.splits = (heads + a.per_split - 1) / a.per_split;
  a.items = tiles * a.splits;
  return a;
}

template <typename T, int D, bool BWD>
static void launch_mode(int mode, int blocks, const Args& a, cudaStream_t s) {
  if (mode == CONTIG) kernel<T, D, CONTIG, BWD><<<blocks, THREADS, 0, s>>>(a);
  else if (mode == SPLIT4) kernel<T, D, SPLIT4, BWD><<<blocks, THREADS, 0, s>>>(a);
  else kernel<T, D, SINGLES, BWD><<<blocks, THREADS, 0, s>>>(a);
}

template <bool BWD>
static spark_status launch(const spark_rotary_params* p, int blocks, const Args& a, cudaStream_t s) {
  // half-split pairs: four of them per lane as two 4-value copies when R is a
  // multiple of 8, else value by value
  const int mode = p->pairing == SPARK_ROTARY_INTERLEAVED ? CONTIG : (a.npairs % 4 == 0 ? SPLIT4 : SINGLES);
  if (p->d == 128) {
    if (p->dtype == SPARK_BF16) launch_mode<__nv_bfloat16, 128, BWD>(mode, blocks, a, s);
    else if (p->dtype == SPARK_FP16) launch_mode<__half, 128, BWD>(mode, blocks, a, s);
    else launch_mode<float, 128, BWD>(mode, blocks, a, s);
  } else {
    if (p->dtype == SPARK_BF16) launch_mode<__nv_bfloat16, 64, BWD>(mode, blocks, a, s);
    else if (p->dtype == SPARK_FP16) launch_mode<__half, 64, BWD>(mode, blocks, a, s);
    else launch_mode<float, 64, BWD>(mode, blocks, a, s);
  }
  return cudaGetLastError() == cudaSuccess ? SPARK_OK : SPARK_ERR_CUDA;
}

}  // namespace rotary
}  // namespace spark

using namespace spark;

extern "C" {

spark_status spark_rotary_validate(const spark_rotary_params* p) { return rotary::validate(p); }

size_t spark_rotary_workspace_size(const spark_rotary_params* p) {
  return rotary::validate(p) == SPARK_OK ? (size_t)rotary::BWD_BLOCKS * 2 * p->d * sizeof(float) : 0;
}

spark_status spark_rotary(const spark_rotary_params* p, const spark_view* q, const spark_view* k,
                          const float* positions, const void* q_weight, const void* k_weight,
                          const spark_view* q_out, const spark_view* k_out, cudaStream_t stream) {
  const spark_status v = rotary::validate(p);
  if (v != SPARK_OK) return v;
  if (positions == nullptr && !rotary::grid_fits(p)) return SPARK_ERR_INVALID_ARG;
  rotary::Args a = rotary::plan(p, positions);
  const int es = rotary::elem(p);
  if (!make_view(q, p->B, p->Hq, p->N, p->d, es, false, &a.q) ||
      !make_view(q_out, p->B, p->Hq, p->N, p->d, es, true, &a.qo))
    return SPARK_ERR_INVALID_ARG;
  if (p->Hk > 0 && (!make_view(k, p->B, p->Hk, p->N, p->d, es, false, &a.k) ||
                    !make_view(k_out, p->B, p->Hk, p->N, p->d, es, true, &a.ko)))
    return SPARK_ERR_INVALID_ARG;
  if (!aligned(q_weight) || !aligned(k_weight) || ((uintptr_t)positions & 3u) != 0) return SPARK_ERR_INVALID_ARG;
  if (a.items > INT32_MAX) return SPARK_ERR_UNSUPPORTED;
  a.wq = q_weight;
  a.wk = p->Hk > 0 ? k_weight : nullptr;
  return rotary::launch<false>(p, (int)a.items, a, stream);
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
  a.wq = q_weight;
  a.wk = p->Hk > 0 ? k_weight : nullptr;
  if (!make_view(dq_out, p->B, p->Hq, p->N, p->d, es, false, &a.qo) ||
      !make_view(dq, p->B, p->Hq, p->N, p->d, es, true, &a.dq) ||
      (a.wq != nullptr && !make_view(q, p->B, p->Hq, p->N, p->d, es, false, &a.q)))
    return SPARK_ERR_INVALID_ARG;
  if (p->Hk > 0 && (!make_view(dk_out, p->B, p->Hk, p->N, p->d, es, false, &a.ko) ||
                    !make_view(dk, p->B, p->Hk, p->N, p->d, es, true, &a.dk) ||
                    (a.wk != nullptr && !make_view(k, p->B, p->Hk, p->N, p->d, es, false, &a.k))))
    return SPARK_ERR_INVALID_ARG;
  if (!aligned(q_weight) || !aligned(k_weight) || ((uintptr_t)positions & 3u) != 0) return SPARK_ERR_INVALID_ARG;
  if ((a.wq != nullptr && dq_weight == nullptr) || (a.wk != nullptr && dk_weight == nullptr))
    return SPARK_ERR_INVALID_ARG;
  int blocks = (int)std::min<long>(a.items, INT32_MAX);
  const bool norm = a.wq != nullptr || a.wk != nullptr;
  if (norm) {
    if (ws == nullptr || !aligned(ws)) return SPARK_ERR_INVALID_ARG;
    if (ws_bytes < spark_rotary_workspace_size(p)) return SPARK_ERR_WORKSPACE;
    a.part = static_cast<float*>(ws);
    blocks = (int)std::min<long>(a.items, rotary::BWD_BLOCKS);
  }
  const spark_status e = rotary::launch<true>(p, blocks, a, stream);
  if (e != SPARK_OK || !norm) return e;
  rotary::sum_kernel<<<2 * p->d / 32, 1024, 0, stream>>>(a.part, blocks, p->d, a.wq ? dq_weight : nullptr,
                                                         a.wk ? dk_weight : nullptr);
  return cudaGetLastError() == cudaSuccess ? SPARK_OK : SPARK_ERR_CUDA;
}

}  // extern "C"
