// Strided [B,H,N,d] tensors of the operators around the attention: host-side
// checks of the views a caller passes, and what the kernels get of them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "spark.h"

namespace spark {

constexpr int SM_COUNT = 148;   // B200

struct View {                   // strides in elements; 0 for an axis of extent 1
  char* data;
  int64_t b, h, n;
};

inline bool aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// False: a null or misaligned base, a negative stride or one that breaks the
// 16-byte rule, tokens that overlap, or a written view that overlaps itself.
inline bool make_view(const spark_view* v, int B, int H, int N, int d, int elem, bool written, View* out) {
  if (v == nullptr || v->data == nullptr || !aligned(v->data)) return false;
  const int64_t ext[3] = {B, H, N};
  int64_t str[3] = {v->b, v->h, v->n};
  for (int i = 0; i < 3; ++i) {
    if (ext[i] == 1) str[i] = 0;
    if (str[i] < 0 || (str[i] * elem) % 16 != 0 || str[i] > ((int64_t)1 << 38)) return false;
  }
  if (N > 1 && str[2] < d) return false;
  if (written) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int x, int y) { return str[x] < str[y]; });
    int64_t cover = d;          // elements from the first to past the last one so far
    for (int i = 0; i < 3; ++i) {
      const int a = order[i];
      if (ext[a] == 1) continue;
      if (str[a] < cover) return false;
      cover += str[a] * (ext[a] - 1);
    }
  }
  out->data = static_cast<char*>(const_cast<void*>(v->data));
  out->b = str[0];
  out->h = str[1];
  out->n = str[2];
  return true;
}

// Lets a kernel use `bytes` of dynamic shared memory, asked of the runtime once
// per device (done: bits by device number, one word per kernel).
template <typename F>
inline cudaError_t allow_shared(F* kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (bit != 0 && (done->load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A launch that may be set up while the stream's last kernel (one that calls
// let_next_start) still runs; the kernel begins with wait_for_last.
template <typename... P, typename... A>
inline cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, int shared, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#ifdef __CUDACC__
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Returns once the kernel before has ended and what it wrote is visible; nothing
// in global memory is touched before it.
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

// The library's device status word on the current device (spark_get_status).
int* device_status();

}  // namespace spark
