// Tensor maps of strided [B,H,N,d] 16-bit tensors (128-byte swizzle, boxes of
// 64 values by a number of tokens of one head).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "views.h"

namespace spark {

struct TensorMap {
  CUtensorMap map;
  int h_on, b_on;              // 0: the axis has stride 0 (or extent 1), its coordinate is 0
};

inline bool make_tensor_map(TensorMap* m, const View& v, int B, int H, int N, int d, bool fp16, int box_tokens) {
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<Encode>(p) : nullptr;
  }();
  if (fn == nullptr) return false;
  m->h_on = v.h != 0;
  m->b_on = v.b != 0;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)(m->h_on ? H : 1), (cuuint64_t)(m->b_on ? B : 1)};
  const cuuint64_t row = 2 * (cuuint64_t)(N > 1 ? v.n : d);
  const cuuint64_t strides[3] = {row, m->h_on ? 2 * (cuuint64_t)v.h : row, m->b_on ? 2 * (cuuint64_t)v.b : row};
  const cuuint32_t box[4] = {64u, (cuuint32_t)box_tokens, 1u, 1u};
  const cuuint32_t step[4] = {1u, 1u, 1u, 1u};
  return fn(&m->map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.data, dims,
            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace spark
