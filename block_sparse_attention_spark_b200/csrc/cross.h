// Cross attention to an encoder's states: what its calls hand to the kernels.
#pragma once

#include <cuda_runtime.h>

#include "views.h"

namespace spark {
namespace cross {

struct Problem {
  int B, Hq, Hkv, G, Nq, Nk, d;          // G = Hq / Hkv
  int fp16;
  float scale;
  View q, k, v, out;
  const int32_t* key_len;
  const uint8_t* key_mask;
  float* lse;
  int* status;
};

// Few query rows: 16 rows per tile (mma.sync), keys split over warps and blocks.
size_t few_workspace(const Problem& p);
cudaError_t launch_few(const Problem& p, void* ws, cudaStream_t s);

}  // namespace cross
}  // namespace spark
