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
void few_keys(const Problem& p, int64_t* keys);   // keys of an SM's blocks one after another, 256 for the start of each
cudaError_t launch_few(const Problem& p, void* ws, cudaStream_t s);

// Many query rows: 128 rows per tile (tcgen05). Kept keys are the first
// key_len[b] of an item; key_mask is not looked at.
size_t many_workspace(const Problem& p);
void many_keys(const Problem& p, int64_t* keys, int* shares);   // keys of a CTA's items, shares of a row tile
cudaError_t launch_many(const Problem& p, bool packed, void* ws, cudaStream_t s);   // packed: launch_pack came just before

// The kept keys of each item moved to the front: k and v become contiguous
// [B,Hkv,Nk,d] copies in ws whose first count[b] rows are the kept ones in
// order; place[b,j] is the row key j went to, or -1.
struct Packed {
  size_t bytes, off_k, off_v, off_count, off_place;
};
Packed pack_plan(const Problem& p);
struct PackArgs {
  View k, v;
  const int32_t* key_len;
  const uint8_t* mask;                   // null: nothing to pack
  int B, Hkv, Nk, d;
  char *ko, *vo;
  int32_t *count, *place;
  int* status;
};
PackArgs pack_args(const Problem& p, const Packed& pk, void* ws);
cudaError_t launch_pack(const PackArgs& a, cudaStream_t s);

// Gradients (bf16). p.out is the forward's result. With pack.mask the kept keys
// are packed first, and p.k, p.v and p.key_len are the packed ones.
struct Gradients {
  View dout, dq, dk, dv;
  const float* lse;
};
size_t bwd_workspace(const Problem& p);
cudaError_t launch_bwd(const Problem& p, const Gradients& g, const PackArgs& pack, void* ws, cudaStream_t s);

inline size_t align_up(size_t x) { return (x + 255) & ~(size_t)255; }

// The kernels' workspace begins at the first multiple of 256 bytes in the caller's,
// which is only 16-byte aligned: partial sums are written in 32-byte stores. The
// sizes callers are told have WS_SLACK for that.
constexpr size_t WS_SLACK = 256;
inline char* workspace_base(void* ws) { return reinterpret_cast<char*>(align_up(reinterpret_cast<uintptr_t>(ws))); }

#ifdef __CUDACC__
}  // namespace cross
}  // namespace spark
#include "common.cuh"
namespace spark {
namespace cross {
// Length of item b, clamped; `report` says a bad one to the status word.
__device__ __forceinline__ int item_len(const int32_t* key_len, int Nk, int b, int* status, bool report) {
  if (key_len == nullptr) return Nk;
  const int n = key_len[b];
  if (n >= 0 && n <= Nk) return n;
  if (report) set_status(status, STATUS_BAD_INPUT);
  return n < 0 ? 0 : Nk;
}
// A value of the result before it is rounded. The weights of P V are rounded, those
// of the sum are not, so values near fp16's largest (65,504) may come out up to
// 2^-11 past it, where rounding would make them infinite.
template <bool H>
__device__ __forceinline__ float in_range(float x) {
  if constexpr (H) {
    if (fabsf(x) < 65568.f) x = fminf(fmaxf(x, -65504.f), 65504.f);
  }
  return x;
}
#endif

}  // namespace cross
}  // namespace spark
