// Kept keys of a masked cross attention moved to the front, so that the
// tensor-core kernels see a plain length: what is dropped is not computed, and
// never read again.
//
// grid (64-key chunks, Hkv, B), 256 threads. A block counts the kept keys
// before its chunk (the mask is a byte per key and stays in cache), ranks its own, and
// copies their rows of k and v, four threads a row. Reads and writes each kept
// row once: bound by HBM or L2, a few microseconds for an encoder's states.
#include "common.cuh"
#include "cross.h"

namespace spark {
namespace cross {

constexpr int CHUNK = 64, PACK_THREADS = 256;

struct PackArgs {
  View k, v;
  const int32_t* key_len;
  const uint8_t* mask;
  int Hkv, Nk, d;
  char *ko, *vo;
  int32_t *count, *place;
  int* status;
};

__global__ void __launch_bounds__(PACK_THREADS) pack_kernel(const __grid_constant__ PackArgs a) {
  __shared__ int warp_sum_sh[PACK_THREADS / 32];
  __shared__ int place_sh[CHUNK];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int j0 = blockIdx.x * CHUNK, hk = blockIdx.y, b = blockIdx.z;
  const int len = item_len(a.key_len, a.Nk, b, a.status, tid == 0 && j0 == 0 && hk == 0);
  const uint8_t* mask = a.mask + (size_t)b * a.Nk;
  int c = 0;
  for (int j = tid; j < min(j0, len); j += PACK_THREADS) c += mask[j] != 0;
  c = __reduce_add_sync(0xffffffffu, c);
  if (lane == 0) warp_sum_sh[warp] = c;
  __syncthreads();
  if (warp == 0) {
    int before = 0;
#pragma unroll
    for (int w = 0; w < PACK_THREADS / 32; ++w) before += warp_sum_sh[w];
#pragma unroll
    for (int x = 0; x < CHUNK; x += 32) {
      const int j = j0 + x + lane;
      const bool kept = j < len && mask[j] != 0;
      const unsigned bits = __ballot_sync(0xffffffffu, kept);
      const int at = kept ? before + __popc(bits & ((1u << lane) - 1u)) : -1;
      place_sh[x + lane] = at;
      if (hk == 0 && j < a.Nk) a.place[(size_t)b * a.Nk + j] = at;
      before += __popc(bits);
    }
    if (hk == 0 && lane == 0 && j0 + CHUNK >= a.Nk) a.count[b] = before;
  }
  __syncthreads();
  const int row = tid >> 2, at = place_sh[row];
  if (at < 0) return;
  const int j = j0 + row, chunks = a.d / 8;
  const size_t to = (((size_t)b * a.Hkv + hk) * a.Nk + at) * a.d * 2;
  const char* ks = a.k.data + 2 * (b * a.k.b + hk * a.k.h + (int64_t)j * a.k.n);
  const char* vs = a.v.data + 2 * (b * a.v.b + hk * a.v.h + (int64_t)j * a.v.n);
  for (int x = tid & 3; x < chunks; x += 4) {
    *reinterpret_cast<uint4*>(a.ko + to + 16 * x) = *reinterpret_cast<const uint4*>(ks + 16 * x);
    *reinterpret_cast<uint4*>(a.vo + to + 16 * x) = *reinterpret_cast<const uint4*>(vs + 16 * x);
  }
}

Packed pack_plan(const Problem& p) {
  const size_t rows = (size_t)p.B * p.Hkv * p.Nk;
  Packed k;
  k.off_k = 0;
  k.off_v = align_up(rows * p.d * 2);
  k.off_count = k.off_v + align_up(rows * p.d * 2);
  k.off_place = k.off_count + align_up((size_t)p.B * 4);
  k.bytes = k.off_place + align_up((size_t)p.B * p.Nk * 4);
  return k;
}

cudaError_t launch_pack(const Problem& p, const Packed& pk, void* ws, cudaStream_t s) {
  char* w = static_cast<char*>(ws);
  const PackArgs a{p.k, p.v, p.key_len, p.key_mask, p.Hkv, p.Nk, p.d, w + pk.off_k, w + pk.off_v,
                   reinterpret_cast<int32_t*>(w + pk.off_count), reinterpret_cast<int32_t*>(w + pk.off_place), p.status};
  pack_kernel<<<dim3((p.Nk + CHUNK - 1) / CHUNK, p.Hkv, p.B), PACK_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace cross
}  // namespace spark
