// Packing of a masked cross attention's kept keys as a launch of its own
// (see cross_pack.cuh), and its place in the workspace.
#include "cross_pack.cuh"

namespace spark {
namespace cross {

__global__ void __launch_bounds__(PACK_THREADS) pack_kernel(const __grid_constant__ PackArgs a) {
  let_next_start();
  pack_block(a, blockIdx.x);
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

PackArgs pack_args(const Problem& p, const Packed& pk, void* ws) {
  char* w = static_cast<char*>(ws);
  return PackArgs{p.k, p.v, p.key_len, p.key_mask, p.B, p.Hkv, p.Nk, p.d, w + pk.off_k, w + pk.off_v,
                  reinterpret_cast<int32_t*>(w + pk.off_count), reinterpret_cast<int32_t*>(w + pk.off_place), p.status};
}

cudaError_t launch_pack(const PackArgs& a, cudaStream_t s) {
  pack_kernel<<<(unsigned)pack_blocks(a), PACK_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace cross
}  // namespace spark
