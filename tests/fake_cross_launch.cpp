// Stands in for the kernels of cross attention, so that the entry points run on
// a machine without a GPU: keeps what they were handed.
#include "cross.h"

namespace spark {

struct Seen {
  int64_t many, bwd, packed;                 // launches of the tensor-core forward, the gradient, the packing
  uint64_t ws, pack_ws;                      // workspace of the kernel, of the packed keys
};
static Seen seen;
static size_t own_bytes = 0, pack_bytes = 0;
static bool few_is_less = false;

int* device_status() { return nullptr; }

namespace cross {

size_t few_workspace(const Problem&) { return own_bytes; }
size_t many_workspace(const Problem&) { return own_bytes; }
size_t bwd_workspace(const Problem&) { return own_bytes; }
void few_keys(const Problem&, int64_t* keys) { *keys = few_is_less ? 0 : 1 << 20; }
void many_keys(const Problem&, int64_t* keys, int* shares) { *keys = 0; *shares = 1; }
Packed pack_plan(const Problem&) { return Packed{pack_bytes, 0, 0, 0, 0}; }
PackArgs pack_args(const Problem& p, const Packed&, void* ws) {
  seen.pack_ws = reinterpret_cast<uint64_t>(ws);
  PackArgs a = {};
  a.mask = p.key_mask;
  return a;
}
cudaError_t launch_pack(const PackArgs&, cudaStream_t) { ++seen.packed; return cudaSuccess; }
cudaError_t launch_few(const Problem&, void* ws, cudaStream_t) {
  seen.ws = reinterpret_cast<uint64_t>(ws);
  return cudaSuccess;
}
cudaError_t launch_many(const Problem&, bool, void* ws, cudaStream_t) {
  ++seen.many;
  seen.ws = reinterpret_cast<uint64_t>(ws);
  return cudaSuccess;
}
cudaError_t launch_bwd(const Problem&, const Gradients&, const PackArgs&, void* ws, cudaStream_t) {
  ++seen.bwd;
  seen.ws = reinterpret_cast<uint64_t>(ws);
  return cudaSuccess;
}

}  // namespace cross
}  // namespace spark

extern "C" void fake_set(size_t own, size_t pack, int few) {
  spark::own_bytes = own;
  spark::pack_bytes = pack;
  spark::few_is_less = few != 0;
  spark::seen = {};
}
extern "C" const spark::Seen* fake_seen() { return &spark::seen; }
