// Kept keys of a masked cross attention moved to the front, so that the
// tensor-core kernels see a plain length: what is dropped is not computed, and
// never read again.
//
// One block of 256 threads per chunk of a key head: 64 keys, more once a head
// has over 1,536 chunks, so that what the blocks count stays in proportion to the
// keys. It counts the kept keys before its chunk (the mask is a byte per key and
// stays in cache, 16 read at a time), then, 64 at a time, ranks its own and copies
// their rows of k and v, four threads a row. Reads and writes each kept row once:
// a few microseconds for an encoder's states, most of it launch and latency.
#pragma once

#include "common.cuh"
#include "cross.h"

namespace spark {
namespace cross {

constexpr int PACK_CHUNK = 64, PACK_THREADS = 256;

// Chunks of a key head, and the 64-key pieces of each.
__host__ __device__ inline int pack_pieces(int Nk) { return (Nk + 1536 * PACK_CHUNK - 1) / (1536 * PACK_CHUNK); }
__host__ __device__ inline int pack_chunks(int Nk) {
  const int keys = PACK_CHUNK * pack_pieces(Nk);
  return (Nk + keys - 1) / keys;
}
inline int64_t pack_blocks(const PackArgs& a) { return a.mask == nullptr ? 0 : (int64_t)pack_chunks(a.Nk) * a.Hkv * a.B; }

// Kept keys among the first n of a mask, this thread's share of them.
__device__ __forceinline__ int count_kept(const uint8_t* mask, int n, int tid) {
  const int head = min(n, (int)((16 - ((uintptr_t)mask & 15)) & 15));    // up to a 16-byte boundary
  const int words = (n - head) / 16, tail = head + 16 * words;
  int c = 0;
  for (int j = tid; j < head; j += PACK_THREADS) c += mask[j] != 0;
  const uint4* w = reinterpret_cast<const uint4*>(mask + head);
#pragma unroll 4
  for (int j = tid; j < words; j += PACK_THREADS) {
    const uint4 x = w[j];
    const unsigned zeros = __popc(__vcmpeq4(x.x, 0)) + __popc(__vcmpeq4(x.y, 0)) + __popc(__vcmpeq4(x.z, 0)) + __popc(__vcmpeq4(x.w, 0));
    c += 16 - (int)zeros / 8;
  }
  for (int j = tail + tid; j < n; j += PACK_THREADS) c += mask[j] != 0;
  return c;
}

__device__ __forceinline__ void pack_block(const PackArgs& a, int block) {
  __shared__ int warp_sum_sh[PACK_THREADS / 32];
  __shared__ int place_sh[PACK_CHUNK];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = pack_chunks(a.Nk), pieces = pack_pieces(a.Nk);
  const int first = block % chunks * pieces * PACK_CHUNK, end = min(a.Nk, first + pieces * PACK_CHUNK);
  const int hk = block / chunks % a.Hkv, b = block / chunks / a.Hkv;
  const int len = item_len(a.key_len, a.Nk, b, a.status, tid == 0 && first == 0 && hk == 0);
  const uint8_t* mask = a.mask + (size_t)b * a.Nk;
  const int c = __reduce_add_sync(0xffffffffu, count_kept(mask, min(first, len), tid));
  if (lane == 0) warp_sum_sh[warp] = c;
  __syncthreads();
  int before = 0;                            // kept keys before the piece (of warp 0)
#pragma unroll
  for (int w = 0; w < PACK_THREADS / 32; ++w) before += warp_sum_sh[w];
  for (int j0 = first; j0 < end; j0 += PACK_CHUNK) {
    if (warp == 0) {
#pragma unroll
      for (int x = 0; x < PACK_CHUNK; x += 32) {
        const int j = j0 + x + lane;
        const bool kept = j < len && mask[j] != 0;
        const unsigned bits = __ballot_sync(0xffffffffu, kept);
        const int at = kept ? before + __popc(bits & ((1u << lane) - 1u)) : -1;
        place_sh[x + lane] = at;
        if (hk == 0 && j < a.Nk) a.place[(size_t)b * a.Nk + j] = at;
        before += __popc(bits);
      }
      if (hk == 0 && lane == 0 && j0 + PACK_CHUNK >= a.Nk) a.count[b] = before;
    }
    __syncthreads();
    const int row = tid >> 2, at = place_sh[row];
    if (at >= 0) {
      const int j = j0 + row;
      const size_t to = (((size_t)b * a.Hkv + hk) * a.Nk + at) * a.d * 2;
      const char* ks = a.k.data + 2 * (b * a.k.b + hk * a.k.h + (int64_t)j * a.k.n);
      const char* vs = a.v.data + 2 * (b * a.v.b + hk * a.v.h + (int64_t)j * a.v.n);
      uint4 kx[4], vx[4];                    // a quarter of the row, all on its way at once
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((tid & 3) + 4 * i < a.d / 8) {
          kx[i] = *reinterpret_cast<const uint4*>(ks + 16 * ((tid & 3) + 4 * i));
          vx[i] = *reinterpret_cast<const uint4*>(vs + 16 * ((tid & 3) + 4 * i));
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((tid & 3) + 4 * i < a.d / 8) {
          *reinterpret_cast<uint4*>(a.ko + to + 16 * ((tid & 3) + 4 * i)) = kx[i];
          *reinterpret_cast<uint4*>(a.vo + to + 16 * ((tid & 3) + 4 * i)) = vx[i];
        }
    }
    if (j0 + PACK_CHUNK < end) __syncthreads();          // place_sh has been read
  }
}

}  // namespace cross
}  // namespace spark
