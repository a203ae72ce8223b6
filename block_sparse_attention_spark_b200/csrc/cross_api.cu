// Cross attention entry points: checks, choice of the kernel, workspace.
#include <math.h>

#include "cross.h"

namespace spark {
namespace cross {

static spark_status validate(const spark_cross_params* p) {
  if (p == nullptr || p->B < 1 || p->Hq < 1 || p->Hkv < 1 || p->Nq < 1 || p->Nk < 1 || p->d < 1)
    return SPARK_ERR_INVALID_ARG;
  // (the kernels have scale log2 e in 32 bits)
  if (p->Hq % p->Hkv != 0 || !isfinite((float)(p->scale * 1.4426950408889634)) || p->scale < 0.0)
    return SPARK_ERR_INVALID_ARG;
  if (p->dtype < SPARK_BF16 || p->dtype > SPARK_FP32) return SPARK_ERR_INVALID_ARG;
  if (p->dtype == SPARK_FP32) return SPARK_ERR_UNSUPPORTED;
  if (p->d != 64 && p->d != 128) return SPARK_ERR_UNSUPPORTED;
  if (p->Nq > SPARK_CROSS_MAX_TOKENS || p->Nk > SPARK_CROSS_MAX_TOKENS) return SPARK_ERR_UNSUPPORTED;
  if ((int64_t)p->B * p->Hq > 65535 || (int64_t)p->B * p->Hq * p->Nq > INT32_MAX ||
      (int64_t)p->B * p->Hkv * p->Nk > INT32_MAX)
    return SPARK_ERR_UNSUPPORTED;
  return SPARK_OK;
}

static Problem problem(const spark_cross_params* p) {
  Problem c = {};
  c.B = p->B; c.Hq = p->Hq; c.Hkv = p->Hkv; c.G = p->Hq / p->Hkv;
  c.Nq = p->Nq; c.Nk = p->Nk; c.d = p->d;
  c.fp16 = p->dtype == SPARK_FP16;
  c.scale = (float)(p->scale > 0.0 ? p->scale : 1.0 / sqrt((double)p->d));
  return c;
}

// Up to 16 rows of a key head (query heads of its group times tokens), one tile:
// always the few-row kernel, which reads K and V once. More: the kernel whose
// estimate is less, both in keys' time of the few-row kernel (about 11.5 ns at
// d = 128, 6 at 64): keys a block works on, plus what starting a block, cutting
// the keys into shares and reading the first tile cost. Measured on both sides,
// few / many, us: d = 128: 16 heads of 512 keys: 32 rows 6.6 / 9.3, 64 8.0 / 10.1,
// 128 10.8 / 11.1, 256 19.3 / 14.2; 8 heads of 8192: 16 rows 13.6 / 17.8, 32 19.2 /
// 17.8, 128 51 / 21; 256 heads of 77: 32 rows 6.3 / 7.3, 64 11.1 / 7.3; one key head
// of 16384: 64 rows 14.5 / 16.6, 128 19.2 / 16.5. d = 64: 160 heads of 512: 32 rows
// 12.0 / 16.0, 64 18.3 / 16.6; 2 key heads of 2048: 512 rows 10.8 / 13.1, 768 14.8 / 13.2.
static bool few_rows(const Problem& c) {
  if ((int64_t)c.G * c.Nq <= 16) return true;
  int64_t few, many;
  int shares;
  few_keys(c, &few);
  many_keys(c, &many, &shares);
  if (c.d == 128) return few <= 300 + many + (shares > 1 ? 220 + 8 * std::min(shares, 32) : 0);
  return few <= 450 + many * 8 / 5 + (shares > 1 ? 600 + 15 * std::min(shares, 24) : 0);
}

// Workspace: what the kernels themselves need, and behind it room for the kept
// keys of a masked call, packed to the front for the tensor-core kernels (the
// size covers calls with and without a mask).
static size_t forward_bytes(const Problem& c, bool few) { return few ? few_workspace(c) : align_up(many_workspace(c)); }
static size_t backward_bytes(const Problem& c) { return align_up(bwd_workspace(c)); }
static size_t total_bytes(const Problem& c, size_t own, bool packs) { return own + (packs ? pack_plan(c).bytes : 0) + WS_SLACK; }

// What packing a masked problem's keys into ws takes; the problem is then the packed one.
static PackArgs pack(Problem* c, char* ws) {
  const Packed pk = pack_plan(*c);
  const PackArgs a = pack_args(*c, pk, ws);
  if (c->key_mask != nullptr) {
    const int64_t head = (int64_t)c->Nk * c->d;
    c->k = View{a.ko, c->Hkv * head, head, c->d};
    c->v = View{a.vo, c->Hkv * head, head, c->d};
    c->key_len = a.count;
  }
  return a;
}

}  // namespace cross
}  // namespace spark

using namespace spark;

extern "C" {

spark_status spark_cross_validate(const spark_cross_params* p) { return cross::validate(p); }

size_t spark_cross_workspace_size(const spark_cross_params* p, int32_t bwd) {
  if (cross::validate(p) != SPARK_OK || (bwd && p->dtype != SPARK_BF16)) return 0;
  const cross::Problem c = cross::problem(p);
  if (bwd) return cross::total_bytes(c, cross::backward_bytes(c), true);
  const bool few = cross::few_rows(c);
  return cross::total_bytes(c, cross::forward_bytes(c, few), !few);
}

spark_status spark_cross_attn(const spark_cross_params* p, const spark_view* q, const spark_view* k,
                              const spark_view* v, const int32_t* key_len, const uint8_t* key_mask,
                              const spark_view* out, float* lse, void* ws, size_t ws_bytes,
                              cudaStream_t stream) {
  const spark_status vs = cross::validate(p);
  if (vs != SPARK_OK) return vs;
  cross::Problem c = cross::problem(p);
  if (!make_view(q, c.B, c.Hq, c.Nq, c.d, 2, false, &c.q) || !make_view(k, c.B, c.Hkv, c.Nk, c.d, 2, false, &c.k) ||
      !make_view(v, c.B, c.Hkv, c.Nk, c.d, 2, false, &c.v) || !make_view(out, c.B, c.Hq, c.Nq, c.d, 2, true, &c.out))
    return SPARK_ERR_INVALID_ARG;
  if (((uintptr_t)key_len & 3u) != 0 || ((uintptr_t)lse & 3u) != 0) return SPARK_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws)) return SPARK_ERR_INVALID_ARG;
  const bool few = cross::few_rows(c);
  const size_t own = cross::forward_bytes(c, few);
  if (ws_bytes < cross::total_bytes(c, own, !few)) return SPARK_ERR_WORKSPACE;
  c.key_len = key_len;
  c.key_mask = key_mask;
  c.lse = lse;
  c.status = device_status();
  char* base = cross::workspace_base(ws);
  if (few) return cross::launch_few(c, base, stream) == cudaSuccess ? SPARK_OK : SPARK_ERR_CUDA;
  const cross::PackArgs packed = cross::pack(&c, base + own);
  if (packed.mask != nullptr && cross::launch_pack(packed, stream) != cudaSuccess) return SPARK_ERR_CUDA;
  return cross::launch_many(c, packed.mask != nullptr, base, stream) == cudaSuccess ? SPARK_OK : SPARK_ERR_CUDA;
}

spark_status spark_cross_attn_bwd(const spark_cross_params* p, const spark_view* q, const spark_view* k,
                                  const spark_view* v, const spark_view* out, const float* lse,
                                  const spark_view* dout, const int32_t* key_len, const uint8_t* key_mask,
                                  const spark_view* dq, const spark_view* dk, const spark_view* dv, void* ws,
                                  size_t ws_bytes, cudaStream_t stream) {
  const spark_status vs = cross::validate(p);
  if (vs != SPARK_OK) return vs;
  if (p->dtype != SPARK_BF16) return SPARK_ERR_UNSUPPORTED;
  cross::Problem c = cross::problem(p);
  cross::Gradients g = {};
  if (!make_view(q, c.B, c.Hq, c.Nq, c.d, 2, false, &c.q) || !make_view(k, c.B, c.Hkv, c.Nk, c.d, 2, false, &c.k) ||
      !make_view(v, c.B, c.Hkv, c.Nk, c.d, 2, false, &c.v) || !make_view(out, c.B, c.Hq, c.Nq, c.d, 2, false, &c.out) ||
      !make_view(dout, c.B, c.Hq, c.Nq, c.d, 2, false, &g.dout) ||
      !make_view(dq, c.B, c.Hq, c.Nq, c.d, 2, true, &g.dq) || !make_view(dk, c.B, c.Hkv, c.Nk, c.d, 2, true, &g.dk) ||
      !make_view(dv, c.B, c.Hkv, c.Nk, c.d, 2, true, &g.dv))
    return SPARK_ERR_INVALID_ARG;
  if (lse == nullptr || ((uintptr_t)lse & 3u) != 0 || ((uintptr_t)key_len & 3u) != 0) return SPARK_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws)) return SPARK_ERR_INVALID_ARG;
  const size_t own = cross::backward_bytes(c);
  if (ws_bytes < cross::total_bytes(c, own, true)) return SPARK_ERR_WORKSPACE;
  g.lse = lse;
  c.key_len = key_len;
  c.key_mask = key_mask;
  c.status = device_status();
  char* base = cross::workspace_base(ws);
  const cross::PackArgs packed = cross::pack(&c, base + own);
  return cross::launch_bwd(c, g, packed, base, stream) == cudaSuccess ? SPARK_OK : SPARK_ERR_CUDA;
}

}  // extern "C"
