"""Spark-Attn block-sparse attention forward pass on B200 (sm_100a).

Thin ctypes binding of libspark (include/spark.h): every function marshals
torch tensors into pointers and calls the C ABI on the current CUDA stream.
All arithmetic runs in the library's CUDA kernels; there is no CPU path.
Build the library first:  python -m block_sparse_attention_spark_b200.build
"""

from __future__ import annotations

import ctypes
import os

__all__ = ["SparkError", "Params", "lib", "params", "num_selected", "workspace_size",
           "host_workspace_size", "workspace_region", "alloc_workspace", "moments", "reblock",
           "positional_perm", "select", "attn_fwd", "attn_fwd_joint", "forward", "forward_joint",
           "forward_host", "get_status", "selftest_wait", "RotaryParams", "rotary_params",
           "rotary_validate", "rotary_workspace_size", "alloc_rotary_workspace", "rotary", "rotary_bwd",
           "forward_rotary", "forward_rotary_workspace_size",
           "CrossParams", "cross_params", "cross_validate", "cross_workspace_size",
           "alloc_cross_workspace", "cross_attn", "cross_attn_bwd",
           "LAYOUTS", "SUMMARIES", "TAILS", "WS", "DTYPES", "PAIRINGS", "SPECTRA"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspark.so")

LAYOUTS = {"q_reuse_k": 0, "k_reuse_q": 1, "separate": 2}
SUMMARIES = {"reweight": 0, "meanpool": 1}
TAILS = {"query": 0, "block": 1}
WS = {"MQ": 0, "MK": 1, "QMEAN": 2, "PERM": 3, "SEL": 4, "QM": 5, "KM": 6, "KT": 7, "VT": 8,
      "BETA": 9, "UHAT": 10, "PAIRS": 11}
DTYPES = {"bf16": 0, "fp16": 1, "fp32": 2}
PAIRINGS = {"interleaved": 0, "halves": 1}
SPECTRA = {"axis": 0, "shared": 1}
STATUS = {0: "SPARK_OK", 1: "SPARK_ERR_INVALID_ARG", 2: "SPARK_ERR_UNSUPPORTED",
          3: "SPARK_ERR_WORKSPACE", 4: "SPARK_ERR_CUDA", 5: "SPARK_ERR_TIMEOUT"}


class SparkError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = lib().spark_strerror(code).decode() if _LIB is not None else ""
        super().__init__(f"{where}: {STATUS.get(code, code)} ({msg})")


class Params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32),
                ("d", ctypes.c_int32), ("topk_ratio", ctypes.c_double),
                ("topk_blocks", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("summary", ctypes.c_int32), ("tail", ctypes.c_int32),
                ("power_iters", ctypes.c_int32)]

    def __repr__(self):
        return (f"Params(B={self.B}, H={self.H}, N={self.N}, d={self.d}, "
                f"topk_ratio={self.topk_ratio}, topk_blocks={self.topk_blocks}, "
                f"layout={self.layout}, summary={self.summary}, tail={self.tail})")


class RotaryParams(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32),
                ("N", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("dims", ctypes.c_int32 * 3),
                ("pairing", ctypes.c_int32), ("spectrum", ctypes.c_int32),
                ("grid", ctypes.c_int32 * 3), ("theta", ctypes.c_double),
                ("start", ctypes.c_double * 3), ("scale", ctypes.c_double * 3),
                ("eps", ctypes.c_double)]

    def __repr__(self):
        return (f"RotaryParams(B={self.B}, Hq={self.Hq}, Hk={self.Hk}, N={self.N}, d={self.d}, "
                f"dims={tuple(self.dims)[:self.axes]}, grid={tuple(self.grid)[:self.axes]}, "
                f"dtype={self.dtype}, pairing={self.pairing}, spectrum={self.spectrum})")


class CrossParams(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("Nq", ctypes.c_int32), ("Nk", ctypes.c_int32), ("d", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_double)]

    def __repr__(self):
        return (f"CrossParams(B={self.B}, Hq={self.Hq}, Hkv={self.Hkv}, Nq={self.Nq}, Nk={self.Nk}, "
                f"d={self.d}, dtype={self.dtype}, scale={self.scale})")


class View(ctypes.Structure):
    """A [B,H,N,d] tensor's address and its strides in elements."""
    _fields_ = [("data", ctypes.c_void_p), ("b", ctypes.c_int64), ("h", ctypes.c_int64),
                ("n", ctypes.c_int64)]


_LIB = None
_P = ctypes.POINTER(Params)
_RP = ctypes.POINTER(RotaryParams)
_CP = ctypes.POINTER(CrossParams)
_V = ctypes.POINTER(View)
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_i32 = ctypes.c_int32

_SIGS = {
    "spark_validate": (_i32, [_P]),
    "spark_num_selected": (_i32, [_P]),
    "spark_workspace_size": (_sz, [_P]),
    "spark_host_workspace_size": (_sz, [_P]),
    "spark_forward_launches": (_i32, [_P]),
    "spark_workspace_region": (_sz, [_P, _i32, ctypes.POINTER(_sz)]),
    "spark_moments": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spark_moments_noalloc": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp]),
    "spark_reblock": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spark_positional_perm": (_i32, [_P, _i32, _i32, _i32, _vp, _vp]),
    "spark_select": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spark_attn_fwd": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spark_forward": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spark_attn_fwd_joint": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spark_forward_joint": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _sz,
                                   _vp]),
    "spark_forward_host": (_i32, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spark_get_status": (_i32, [_vp]),
    "spark_selftest_wait": (_i32, [ctypes.c_int64, _vp]),
    "spark_strerror": (ctypes.c_char_p, [_i32]),
    "spark_rotary_validate": (_i32, [_RP]),
    "spark_rotary_workspace_size": (_sz, [_RP]),
    "spark_rotary": (_i32, [_RP, _V, _V, _vp, _vp, _vp, _V, _V, _vp]),
    "spark_rotary_bwd": (_i32, [_RP, _V, _V, _V, _V, _vp, _vp, _vp, _V, _V, _vp, _vp, _vp, _sz, _vp]),
    "spark_forward_rotary_workspace_size": (_sz, [_P]),
    "spark_forward_rotary": (_i32, [_P, _RP, _V, _V, _V, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "spark_cross_validate": (_i32, [_CP]),
    "spark_cross_workspace_size": (_sz, [_CP, _i32]),
    "spark_cross_attn": (_i32, [_CP, _V, _V, _V, _vp, _vp, _V, _vp, _vp, _sz, _vp]),
    "spark_cross_attn_bwd": (_i32, [_CP, _V, _V, _V, _V, _vp, _V, _vp, _vp, _V, _V, _V, _vp, _sz, _vp]),
}


def lib():
    """The loaded libspark (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libspark.so not found at {LIB_PATH}; build it with "
                               "`python -m block_sparse_attention_spark_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _check(code: int, where: str):
    if code != 0:
        raise SparkError(code, where)


def params(B, H, N, d, topk_ratio=0.2, topk_blocks=0, layout="q_reuse_k",
           summary="reweight", tail="query", power_iters=0) -> Params:
    return Params(B, H, N, d, float(topk_ratio), int(topk_blocks), LAYOUTS[layout],
                  SUMMARIES[summary], TAILS[tail], int(power_iters))


def validate(p: Params) -> int:
    return lib().spark_validate(ctypes.byref(p))


def num_selected(p: Params) -> int:
    return lib().spark_num_selected(ctypes.byref(p))


def workspace_size(p: Params) -> int:
    return lib().spark_workspace_size(ctypes.byref(p))


def forward_launches(p: Params) -> int:
    """Kernel launches one spark_forward call makes."""
    return lib().spark_forward_launches(ctypes.byref(p))


def host_workspace_size(p: Params) -> int:
    return lib().spark_host_workspace_size(ctypes.byref(p))


def workspace_region(p: Params, name: str):
    """(byte offset, byte size) of a named workspace region."""
    n = _sz(0)
    off = lib().spark_workspace_region(ctypes.byref(p), WS[name], ctypes.byref(n))
    if off == ctypes.c_size_t(-1).value:
        raise SparkError(1, "spark_workspace_region")
    return off, n.value


# ---------------------------------------------------------------- torch glue

_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream():
    return _torch().cuda.current_stream().cuda_stream


def _ptr(t):
    if t is None:
        return None
    return t.data_ptr()


def _need(t, dtype, shape, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                        f"got {t.dtype} {tuple(t.shape)}")


def alloc_workspace(p: Params, host=False):
    torch = _torch()
    n = host_workspace_size(p) if host else workspace_size(p)
    if n == 0:
        _check(validate(p) or 1, "workspace_size")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def ws_view(ws, p: Params, name: str, dtype, shape):
    """A typed view of one workspace region (no copy)."""
    off, n = workspace_region(p, name)
    esz = _torch().tensor([], dtype=dtype).element_size()
    count = 1
    for s in shape:
        count *= s
    assert count * esz <= n
    return ws[off:off + count * esz].view(dtype).view(*shape)


def moments(p: Params, q, k, ws, which="both"):
    """M_Q, M_K (float64 [B,H,d,d]) and the anchor qbar ([B,H,d]).
    which="layout" forms only the moment(s) the layout partitions under (the
    others come back as None), as spark_forward does."""
    torch = _torch()
    shp = (p.B, p.H, p.N, p.d)
    _need(q, torch.bfloat16, shp, "q")
    _need(k, torch.bfloat16, shp, "k")
    if which not in ("both", "layout"):
        raise ValueError(which)
    lay = p.layout
    want_q = which == "both" or lay != LAYOUTS["q_reuse_k"]
    want_k = which == "both" or lay != LAYOUTS["k_reuse_q"]
    MQ = torch.empty(p.B, p.H, p.d, p.d, dtype=torch.float64, device="cuda") if want_q else None
    MK = torch.empty(p.B, p.H, p.d, p.d, dtype=torch.float64, device="cuda") if want_k else None
    qmean = torch.empty(p.B, p.H, p.d, dtype=torch.float64, device="cuda")
    _check(lib().spark_moments(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(MQ), _ptr(MK), _ptr(qmean),
                               _ptr(ws), ws.numel(), _stream()), "spark_moments")
    return MQ, MK, qmean


def moments_noalloc(p: Params, q, k, MQ, MK, qmean):
    """spark_moments without a workspace: the library's own fixed device
    array holds the partial sums (see include/spark.h for its limit and the
    rules on overlapping calls). Outputs are written into the given tensors."""
    torch = _torch()
    shp = (p.B, p.H, p.N, p.d)
    _need(q, torch.bfloat16, shp, "q")
    _need(k, torch.bfloat16, shp, "k")
    _need(MQ, torch.float64, (p.B, p.H, p.d, p.d), "MQ")
    _need(MK, torch.float64, (p.B, p.H, p.d, p.d), "MK")
    _need(qmean, torch.float64, (p.B, p.H, p.d), "qmean")
    _check(lib().spark_moments_noalloc(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(MQ), _ptr(MK),
                                       _ptr(qmean), _stream()), "spark_moments_noalloc")
    return MQ, MK, qmean


def perm_shape(p: Params):
    """[B, H, N], or [2, B, H, N] (query, then key permutation) for the separate layout."""
    return (2, p.B, p.H, p.N) if p.layout == LAYOUTS["separate"] else (p.B, p.H, p.N)


def reblock(p: Params, q, k, MQ, MK, ws):
    torch = _torch()
    perm = torch.empty(perm_shape(p), dtype=torch.int32, device="cuda")
    _check(lib().spark_reblock(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(MQ), _ptr(MK), _ptr(perm),
                               _ptr(ws), ws.numel(), _stream()), "spark_reblock")
    return perm


def positional_perm(p: Params, grid):
    torch = _torch()
    F, Hl, Wl = grid
    perm = torch.empty(perm_shape(p), dtype=torch.int32, device="cuda")
    _check(lib().spark_positional_perm(ctypes.byref(p), F, Hl, Wl, _ptr(perm), _stream()),
           "spark_positional_perm")
    return perm


def select(p: Params, q, k, v, perm, qmean, ws):
    torch = _torch()
    ksel = num_selected(p)
    sel = torch.empty(p.B, p.H, p.N // 64, ksel, dtype=torch.int32, device="cuda")
    _check(lib().spark_select(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(perm), _ptr(qmean),
                              _ptr(sel), _ptr(ws), ws.numel(), _stream()), "spark_select")
    return sel


def attn_fwd(p: Params, perm, sel, ws, return_lse=False):
    torch = _torch()
    out = torch.empty(p.B, p.H, p.N, p.d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(p.B, p.H, p.N, dtype=torch.float32, device="cuda") if return_lse else None
    _check(lib().spark_attn_fwd(ctypes.byref(p), _ptr(perm), _ptr(sel), _ptr(out), _ptr(lse),
                                _ptr(ws), ws.numel(), _stream()), "spark_attn_fwd")
    return (out, lse) if return_lse else out


def attn_fwd_joint(p: Params, perm, sel, qc, kc, vc, ws, return_lse=False):
    """Video rows with the context segment, and the context rows (dense).
    qc, kc, vc: [B, H, C, d] bf16. Returns (out, outc) or (out, outc, lse, lsec)."""
    torch = _torch()
    C = qc.shape[2]
    for t, n in ((qc, "qc"), (kc, "kc"), (vc, "vc")):
        _need(t, torch.bfloat16, (p.B, p.H, C, p.d), n)
    out = torch.empty(p.B, p.H, p.N, p.d, dtype=torch.bfloat16, device="cuda")
    outc = torch.empty(p.B, p.H, C, p.d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(p.B, p.H, p.N, dtype=torch.float32, device="cuda") if return_lse else None
    lsec = torch.empty(p.B, p.H, C, dtype=torch.float32, device="cuda") if return_lse else None
    _check(lib().spark_attn_fwd_joint(ctypes.byref(p), _ptr(perm), _ptr(sel), _ptr(qc), _ptr(kc), _ptr(vc), C,
                                      _ptr(out), _ptr(lse), _ptr(outc), _ptr(lsec), _ptr(ws), ws.numel(),
                                      _stream()), "spark_attn_fwd_joint")
    return (out, outc, lse, lsec) if return_lse else (out, outc)


def forward_joint(p: Params, q, k, v, qc, kc, vc, ws=None):
    """The whole pass with a context segment. Returns (out, outc)."""
    torch = _torch()
    C = qc.shape[2]
    shp = (p.B, p.H, p.N, p.d)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, shp, n)
    for t, n in ((qc, "qc"), (kc, "kc"), (vc, "vc")):
        _need(t, torch.bfloat16, (p.B, p.H, C, p.d), n)
    if ws is None:
        ws = alloc_workspace(p)
    out = torch.empty(shp, dtype=torch.bfloat16, device="cuda")
    outc = torch.empty(p.B, p.H, C, p.d, dtype=torch.bfloat16, device="cuda")
    _check(lib().spark_forward_joint(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(qc), _ptr(kc), _ptr(vc), C,
                                     _ptr(out), None, _ptr(outc), None, _ptr(ws), ws.numel(), _stream()),
           "spark_forward_joint")
    return out, outc


def forward(p: Params, q, k, v, ws=None, out=None, lse=None, perm=None, sel=None):
    """The whole pass on device tensors. Returns out (and writes lse/perm/sel
    into the given tensors when they are passed)."""
    torch = _torch()
    shp = (p.B, p.H, p.N, p.d)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, shp, n)
    if ws is None:
        ws = alloc_workspace(p)
    if out is None:
        out = torch.empty(shp, dtype=torch.bfloat16, device="cuda")
    _check(lib().spark_forward(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                               _ptr(perm), _ptr(sel), _ptr(ws), ws.numel(), _stream()),
           "spark_forward")
    return out


def forward_host(p: Params, q_host, k_host, v_host, out_host, ws, lse_host=None):
    """The whole pass on host tensors (CPU torch tensors, pinned for speed)."""
    _check(lib().spark_forward_host(ctypes.byref(p), _ptr(q_host), _ptr(k_host), _ptr(v_host),
                                    _ptr(out_host), _ptr(lse_host), _ptr(ws), ws.numel(),
                                    _stream()), "spark_forward_host")
    return out_host


# ------------------------------------------- rotary positions, cross attention
# Tensors are [B, H, N, d] views: any strides over batch, head and token with
# the last axis contiguous (a projection's [B, N, H, d] result goes in as
# x.transpose(1, 2)). All tensors of a call are on one device, the call's
# kernels on that device's current stream.

_DT = None            # torch's types by code


def _dtype_of(code):
    global _DT
    if _DT is None:
        torch = _torch()
        _DT = (torch.bfloat16, torch.float16, torch.float32)
    return _DT[code]


def _wrong(t, name, dev, dtype, shape, what):
    """The error of a tensor that is not the one asked for."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != dev:
        return TypeError(f"{name} must be a CUDA tensor on cuda:{dev}")
    return TypeError(f"{name} must be {what} {dtype} tensor of shape {tuple(shape)}, "
                     f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()}")


def _on(t, name, dev, dtype, shape):
    """Address of a contiguous tensor of this device (by number), type and shape."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    raise _wrong(t, name, dev, dtype, shape, "a contiguous")


def _view(t, name, dev, dtype, shape):
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            b, h, n, one = t.stride()
            if one == 1:
                return View(t.data_ptr(), b, h, n)
    except AttributeError:
        pass
    raise _wrong(t, name, dev, dtype, shape, "a (last axis contiguous)")


def _made(t):
    """View of a tensor made here like one that _view has looked at."""
    b, h, n, one = t.stride()
    if one != 1:
        raise RuntimeError(f"a result's last axis has stride {one}")
    return View(t.data_ptr(), b, h, n)


def _device(t, name):
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _call(fn, where, dev, *args):
    """A library call on the device's current stream, with that device current."""
    torch = _torch()
    if torch._C._cuda_getDevice() == dev:
        code = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if code != 0:
        raise SparkError(code, where)


def _scratch(ws, size, dev, where):
    torch = _torch()
    if ws is None:
        return torch.empty(size(), dtype=torch.uint8, device=dev)
    if not isinstance(ws, torch.Tensor) or ws.get_device() != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise TypeError(f"{where}: ws must be a contiguous uint8 tensor on cuda:{dev}")
    return ws


def rotary_params(B, H, N, d, dims, heads_k=None, grid=None, dtype="bf16", pairing="interleaved",
                  spectrum="axis", theta=10000.0, start=(0.0, 0.0, 0.0), scale=(1.0, 1.0, 1.0),
                  eps=1e-6) -> RotaryParams:
    """Parameters of rotary / rotary_bwd for H query and heads_k (default H; 0:
    none) key heads. dims: rotated values per axis (one to three axes); grid:
    the tokens' raster grid, as many extents as dims, or None when every call
    gets positions."""
    dims = tuple(int(x) for x in dims)
    axes = len(dims)
    if not 1 <= axes <= 3:
        raise ValueError("dims: one to three axes")
    grid = (0,) * axes if grid is None else tuple(int(x) for x in grid)
    if len(grid) != axes:
        raise ValueError("grid: as many extents as dims")
    i3, d3 = ctypes.c_int32 * 3, ctypes.c_double * 3
    return RotaryParams(B, H, H if heads_k is None else heads_k, N, d, DTYPES[dtype], axes, i3(*dims),
                        PAIRINGS[pairing], SPECTRA[spectrum], i3(*grid), float(theta),
                        d3(*(float(x) for x in start)), d3(*(float(x) for x in scale)), float(eps))


def rotary_validate(p: RotaryParams) -> int:
    return lib().spark_rotary_validate(ctypes.byref(p))


def rotary_workspace_size(p: RotaryParams) -> int:
    """Bytes of workspace rotary_bwd needs when a norm weight is given."""
    return lib().spark_rotary_workspace_size(ctypes.byref(p))


def alloc_rotary_workspace(p: RotaryParams, device="cuda"):
    n = rotary_workspace_size(p)
    if n == 0:
        _check(rotary_validate(p) or 1, "rotary_workspace_size")
    return _torch().empty(n, dtype=_torch().uint8, device=device)


def _rotary_extras(p, device, dtype, positions, q_weight, k_weight):
    pos = None if positions is None else _on(positions, "positions", device, _dtype_of(2), (p.B, p.N, p.axes))
    wq = None if q_weight is None else _on(q_weight, "q_weight", device, dtype, (p.d,))
    wk = None if k_weight is None else _on(k_weight, "k_weight", device, dtype, (p.d,))
    return pos, wq, wk


def rotary(p: RotaryParams, q, k=None, positions=None, q_weight=None, k_weight=None, out=None):
    """Rotary positions of q [B,Hq,N,d] and k [B,Hk,N,d] (None when heads_k is
    0), after the per-head RMS norm of those with a weight ([d]). positions:
    [B,N,axes] float32, default the parameters' grid. Returns (q_out, k_out),
    contiguous [B,H,N,d] as forward() reads them, or the tensors of
    out=(q_out, k_out), which may be q and k themselves."""
    torch = _torch()
    dev, dt = _device(q, "q"), _dtype_of(p.dtype)
    qs, ks = (p.B, p.Hq, p.N, p.d), (p.B, p.Hk, p.N, p.d)
    if (k is None) != (p.Hk == 0):
        raise TypeError("k: given exactly when the parameters have key heads")
    vq = _view(q, "q", dev, dt, qs)
    vk = None if k is None else _view(k, "k", dev, dt, ks)
    pos = wq = wk = None
    if positions is not None or q_weight is not None or k_weight is not None:
        pos, wq, wk = _rotary_extras(p, dev, dt, positions, q_weight, k_weight)
    if out is None:
        qo = torch.empty_like(q, memory_format=torch.contiguous_format)
        ko = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
        wqo, wko = _made(qo), None if k is None else _made(ko)
    else:
        qo, ko = out
        wqo = _view(qo, "q_out", dev, dt, qs)
        wko = None if k is None else _view(ko, "k_out", dev, dt, ks)
    _call(lib().spark_rotary, "spark_rotary", dev, p, vq, vk, pos, wq, wk, wqo, wko)
    return qo, ko


def rotary_bwd(p: RotaryParams, dq_out, dk_out=None, q=None, k=None, positions=None, q_weight=None,
               k_weight=None, ws=None):
    """Gradient of rotary: (dq, dk, dq_weight, dk_weight) from the gradients of
    its outputs. q and k, its inputs, are needed where that tensor has a
    weight; dq and dk come in their layout when they are given (contiguous
    otherwise), weight gradients as float32 [d] (None without a weight)."""
    torch = _torch()
    dev, dt = _device(dq_out, "dq_out"), _dtype_of(p.dtype)
    qs, ks = (p.B, p.Hq, p.N, p.d), (p.B, p.Hk, p.N, p.d)
    if (dk_out is None) != (p.Hk == 0):
        raise TypeError("dk_out: given exactly when the parameters have key heads")
    pos, wq, wk = _rotary_extras(p, dev, dt, positions, q_weight, k_weight)
    if (wq is not None and q is None) or (wk is not None and p.Hk and k is None):
        raise TypeError("a tensor with a norm weight is needed for its gradient")
    vq = None if q is None else _view(q, "q", dev, dt, qs)
    vk = None if k is None or p.Hk == 0 else _view(k, "k", dev, dt, ks)
    gq = _view(dq_out, "dq_out", dev, dt, qs)
    gk = None if dk_out is None else _view(dk_out, "dk_out", dev, dt, ks)
    dq = torch.empty(qs, dtype=dt, device=dev) if q is None else torch.empty_like(q)
    dk = None if dk_out is None else torch.empty(ks, dtype=dt, device=dev) if k is None else torch.empty_like(k)
    dwq = None if wq is None else torch.empty(p.d, dtype=torch.float32, device=dev)
    dwk = None if wk is None or p.Hk == 0 else torch.empty(p.d, dtype=torch.float32, device=dev)
    if wq is not None or wk is not None:
        ws = _scratch(ws, lambda: rotary_workspace_size(p), dev, "rotary_bwd")
    else:
        ws = None
    odq, odk = _made(dq), None if dk is None else _made(dk)
    _call(lib().spark_rotary_bwd, "spark_rotary_bwd", dev, p, gq, gk, vq, vk, pos, wq, wk, odq, odk, _ptr(dwq),
          _ptr(dwk), _ptr(ws), 0 if ws is None else ws.numel())
    return dq, dk, dwq, dwk


def forward_rotary_workspace_size(p: Params) -> int:
    return lib().spark_forward_rotary_workspace_size(ctypes.byref(p))


def forward_rotary(p: Params, r: RotaryParams, q, k, v, positions=None, q_weight=None, k_weight=None, ws=None,
                   out=None, lse=None):
    """The whole pass from a layer's projections: rotary(r, q, k, ...) and then
    forward(p, ...), q, k and v [B,H,N,d] of any layout. Returns out."""
    torch = _torch()
    dev, dt, shp = _device(q, "q"), _dtype_of(0), (p.B, p.H, p.N, p.d)
    views = [_view(t, n, dev, dt, shp) for t, n in ((q, "q"), (k, "k"), (v, "v"))]
    pos, wq, wk = _rotary_extras(r, dev, dt, positions, q_weight, k_weight)
    ws = _scratch(ws, lambda: forward_rotary_workspace_size(p), dev, "forward_rotary")
    if out is None:
        out = torch.empty(shp, dtype=dt, device=dev)
    _call(lib().spark_forward_rotary, "spark_forward_rotary", dev, p, r, *views, pos, wq, wk, _on(out, "out", dev, dt, shp),
          None if lse is None else _on(lse, "lse", dev, _dtype_of(2), shp[:3]), ws.data_ptr(), ws.numel())
    return out


def cross_params(B, H, Nq, Nk, d, heads_kv=None, dtype="bf16", scale=None) -> CrossParams:
    """Parameters of cross_attn / cross_attn_bwd: H query heads over heads_kv
    (default H) key heads, Nq query tokens over Nk states; scale of the logits
    (default 1/sqrt(d))."""
    if scale is not None and not scale > 0:
        raise ValueError("scale must be positive")
    return CrossParams(B, H, H if heads_kv is None else heads_kv, Nq, Nk, d, DTYPES[dtype],
                       0.0 if scale is None else float(scale))


def cross_validate(p: CrossParams) -> int:
    return lib().spark_cross_validate(ctypes.byref(p))


def cross_workspace_size(p: CrossParams, bwd=False) -> int:
    return lib().spark_cross_workspace_size(ctypes.byref(p), int(bwd))


def alloc_cross_workspace(p: CrossParams, bwd=False, device="cuda"):
    n = cross_workspace_size(p, bwd)
    if n == 0:
        _check(cross_validate(p) or 2, "cross_workspace_size")
    return _torch().empty(n, dtype=_torch().uint8, device=device)


def _cross_masks(p, device, key_len, key_mask):
    if key_len is None and key_mask is None:
        return None, None
    torch = _torch()
    kl = None if key_len is None else _on(key_len, "key_len", device, torch.int32, (p.B,))
    kind = torch.bool if isinstance(key_mask, torch.Tensor) and key_mask.dtype == torch.bool else torch.uint8
    km = None if key_mask is None else _on(key_mask, "key_mask", device, kind, (p.B, p.Nk))
    return kl, km


def cross_attn(p: CrossParams, q, k, v, ws=None, key_len=None, key_mask=None, return_lse=False, out=None):
    """Attention of q [B,H,Nq,d] over an encoder's k, v [B,heads_kv,Nk,d].
    key_len: [B] int32, keys kept per item; key_mask: [B,Nk] bool or uint8,
    true where a key is kept; both: their intersection. Rows without a key give
    zeros (lse -inf). Returns out (contiguous, or the tensor out=, of any
    layout), with return_lse also lse [B,H,Nq] float32."""
    torch = _torch()
    dev, dt = _device(q, "q"), _dtype_of(p.dtype)
    qs, ks = (p.B, p.Hq, p.Nq, p.d), (p.B, p.Hkv, p.Nk, p.d)
    vq, vk, vv = _view(q, "q", dev, dt, qs), _view(k, "k", dev, dt, ks), _view(v, "v", dev, dt, ks)
    kl, km = _cross_masks(p, dev, key_len, key_mask)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        vo = _made(out)
    else:
        vo = _view(out, "out", dev, dt, qs)
    lse = q.new_empty(qs[:3], dtype=_dtype_of(2)) if return_lse else None
    ws = _scratch(ws, lambda: cross_workspace_size(p), dev, "cross_attn")
    _call(lib().spark_cross_attn, "spark_cross_attn", dev, p, vq, vk, vv, kl, km, vo, _ptr(lse), ws.data_ptr(),
          ws.numel())
    return (out, lse) if return_lse else out


def cross_attn_bwd(p: CrossParams, q, k, v, out, lse, dout, ws=None, key_len=None, key_mask=None):
    """Gradient of cross_attn: (dq, dk, dv), in the layouts of q, k and v, from
    dout and the out and lse that cross_attn gave for the same arguments."""
    torch = _torch()
    dev, dt = _device(q, "q"), _dtype_of(p.dtype)
    qs, ks = (p.B, p.Hq, p.Nq, p.d), (p.B, p.Hkv, p.Nk, p.d)
    views = [_view(t, n, dev, dt, s) for t, n, s in ((q, "q", qs), (k, "k", ks), (v, "v", ks), (out, "out", qs),
                                                     (dout, "dout", qs))]
    pl = _on(lse, "lse", dev, _dtype_of(2), qs[:3])
    kl, km = _cross_masks(p, dev, key_len, key_mask)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    grads = [_made(t) for t in (dq, dk, dv)]
    ws = _scratch(ws, lambda: cross_workspace_size(p, True), dev, "cross_attn_bwd")
    _call(lib().spark_cross_attn_bwd, "spark_cross_attn_bwd", dev, p, *views[:4], pl, views[4], kl, km, *grads,
          ws.data_ptr(), ws.numel())
    return dq, dk, dv


def selftest_wait(limit_ns: int):
    """Launch the bounded-wait diagnostic (see include/spark.h); the timeout
    shows up in the next get_status()."""
    _check(lib().spark_selftest_wait(int(limit_ns), _stream()), "spark_selftest_wait")


def get_status():
    """Synchronises the current stream and returns the device status code."""
    return lib().spark_get_status(_stream())
