"""Rotary positions and their gradient where a call is unusual and allowed."""

import ctypes

import pytest
import torch

import block_sparse_attention_spark_b200 as spark
from tests import operators64 as o64
from tests.test_gpu_rotary import CASES, case, rand

pytestmark = pytest.mark.gpu


def gradient_in_place(p, dqo, dko, q, k, wq, wk, pos):
    """rotary_bwd with dq, dk written over copies of dq_out, dk_out."""
    dq, dk = dqo.clone(), None if dko is None else dko.clone()
    dw = [None if w is None else torch.empty(p.d, dtype=torch.float32, device="cuda") for w in (wq, wk)]
    ws = spark.alloc_rotary_workspace(p)
    vq, vk, xq, xk = (None if t is None else spark.View(t.data_ptr(), *t.stride()[:3]) for t in (dq, dk, q, k))
    at = [None if t is None else t.data_ptr() for t in (pos, wq, wk, *dw)]
    code = spark.lib().spark_rotary_bwd(ctypes.byref(p), vq, vk, xq, xk, *at[:3], vq, vk, *at[3:], ws.data_ptr(), ws.numel(),
                                        torch.cuda.current_stream().cuda_stream)
    assert code == 0
    return dq, dk, *dw


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_rotary_gradient_in_place(c):
    p, q, k, wq, wk, pos, ang, pairing = case(c)
    g = torch.Generator(device="cuda").manual_seed(11)
    dqo = rand(g, q.shape, q.dtype)
    dko = None if k is None else rand(g, k.shape, k.dtype)
    want = spark.rotary_bwd(p, dqo, dko, q, k, positions=pos, q_weight=wq, k_weight=wk)
    got = gradient_in_place(p, dqo, dko, q, k, wq, wk, pos)
    for a, b in zip(got, want):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))


@pytest.mark.parametrize("N", [1, 17, 33])
def test_rotary_gradient_in_place_of_rows_that_overflow(N):
    """fp16 rows of 1e-5 (1 / rms about 1,000) whose gradients pass 65,504: those are infinite, the weight's is not,
    whatever the lanes past the last token see of the row they follow."""
    H, d = 64, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    q, dy = rand(g, (1, H, N, d), torch.float16, 1e-5), rand(g, (1, H, N, d), torch.float16, 1e3)
    w = torch.ones(d, dtype=torch.float16, device="cuda")
    p = spark.rotary_params(1, H, N, d, (44, 42, 42), heads_k=0, grid=(N, 1, 1), dtype="fp16")
    dx, _, want, _ = spark.rotary_bwd(p, dy, None, q, q_weight=w)
    assert dx.isinf().any() and want.isfinite().all()
    for _ in range(10):
        got = gradient_in_place(p, dy, None, q, None, w, None, None)
        assert torch.equal(got[0], dx) and torch.equal(got[2], want)


@pytest.mark.parametrize("spectrum,dims,d", [("axis", (44, 42, 42), 128), ("shared", (16, 24, 24), 64)])
def test_rotary_of_far_positions(spectrum, dims, d):
    """Positions as far as float32 counts tokens, whole and fractional, on both sides of zero."""
    g = torch.Generator(device="cuda").manual_seed(9)
    B, H, N = 2, 2, 500
    q = rand(g, (B, H, N, d), torch.float32)
    pos = torch.randint(-2 ** 24, 2 ** 24, (B, N, 3), generator=g, device="cuda").float()
    pos[:, ::3] = pos[:, ::3] / 64
    p = spark.rotary_params(B, H, N, d, dims, heads_k=0, dtype="fp32", spectrum=spectrum)
    ang = o64.angles(dims, spectrum, 10000.0, pos)
    got, _ = spark.rotary(p, q, positions=pos)
    want, bound = o64.rotary(q, None, ang, "interleaved", 0.0)
    # both forms of a frequency are off by at most 2^-45 of it, and the far pairs turn slowly: below a step of 2^-24 each
    o64.check(got, want, bound + 2 * 2.0 ** -24 * o64.pair_size(q.double(), sum(dims), "interleaved"), "q")
