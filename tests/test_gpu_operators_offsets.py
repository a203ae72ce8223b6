"""Rows that lie more than 2^32 elements apart: every kernel's offsets are 64 bits."""

import pytest
import torch

import block_sparse_attention_spark_b200 as spark
from tests.test_gpu_cross import inputs
from tests.test_gpu_cross_logits import uses_tensor_cores

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def memory():
    """20 GB, of which a test uses the rows it writes."""
    t = torch.empty(10 << 30, dtype=torch.bfloat16, device="cuda")
    yield t
    del t
    torch.cuda.empty_cache()


def far(memory, like, at=0):
    """A copy of `like` [B,H,N,d] whose tokens are as far apart as the memory allows, items and heads beside each other."""
    B, H, N, d = like.shape
    step = (memory.numel() // N - 4096) // 64 * 64
    assert step * (N - 1) > 1 << 32 and B * H * d <= step
    t = memory.as_strided((B, H, N, d), (H * d, d, step, 1), at)
    t.copy_(like)
    return t


# few rows in a block, a cluster and split; tensor-core rows, with a mask (packed), with split keys
@pytest.mark.parametrize("c,many", [
    ((1, 3, 3, 2, 90, 64, "bf16", "none"), False), ((2, 4, 2, 3, 500, 64, "bf16", "mask"), False),
    ((1, 1, 1, 1, 40000, 64, "bf16", "none"), False), ((1, 120, 120, 300, 300, 64, "bf16", "none"), True),
    ((2, 60, 30, 150, 200, 128, "bf16", "mask"), True), ((1, 2, 2, 300, 5000, 64, "bf16", "lengths"), True),
])
def test_cross_attention_and_gradient_of_far_rows(memory, c, many):
    p, q, k, v, kw = inputs(*c)
    assert uses_tensor_cores(p) == many
    g = torch.Generator(device="cuda").manual_seed(3)
    dout = torch.randn(q.shape, generator=g, device="cuda").to(q.dtype)
    want, lse = spark.cross_attn(p, q, k, v, return_lse=True, **kw)
    grads = spark.cross_attn_bwd(p, q, k, v, want, lse, dout, **kw)
    names = ["k", "v"] + (["q", "out"] if p.Nq > 1 else [])
    for name in names:
        t = {"q": q, "k": k, "v": v, "out": want}
        t[name] = far(memory, t[name])
        if name == "out":
            t["out"].zero_()
            got = spark.cross_attn(p, q, k, v, out=t["out"], **kw)
            assert got.data_ptr() == t["out"].data_ptr() and torch.equal(got, want)
        else:
            got, got_lse = spark.cross_attn(p, t["q"], t["k"], t["v"], return_lse=True, **kw)
            assert torch.equal(got, want) and torch.equal(got_lse, lse)
        again = spark.cross_attn_bwd(p, t["q"], t["k"], t["v"], t["out"], lse, dout, **kw)
        assert all(torch.equal(a, b) for a, b in zip(again, grads))
    if p.Nq > 1:
        again = spark.cross_attn_bwd(p, q, k, v, want, lse, far(memory, dout), **kw)
        assert all(torch.equal(a, b) for a, b in zip(again, grads))
    assert spark.get_status() == 0


@pytest.mark.parametrize("dtype,pairing,norm", [("bf16", "interleaved", True), ("bf16", "halves", False)])
def test_rotary_of_far_rows(memory, dtype, pairing, norm):
    g = torch.Generator(device="cuda").manual_seed(4)
    B, H, N, d = 2, 3, 77, 128
    q, k, dq, dk = (torch.randn(B, H, N, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda") if norm else None
    p = spark.rotary_params(B, H, N, d, (44, 42, 42), grid=(7, 11, 1), dtype=dtype, pairing=pairing)
    want = spark.rotary(p, q, k, q_weight=w)
    grads = spark.rotary_bwd(p, dq, dk, q, k, q_weight=w)
    got = spark.rotary(p, far(memory, q), k, q_weight=w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = far(memory, q)
    got = spark.rotary(p, x, k, q_weight=w, out=(x, torch.empty_like(k)))
    assert torch.equal(x, want[0]) and torch.equal(got[1], want[1])
    got = spark.rotary_bwd(p, far(memory, dq), dk, q, k, q_weight=w)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, grads))
    got = spark.rotary_bwd(p, dq, dk, far(memory, q), k, q_weight=w)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, grads))
