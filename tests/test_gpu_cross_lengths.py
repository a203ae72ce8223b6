"""Lengths out of range in every kernel that reads them: clamped and reported."""

import pytest
import torch

import block_sparse_attention_spark_b200 as spark
from tests.test_gpu_cross import inputs
from tests.test_gpu_cross_logits import uses_tensor_cores

pytestmark = pytest.mark.gpu


def lengths(B, Nk):
    """Bad and good lengths of B items: below 0, past Nk, the 32-bit extremes, and some in range."""
    bad = [(-5, 0), (Nk + 1, Nk), (Nk // 2, Nk // 2), (-2 ** 31, 0), (2 ** 31 - 1, Nk), (1, 1)]
    t = torch.tensor([bad[b % len(bad)] for b in range(B)], dtype=torch.int32, device="cuda")
    return t[:, 0].contiguous(), t[:, 1].contiguous()


# few rows; many rows, keys whole and split; the gradient's tiles shared out by the host and by the device
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("B,H,Nq,Nk,d,many", [
    (6, 2, 1, 70, 64, False), (2, 2, 1, 5000, 128, False), (6, 40, 200, 300, 64, True), (4, 60, 200, 70, 128, True),
    (2, 1, 300, 9000, 128, True), (6, 4, 700, 400, 64, None), (2, 2, 130, 200, 128, None), (70, 1, 130, 140, 64, None),
])
def test_lengths_out_of_range(B, H, Nq, Nk, d, many, masked):
    p, q, k, v, kw = inputs(B, H, H, Nq, Nk, d, mask="mask" if masked else "none")
    assert many is None or uses_tensor_cores(p) == many
    bad, good = lengths(B, Nk)
    out, lse = spark.cross_attn(p, q, k, v, key_len=good, return_lse=True, **kw)
    assert spark.get_status() == 0
    got, got_lse = spark.cross_attn(p, q, k, v, key_len=bad, return_lse=True, **kw)
    assert spark.get_status() == 2
    assert torch.equal(got, out) and torch.equal(got_lse, lse)
    g = torch.Generator(device="cuda").manual_seed(5)
    dout = torch.randn(q.shape, generator=g, device="cuda").to(q.dtype)
    want = spark.cross_attn_bwd(p, q, k, v, out, lse, dout, key_len=good, **kw)
    assert spark.get_status() == 0
    grads = spark.cross_attn_bwd(p, q, k, v, out, lse, dout, key_len=bad, **kw)
    assert spark.get_status() == 2
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    assert spark.get_status() == 0
