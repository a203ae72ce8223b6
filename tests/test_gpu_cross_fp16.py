"""fp16 cross attention at the ends of the type's range."""

import math

import pytest
import torch

import block_sparse_attention_spark_b200 as spark
from tests.test_gpu_cross_logits import uses_tensor_cores

pytestmark = pytest.mark.gpu


# few rows: one block a row tile, a cluster, many blocks; many rows: whole keys, keys split over CTAs
@pytest.mark.parametrize("H,Nq,Nk,d,many", [
    (150, 1, 120, 64, False), (4, 3, 700, 128, False), (1, 1, 1 << 20, 64, False), (1, 2, 1 << 22, 64, False),
    (150, 200, 1 << 14, 64, True), (80, 200, 5000, 128, True), (1, 600, 1 << 20, 64, True),
])
def test_many_small_weights_count(H, Nq, Nk, d, many):
    """One key with almost all of the weight, the others at 2^-26.2 of it each: their values count by their number."""
    p = spark.cross_params(1, H, Nq, Nk, d, heads_kv=1, dtype="fp16")
    q = torch.zeros(1, H, Nq, d, dtype=torch.float16, device="cuda")
    k, v = (torch.zeros(1, 1, Nk, d, dtype=torch.float16, device="cuda") for _ in range(2))
    q[..., 0] = 8
    k[:, :, Nk // 3, 0] = 26.2 * math.log(2) * math.sqrt(d) / 8
    v[:] = 1000.0
    v[:, :, Nk // 3] = 0
    assert uses_tensor_cores(p) == many
    out, lse = spark.cross_attn(p, q, k, v, return_lse=True)
    assert spark.get_status() == 0
    logit = 8 * float(k[0, 0, Nk // 3, 0]) / math.sqrt(d)
    share = (Nk - 1) * math.exp(-logit) / (1 + (Nk - 1) * math.exp(-logit))
    # a weight is off by 2^-11 of itself or by half a step of fp16's subnormals, 2^-25, where the largest is 2^9 (few
    # rows: 2^7), the result by half a step (2^-25 among the subnormals); logits, exponentials and sums in 32 bits:
    # 2^-24 of 64 steps of 26.2
    lost = Nk * 2.0 ** (-34 if many else -32)
    bound = 1000 * (share * (2 * 2.0 ** -11 + 64 * 27 * 2.0 ** -24) + lost) + 2.0 ** -25
    assert (out.double() - 1000 * share).abs().max() <= bound
    assert (lse.double() - (logit - math.log1p(-share))).abs().max() <= 64 * 27 * 2.0 ** -24


# the kernels as above; the last key's weight runs from half of the others' to 64 times theirs
@pytest.mark.parametrize("H,Nq,Nk,d,many", [
    (2000, 1, 5, 64, False), (40, 3, 700, 128, False), (1, 16, 40000, 64, False),
    (160, 200, 5, 64, True), (100, 200, 130, 128, True), (1, 600, 20000, 64, True),
])
@pytest.mark.parametrize("sign", [1, -1])
def test_values_at_the_largest_of_the_type(H, Nq, Nk, d, many, sign):
    """A mean of equal values is that value, the type's largest too: rounded weights do not carry it to infinity."""
    p = spark.cross_params(1, H, Nq, Nk, d, heads_kv=1, dtype="fp16")
    assert uses_tensor_cores(p) == many
    n = H * Nq
    q = torch.zeros(1, H, Nq, d, dtype=torch.float16, device="cuda")
    q[..., 0] = torch.linspace(-1, 6, n, device="cuda").view(1, H, Nq)
    k, v = (torch.zeros(1, 1, Nk, d, dtype=torch.float16, device="cuda") for _ in range(2))
    k[:, :, -1, 0] = math.log(2) * math.sqrt(d)
    v[:] = sign * 65504.0
    v[..., 1::2] = 1.0
    out = spark.cross_attn(p, q, k, v)
    assert spark.get_status() == 0
    # weights off by 2^-11 each, and the rounding of the result
    assert out.isfinite().all()
    assert (out[..., ::2].double() - sign * 65504).abs().max() <= 65504 * 2 * 2.0 ** -11
    assert (out[..., 1::2].double() - 1).abs().max() <= 2 * 2.0 ** -11


def test_infinite_values_stay_infinite():
    for H, Nq in ((2, 1), (160, 200)):
        p = spark.cross_params(1, H, Nq, 70, 64, dtype="fp16")
        g = torch.Generator(device="cuda").manual_seed(1)
        q, k, v = (torch.randn(1, H, n, 64, generator=g, device="cuda").half() for n in (Nq, 70, 70))
        v[:, :, 3, 5], v[:, :, 3, 6] = float("inf"), float("-inf")
        out = spark.cross_attn(p, q, k, v)
        assert torch.isposinf(out[..., 5]).all() and torch.isneginf(out[..., 6]).all()
        assert out[..., 7:].isfinite().all()


@pytest.mark.parametrize("H,Nq,Nk,d,many", [
    (3, 1, 120, 64, False), (4, 3, 700, 128, False), (1, 2, 40000, 64, False),
    (160, 200, 300, 64, True), (100, 200, 600, 128, True), (1, 600, 20000, 64, True),
])
@pytest.mark.parametrize("size", [2.0 ** 17, 2.0 ** 21, 2.0 ** 24, 2.0 ** 25.5])
@pytest.mark.parametrize("sign", [1, -1])
def test_logits_of_millions(H, Nq, Nk, d, many, size, sign):
    """Logits so large that float32 counts them in steps of up to 4: the key far above the others takes the row."""
    p = spark.cross_params(1, H, Nq, Nk, d, heads_kv=1, dtype="fp16")
    assert uses_tensor_cores(p) == many
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.zeros(1, H, Nq, d, dtype=torch.float16, device="cuda")
    k = torch.zeros(1, 1, Nk, d, dtype=torch.float16, device="cuda")
    v = torch.randn(1, 1, Nk, d, generator=g, device="cuda").half()
    # logits in powers of two about `size`; rows differ by up to 3%, keys rise by 6% on the way, the last one by 12%
    unit = (size * math.sqrt(d) / 1.4427) ** 0.5
    q[..., 0] = sign * unit * (1 + torch.rand(1, H, Nq, generator=g, device="cuda") / 32)
    rise = torch.arange(Nk, device="cuda") / (16 * Nk)
    rise[-1] = 1 / 8
    k[..., 0] = unit * (1 + rise if sign > 0 else 1 + 1 / 8 - rise)
    top = int((sign * k[0, 0, :, 0].float()).argmax())
    assert top == Nk - 1 and float(k[0, 0, :-1, 0].float().mul(sign).max()) < float(k[0, 0, -1, 0]) * sign
    out, lse = spark.cross_attn(p, q, k, v, return_lse=True)
    assert spark.get_status() == 0
    # every other weight is below 2^-(size / 32); the one that is left is 2^-11 off beside its sum
    want = v[:, :, -1:].double()
    assert ((out.double() - want).abs() <= 2 * 2.0 ** -11 * want.abs() + 2.0 ** -24).all()
    logit = q[..., 0].double() * k[0, 0, -1, 0].double() / math.sqrt(d)
    assert ((lse.double() - logit).abs() <= 4 * 2.0 ** -24 * logit.abs() + 2.0 ** -10).all()
