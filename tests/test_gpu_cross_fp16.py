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
    # a weight is off by 2^-11 of itself or by 2^-34 of the largest, the result by half a step (2^-25 among the
    # subnormals); logits, exponentials and sums in 32 bits: 2^-24 of 64 steps of 26.2
    bound = 1000 * (share * (2 * 2.0 ** -11 + 64 * 27 * 2.0 ** -24) + Nk * 2.0 ** -34) + 2.0 ** -25
    assert (out.double() - 1000 * share).abs().max() <= bound
    assert (lse.double() - (logit - math.log1p(-share))).abs().max() <= 64 * 27 * 2.0 ** -24
