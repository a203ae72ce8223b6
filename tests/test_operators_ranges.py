"""Parameters that double holds and the kernels' float32 does not (no GPU needed)."""

import pytest

import block_sparse_attention_spark_b200 as spark
from tests.test_operators_abi import C, INVALID, OK, R, view, FAKE


@pytest.mark.parametrize("scale,code", [(1e39, INVALID), (3e38, INVALID), (1e300, INVALID), (2e38, OK), (1e-3, OK), (1e-300, OK)])
def test_cross_scale_in_float32(scale, code):
    p = C(scale=scale)
    assert spark.cross_validate(p) == code
    assert (spark.cross_workspace_size(p) > 0) == (code == OK) and (spark.cross_workspace_size(p, True) > 0) == (code == OK)
    if code != OK:
        q, k = view(2, 4, 100, 64), view(2, 2, 70, 64)
        assert spark.lib().spark_cross_attn(p, q, k, k, None, None, q, None, FAKE, 1 << 30, None) == code


@pytest.mark.parametrize("eps,code", [(1e39, INVALID), (3e38, OK), (1e-6, OK), (1e-300, OK), (0.0, OK)])
def test_rotary_eps_in_float32(eps, code):
    assert spark.rotary_validate(R(eps=eps)) == code
