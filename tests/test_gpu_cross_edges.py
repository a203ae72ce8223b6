"""Cross attention and its gradient where a call is unusual and allowed."""

import pytest
import torch

import block_sparse_attention_spark_b200 as spark
from tests.test_gpu_cross import ids, inputs
from tests.test_gpu_cross_bwd import gradient

pytestmark = pytest.mark.gpu


# few rows joined by a second launch; tensor-core rows with split keys, with a mask; query tiles with split keys
@pytest.mark.parametrize("c", [
    (1, 1, 1, 1, 40000, 128, "bf16", "mask"),
    (1, 4, 4, 256, 5000, 128, "bf16", "mask"),
    (2, 40, 20, 200, 300, 64, "bf16", "lengths"),
    (1, 2, 2, 64, 3000, 128, "bf16", "mask"),
], ids=ids)
def test_workspace_at_any_16_bytes(c):
    """A workspace cut from an arena at 16 bytes past a larger boundary: the same bits, nothing written outside of it."""
    p, q, k, v, kw = inputs(*c)
    dout, out, lse, grads = gradient(p, q, k, v, kw)
    for at in (16, 48, 240):
        for bwd in (False, True):
            n = spark.cross_workspace_size(p, bwd)
            arena = torch.full((at + n + 512,), 77, dtype=torch.uint8, device="cuda")
            ws = arena[at:at + n]
            assert ws.data_ptr() % 256 == at
            if bwd:
                got = spark.cross_attn_bwd(p, q, k, v, out, lse, dout, ws=ws, **kw)
                assert all(torch.equal(a, b) for a, b in zip(got, grads))
            else:
                got, got_lse = spark.cross_attn(p, q, k, v, ws=ws, return_lse=True, **kw)
                assert torch.equal(got, out) and torch.equal(got_lse, lse)
            assert (arena[:at] == 77).all() and (arena[at + n:] == 77).all()
    assert spark.get_status() == 0
