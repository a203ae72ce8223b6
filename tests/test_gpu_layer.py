"""The operators together, as a layer uses them: projections -> norm, rotary
positions -> block-sparse attention -> cross attention to the encoder, and the
gradient of the conditioning path."""

import pytest
import torch

import block_sparse_attention_spark_b200 as spark
from tests import operators64 as o64

pytestmark = pytest.mark.gpu


def rand(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).bfloat16()


@pytest.mark.parametrize("B,H,grid,d,dims,contiguous_v", [
    (1, 2, (4, 16, 64), 64, (16, 24, 24), False),
    (2, 3, (2, 8, 16), 128, (44, 42, 42), True),
    (2, 3, (2, 8, 16), 128, (44, 42, 42), False),
])
def test_layer(B, H, grid, d, dims, contiguous_v):
    g = torch.Generator(device="cuda").manual_seed(4)
    N, C = grid[0] * grid[1] * grid[2], 77
    x = rand(g, B, N, 3, H, d)                                   # the packed projection
    q, k, v = (x[:, :, i].transpose(1, 2) for i in range(3))
    if contiguous_v:
        v = v.contiguous()
    wq, wk = (1 + rand(g, d, scale=0.1).float()).bfloat16(), (1 + rand(g, d, scale=0.1).float()).bfloat16()
    p = spark.params(B, H, N, d, topk_ratio=0.3)
    r = spark.rotary_params(B, H, N, d, dims, grid=grid)
    out = spark.forward_rotary(p, r, q, k, v, q_weight=wq, k_weight=wk)
    qo, ko = spark.rotary(r, q, k, q_weight=wq, k_weight=wk)
    want = spark.forward(p, qo, ko, v.contiguous())
    assert torch.equal(out, want)
    # the second attention of the layer, over a padded prompt, written in the projection's layout
    c = spark.cross_params(B, H, N, C, d)
    kc, vc = (rand(g, B, C, H, d).transpose(1, 2) for _ in range(2))
    lens = torch.tensor([C, 20][:B], dtype=torch.int32, device="cuda")
    y = torch.empty(B, N, H, d, dtype=torch.bfloat16, device="cuda")
    res, lse = spark.cross_attn(c, out, kc, vc, key_len=lens, return_lse=True, out=y.transpose(1, 2))
    assert res.data_ptr() == y.data_ptr()
    ref = o64.Cross(out, kc, vc, key_len=lens)
    o64.check(res, ref.out, ref.forward_bounds()[0], "cross")
    dout = rand(g, B, N, H, d).transpose(1, 2)
    grads = spark.cross_attn_bwd(c, out, kc, vc, res, lse, dout, key_len=lens)
    wants, bounds = ref.backward(dout)
    for got, w, b, name in zip(grads, wants, bounds, ("dq", "dk", "dv")):
        o64.check(got, w, b, name)
    assert spark.get_status() == 0


def test_layer_with_positions_and_lse():
    g = torch.Generator(device="cuda").manual_seed(8)
    B, H, N, d = 1, 2, 512, 64
    q, k, v = (rand(g, B, N, H, d).transpose(1, 2) for _ in range(3))
    pos = torch.randint(0, 500, (B, N, 2), generator=g, device="cuda").float()
    p = spark.params(B, H, N, d, topk_blocks=3)
    r = spark.rotary_params(B, H, N, d, (32, 32), pairing="halves", spectrum="shared")
    lse = torch.empty(B, H, N, dtype=torch.float32, device="cuda")
    out = spark.forward_rotary(p, r, q, k, v, positions=pos, lse=lse)
    qo, ko = spark.rotary(r, q, k, positions=pos)
    want_lse = torch.empty_like(lse)
    want = spark.forward(p, qo, ko, v.contiguous(), lse=want_lse)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert spark.get_status() == 0
