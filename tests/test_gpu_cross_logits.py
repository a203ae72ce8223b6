"""Cross attention and its gradient with large logits: references that move from
key tile to key tile, keys that take a whole row, leading keys without weight."""

import pytest
import torch

import block_sparse_attention_spark_b200 as spark
from tests import operators64 as o64
from tests.test_gpu_cross import ids, inputs
from tests.test_gpu_cross_bwd import gradient

pytestmark = pytest.mark.gpu

# B, Hq, Hkv, Nq, Nk, d, dtype, mask: tensor-core kernel, whole keys and keys split over CTAs
MANY = [
    (1, 120, 120, 300, 600, 64, "bf16", "none"),
    (1, 120, 120, 300, 600, 128, "bf16", "none"),
    (2, 60, 30, 300, 555, 64, "fp16", "none"),
    (2, 60, 30, 300, 555, 128, "fp16", "mask"),
    (2, 60, 60, 260, 700, 128, "bf16", "lengths"),
    (1, 3, 1, 400, 4000, 128, "fp16", "none"),
    (1, 2, 2, 300, 5000, 64, "bf16", "none"),
]
FEW = [
    (2, 4, 2, 3, 900, 64, "fp16", "mask"),
    (1, 8, 8, 1, 5000, 128, "bf16", "none"),
    (1, 1, 1, 2, 40000, 64, "bf16", "none"),
    (2, 4, 2, 40, 300, 128, "fp16", "lengths"),
]


def uses_tensor_cores(p):
    """Its workspace has room for packed keys."""
    return spark.cross_workspace_size(p) >= 4 * p.B * p.Hkv * p.Nk * p.d


def along(q, k, step):
    """q and k with a common direction added: logits grow by `step` (in units of log 2) every 128 keys."""
    d = q.shape[-1]
    u = torch.zeros(d, device="cuda")
    u[::2] = (2.0 / d) ** 0.5
    size = 8.0
    grow = torch.arange(k.shape[2], device="cuda").float() * (step * 0.6931 / 128)
    k2 = k.float() + (grow * d ** 0.5 / size)[:, None] * u
    return (0.5 * q.float() + size * u).to(q.dtype), k2.to(k.dtype)


def compare(p, q, k, v, kw):
    out, lse = spark.cross_attn(p, q, k, v, return_lse=True, **kw)
    assert spark.get_status() == 0
    ref = o64.Cross(q, k, v, **kw)
    bo, bl = ref.forward_bounds()
    o64.check(out, ref.out, bo, "out")
    o64.check(lse, ref.lse, bl, "lse")
    return ref


# a step of 5 moves a reference every other tile or so, of 12 at each, of -12 never
@pytest.mark.parametrize("step", [5.0, 12.0, -12.0])
@pytest.mark.parametrize("c", MANY + FEW, ids=ids)
def test_logits_that_grow_from_tile_to_tile(c, step):
    p, q, k, v, kw = inputs(*c)
    assert uses_tensor_cores(p) == (c in MANY)
    if step * c[4] > 128 * 60:                      # a rise of 60 in all: further keys add nothing but overflow
        step = 128 * 60 / c[4]
    q, k = along(q, k, step)
    compare(p, q, k, v, kw)


@pytest.mark.parametrize("c", MANY + FEW, ids=ids)
def test_logits_of_hundreds(c):
    p, q, k, v, kw = inputs(*c, q_scale=25.0)
    compare(p, q, k, v, kw)


@pytest.mark.parametrize("c", MANY[:2] + MANY[-1:] + FEW[1:3], ids=ids)
@pytest.mark.parametrize("low", [100, 128, 300])
def test_leading_keys_without_weight(c, low):
    """The first keys' logits overflow to -inf, whole tiles of them, before finite ones."""
    p, q, k, v, _ = inputs(*c)
    q, k = q.abs(), k.clone()
    k[:, :, :low] = torch.finfo(q.dtype).min
    out, lse = spark.cross_attn(p, q, k, v, return_lse=True)
    assert spark.get_status() == 0
    ref = o64.Cross(q, k[:, :, low:], v[:, :, low:])
    bo, bl = ref.forward_bounds()
    o64.check(out, ref.out, bo, "out")
    o64.check(lse, ref.lse, bl, "lse")


GRADIENTS = [
    (1, 12, 12, 300, 600, 64, "bf16", "none"),
    (1, 12, 6, 300, 500, 128, "bf16", "mask"),
    (2, 20, 20, 260, 700, 128, "bf16", "lengths"),
    (3, 6, 2, 700, 99, 64, "bf16", "none"),
]


@pytest.mark.parametrize("kind", ["grow", "hundreds"])
@pytest.mark.parametrize("c", GRADIENTS, ids=ids)
def test_gradient_of_large_logits(c, kind):
    p, q, k, v, kw = inputs(*c, q_scale=1.3 if kind == "grow" else 25.0)
    if kind == "grow":
        q, k = along(q, k, 12.0)
    dout, out, lse, grads = gradient(p, q, k, v, kw)
    assert spark.get_status() == 0
    wants, bounds = o64.Cross(q, k, v, **kw).backward(dout)
    for got, want, bound, name in zip(grads, wants, bounds, ("dq", "dk", "dv")):
        o64.check(got, want, bound, name)


@pytest.mark.parametrize("c", GRADIENTS[:1] + GRADIENTS[3:], ids=ids)
@pytest.mark.parametrize("low", [70, 128])
def test_gradient_of_keys_without_weight(c, low):
    """Keys whose logits are -inf get zeros; where there are no others, everything is zero."""
    p, q, k, v, kw = inputs(*c)
    q, k = q.abs(), k.clone()
    k[:, :, :low] = torch.finfo(q.dtype).min
    dout, out, lse, (dq, dk, dv) = gradient(p, q, k, v, kw)
    assert spark.get_status() == 0
    assert (dk[:, :, :low] == 0).all() and (dv[:, :, :low] == 0).all()
    if low >= p.Nk:
        assert torch.isneginf(lse).all() and (dq == 0).all()
        return
    wants, bounds = o64.Cross(q, k[:, :, low:], v[:, :, low:]).backward(dout)
    for got, want, bound, name in zip((dq, dk[:, :, low:], dv[:, :, low:]), wants, bounds, ("dq", "dk", "dv")):
        o64.check(got, want, bound, name)
