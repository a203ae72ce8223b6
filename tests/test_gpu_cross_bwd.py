"""The gradient of cross attention, against the formulas in 64 bits and
against differences of the forward pass."""

import pytest
import torch

import block_sparse_attention_spark_b200 as spark
from tests import operators64 as o64
from tests.test_gpu_cross import ids, inputs, keep_of, rand, spoil

pytestmark = pytest.mark.gpu

# B, Hq, Hkv, Nq, Nk, d, dtype, mask
CASES = [
    (1, 1, 1, 1, 1, 64, "bf16", "none"),
    (1, 2, 2, 1, 77, 128, "bf16", "none"),
    (2, 2, 1, 128, 128, 128, "bf16", "none"),
    (1, 1, 1, 300, 40, 64, "bf16", "none"),
    (2, 4, 2, 129, 129, 128, "bf16", "lengths"),
    (3, 6, 2, 777, 99, 64, "bf16", "mask"),
    (1, 3, 3, 500, 257, 128, "bf16", "lengths mask"),
    (3, 2, 1, 257, 333, 128, "bf16", "empty"),
    (1, 2, 2, 64, 3000, 128, "bf16", "mask"),
    (2, 5, 5, 2000, 260, 64, "bf16", "none"),
    (5, 10, 5, 900, 250, 128, "bf16", "lengths"),
    (4, 10, 2, 900, 200, 64, "bf16", "lengths mask"),
    (1, 40, 40, 1500, 200, 128, "bf16", "none"),
    (1, 40, 20, 1000, 100, 64, "bf16", "none"),
    (1, 8, 2, 5000, 512, 128, "bf16", "none"),
]


def gradient(p, q, k, v, kw, seed=9):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dout = rand(g, q.shape, q.dtype)
    out, lse = spark.cross_attn(p, q, k, v, return_lse=True, **kw)
    return dout, out, lse, spark.cross_attn_bwd(p, q, k, v, out, lse, dout, **kw)


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_cross_gradient(c):
    p, q, k, v, kw = inputs(*c)
    dout, out, lse, grads = gradient(p, q, k, v, kw)
    assert spark.get_status() == 0
    ref = o64.Cross(q, k, v, **kw)
    wants, bounds = ref.backward(dout)
    for got, like, want, bound, name in zip(grads, (q, k, v), wants, bounds, ("dq", "dk", "dv")):
        assert got.shape == like.shape and got.stride() == like.stride()
        o64.check(got, want, bound, name)
    # equal calls, equal bits; what stands in the dropped rows is never used
    keep = keep_of(p, kw)
    for value in (None,) if keep.all() else (float("nan"), float("inf"), torch.finfo(q.dtype).min):
        k2, v2 = (k, v) if value is None else (spoil(k, keep, value), spoil(v, keep, value))
        again = spark.cross_attn_bwd(p, q, k2, v2, out, lse, dout, **kw)
        assert all(torch.equal(a, b) for a, b in zip(again, grads))
    dropped = ~keep[:, None, :, None].expand_as(grads[1])
    assert (grads[1][dropped] == 0).all() and (grads[2][dropped] == 0).all()


def test_cross_gradient_against_differences():
    p, q, k, v, kw = inputs(1, 4, 2, 200, 150, 64, mask="mask")
    dout, out, lse, (dq, dk, dv) = gradient(p, q, k, v, kw)
    g = torch.Generator(device="cuda").manual_seed(3)
    vq, vk, vv = (torch.randn(t.shape, generator=g, device="cuda").double() for t in (q, k, v))

    def value(t):
        c = o64.Cross(q.double() + t * vq, k.double() + t * vk, v.double() + t * vv, **kw)
        return float((c.out * dout.double()).sum())

    want = (value(1e-4) - value(-1e-4)) / 2e-4          # 64 bits: good to 1e-6 of the value
    got = float((dq.double() * vq).sum() + (dk.double() * vk).sum() + (dv.double() * vv).sum())
    wants, bounds = o64.Cross(q, k, v, **kw).backward(dout)
    bound = sum(float((b.expand_as(x) * d.abs()).sum()) for b, x, d in zip(bounds, wants, (vq, vk, vv)))
    assert abs(got - want) <= bound + 1e-5 * abs(want)


def test_cross_gradient_scale_layouts_and_shared_rows():
    _, q, k, v, _ = inputs(2, 4, 2, 130, 99, 64)
    p = spark.cross_params(2, 4, 130, 99, 64, heads_kv=2, scale=0.3)
    dout, out, lse, grads = gradient(p, q, k, v, {})
    wants, bounds = o64.Cross(q, k, v, scale=0.3).backward(dout)
    for got, want, bound, name in zip(grads, wants, bounds, ("dq", "dk", "dv")):
        o64.check(got, want, bound, name)
    # contiguous inputs, the same values: the same gradients
    again = spark.cross_attn_bwd(p, q.contiguous(), k.contiguous(), v.contiguous(), out.transpose(1, 2).contiguous().transpose(1, 2),
                                 lse, dout.transpose(1, 2).contiguous().transpose(1, 2))
    assert all(torch.equal(a, b) for a, b in zip(again, grads))
    # one item's states read by the whole batch (stride 0): each item's own gradient comes back
    one = (k[:1].expand(2, -1, -1, -1), v[:1].expand(2, -1, -1, -1))
    dout, out, lse, shared = gradient(p, q, *one, {})
    full = spark.cross_attn_bwd(p, q, one[0].contiguous(), one[1].contiguous(), out, lse, dout)
    assert all(torch.equal(a, b) for a, b in zip(shared, full))


def test_cross_gradient_captured_beside_an_eager_call():
    p, q, k, v, kw = inputs(2, 4, 4, 300, 300, 128, mask="lengths mask")
    dout, out, lse, want = gradient(p, q, k, v, kw)
    ws = spark.alloc_cross_workspace(p, bwd=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = spark.cross_attn_bwd(p, q, k, v, out, lse, dout, ws=ws, **kw)
    eager = spark.cross_attn_bwd(p, q, k, v, out, lse, dout, ws=ws, **kw)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, eager))
    # another stream at the same time, its own workspace
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = spark.cross_attn_bwd(p, q, k, v, out, lse, dout, **kw)
    here = spark.cross_attn_bwd(p, q, k, v, out, lse, dout, ws=ws, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, other, here))
    assert spark.get_status() == 0


# lengths of many items and many tiles: key tiles and query tiles are shared out on the device
@pytest.mark.parametrize("c", [
    (40, 4, 2, 130, 300, 64, "bf16", "lengths mask"),
    (70, 2, 2, 200, 130, 128, "bf16", "lengths"),
    (3, 20, 20, 500, 300, 128, "bf16", "empty"),
    (2, 16, 16, 700, 600, 128, "bf16", "lengths"),
    (2, 12, 4, 1200, 700, 64, "bf16", "mask"),
    (3, 4, 1, 40, 9000, 64, "bf16", "lengths"),
], ids=ids)
def test_cross_gradient_shared_out(c):
    test_cross_gradient(c)


@pytest.mark.parametrize("lengths", [(0, 0, 0, 0), (0, 600, 0, 3), (256, 1, 128, 129), (600, 600, 600, 600)])
def test_cross_gradient_of_given_lengths(lengths):
    p, q, k, v, _ = inputs(4, 16, 8, 700, 600, 64)
    kw = {"key_len": torch.tensor(lengths, dtype=torch.int32, device="cuda")}
    dout, out, lse, grads = gradient(p, q, k, v, kw)
    assert spark.get_status() == 0
    wants, bounds = o64.Cross(q, k, v, **kw).backward(dout)
    for got, want, bound, name in zip(grads, wants, bounds, ("dq", "dk", "dv")):
        o64.check(got, want, bound, name)
    for b, n in enumerate(lengths):
        assert (grads[1][b, :, n:] == 0).all() and (grads[2][b, :, n:] == 0).all()
        if n == 0:
            assert (grads[0][b] == 0).all()


def test_cross_attention_and_gradient_in_a_forked_capture():
    """Two branches of one captured graph, each with a workspace of its own, behind copies and joined again."""
    p, q, k, v, kw = inputs(2, 20, 20, 300, 200, 64, mask="lengths mask")
    g = torch.Generator(device="cuda").manual_seed(2)
    dout = rand(g, q.shape, q.dtype)
    want, lse = spark.cross_attn(p, q, k, v, return_lse=True, **kw)
    grads = spark.cross_attn_bwd(p, q, k, v, want, lse, dout, **kw)
    plain = spark.cross_attn(p, q, k, v)
    x, other = torch.zeros_like(q), torch.cuda.Stream()
    ws = [spark.alloc_cross_workspace(p, bwd=b) for b in (False, False, True)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(q)
        main = torch.cuda.current_stream()
        other.wait_stream(main)
        with torch.cuda.stream(other):
            a = spark.cross_attn(p, x, k, v, ws=ws[0])
        b, l = spark.cross_attn(p, x, k, v, ws=ws[1], return_lse=True, **kw)
        main.wait_stream(other)
        c = spark.cross_attn_bwd(p, x, k, v, b, l, dout, ws=ws[2], **kw)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, plain) and torch.equal(b, want) and torch.equal(l, lse)
    assert all(torch.equal(s, t) for s, t in zip(c, grads))
    assert spark.get_status() == 0
