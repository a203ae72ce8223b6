"""Cross attention to an encoder's states, against the formulas in 64 bits."""

import pytest
import torch

import block_sparse_attention_spark_b200 as spark
from tests import operators64 as o64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def rand(gen, shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def inputs(B, Hq, Hkv, Nq, Nk, d, dtype="bf16", mask="none", seed=1, q_scale=1.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]
    q = rand(g, (B, Nq, Hq, d), dt, q_scale).transpose(1, 2)
    k = rand(g, (B, Nk, Hkv, d), dt).transpose(1, 2)
    v = rand(g, (B, Nk, Hkv, d), dt).transpose(1, 2)
    kw = {}
    if "lengths" in mask:
        kw["key_len"] = torch.randint(0, Nk + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if "mask" in mask:
        kw["key_mask"] = torch.rand(B, Nk, generator=g, device="cuda") < 0.6
    if mask == "empty":
        kw["key_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        kw["key_len"][0] = min(Nk, 3)
    p = spark.cross_params(B, Hq, Nq, Nk, d, heads_kv=Hkv, dtype=dtype)
    return p, q, k, v, kw


def keep_of(p, kw):
    keep = torch.ones(p.B, p.Nk, dtype=torch.bool, device="cuda")
    if "key_len" in kw:
        keep &= torch.arange(p.Nk, device="cuda") < kw["key_len"].unsqueeze(1)
    if "key_mask" in kw:
        keep &= kw["key_mask"].bool()
    return keep


def spoil(t, keep, value):
    """t with a value in the rows that are not kept."""
    t = t.clone()
    t.masked_fill_(~keep[:, None, :, None], value)
    return t


# B, Hq, Hkv, Nq, Nk, d, dtype, mask
CASES = [
    (1, 1, 1, 1, 1, 64, "bf16", "none"),
    (1, 1, 1, 1, 1, 128, "fp16", "none"),
    (2, 4, 4, 1, 77, 128, "bf16", "lengths"),
    (3, 8, 2, 1, 512, 64, "fp16", "mask"),
    (1, 6, 1, 3, 1000, 128, "bf16", "lengths mask"),
    (4, 16, 16, 1, 512, 128, "bf16", "lengths"),
    (1, 2, 1, 17, 4097, 64, "bf16", "none"),
    (1, 1, 1, 1, 40000, 128, "bf16", "lengths mask"),
    (5, 6, 6, 2, 1500, 64, "bf16", "lengths"),
    (1, 30, 30, 1, 700, 128, "fp16", "mask"),
    (2, 3, 3, 129, 65, 128, "bf16", "mask"),
    (2, 4, 2, 200, 64, 64, "fp16", "none"),
    (1, 5, 5, 255, 127, 128, "fp16", "lengths"),
    (2, 6, 2, 333, 129, 64, "bf16", "lengths mask"),
    (1, 2, 2, 1024, 257, 128, "bf16", "none"),
    (3, 2, 1, 257, 333, 128, "bf16", "empty"),
    (3, 2, 1, 2, 333, 128, "bf16", "empty"),
    (1, 1, 1, 700, 2, 64, "bf16", "none"),
    (1, 4, 4, 256, 5000, 128, "bf16", "mask"),
]
ids = lambda c: "-".join(str(x) for x in c).replace(" ", "_")  # noqa: E731


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_cross_attention(c):
    p, q, k, v, kw = inputs(*c)
    out, lse = spark.cross_attn(p, q, k, v, return_lse=True, **kw)
    assert spark.get_status() == 0
    ref = o64.Cross(q, k, v, **kw)
    bo, bl = ref.forward_bounds()
    o64.check(out, ref.out, bo, "out")
    o64.check(lse, ref.lse, bl, "lse")
    empty = ~keep_of(p, kw).any(1)
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    # what stands in the rows that are not kept is never used
    keep = keep_of(p, kw)
    if not keep.all():
        for value in (float("nan"), float("inf"), torch.finfo(q.dtype).min):
            a, b = spark.cross_attn(p, q, spoil(k, keep, value), spoil(v, keep, value), return_lse=True, **kw)
            assert torch.equal(a, out) and torch.equal(b, lse)


@pytest.mark.parametrize("Nq", [1, 300])
def test_cross_attention_large_logits_and_lowest_values(Nq):
    """Logits of hundreds (one key takes the row), and keys of the type's lowest value: weights exactly 0, no NaN."""
    p, q, k, v, kw = inputs(1, 2, 2, Nq, 300, 128, q_scale=40.0)
    k = k.clone()
    out, lse = spark.cross_attn(p, q, k, v, return_lse=True)
    ref = o64.Cross(q, k, v)
    bo, bl = ref.forward_bounds()
    o64.check(out, ref.out, bo, "out")
    o64.check(lse, ref.lse, bl, "lse")
    q = q.abs()
    k[:, :, 200:] = torch.finfo(torch.bfloat16).min     # logits overflow to -inf
    got = spark.cross_attn(p, q, k, v)
    p2 = spark.cross_params(1, 2, Nq, 200, 128)
    want = o64.Cross(q, k[:, :, :200], v[:, :, :200])
    o64.check(got, want.out, want.forward_bounds()[0], "out")
    assert spark.get_status() == 0 and p2.Nk == 200


@pytest.mark.parametrize("Nq", [1, 2, 130])
def test_cross_attention_scale_layouts_and_rows_left_alone(Nq):
    p, q, k, v, _ = inputs(2, 4, 2, Nq, 99, 64)
    p = spark.cross_params(2, 4, Nq, 99, 64, heads_kv=2, scale=0.3)
    want = spark.cross_attn(p, q, k, v)
    ref = o64.Cross(q, k, v, scale=0.3)
    o64.check(want, ref.out, ref.forward_bounds()[0], "out")
    # out as a slice of a larger buffer, [B, N, H, d]: what is around it stays
    big = torch.full((2, Nq + 3, 6, 64), 7.0, dtype=q.dtype, device="cuda")
    view = big[:, 1:Nq + 1, 1:5].transpose(1, 2)
    spark.cross_attn(p, q, k, v, out=view)
    assert torch.equal(view, want)
    rest = big.clone()
    rest[:, 1:Nq + 1, 1:5] = 7.0
    assert (rest == 7.0).all()
    # k and v packed, [B, Nk, 2, Hkv, d]; one item's states for the batch
    kv = torch.stack([k.transpose(1, 2), v.transpose(1, 2)], 2)
    assert torch.equal(spark.cross_attn(p, q, kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)), want)
    one = spark.cross_attn(p, q, k[:1].expand(2, -1, -1, -1), v[:1].expand(2, -1, -1, -1))
    assert torch.equal(one[0], want[0])
    assert torch.equal(one[1], spark.cross_attn(p, q, k.flip(0).clone(), v.flip(0).clone())[1])


def test_cross_attention_lengths_out_of_range_are_clamped_and_reported():
    for Nq in (1, 200):
        p, q, k, v, _ = inputs(2, 2, 2, Nq, 70, 64)
        bad = torch.tensor([-5, 71], dtype=torch.int32, device="cuda")
        good = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
        got = spark.cross_attn(p, q, k, v, key_len=bad)
        assert spark.get_status() == 2
        assert torch.equal(got, spark.cross_attn(p, q, k, v, key_len=good))
        assert spark.get_status() == 0


@pytest.mark.parametrize("Nq", [1, 300])
def test_cross_attention_on_another_stream_and_in_two_graphs(Nq):
    p, q, k, v, kw = inputs(2, 4, 4, Nq, 300, 128, mask="lengths mask")
    want = spark.cross_attn(p, q, k, v, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = spark.cross_attn(p, q, k, v, **kw)
    s.synchronize()
    assert torch.equal(got, want)
    # two graphs that share one workspace, replayed in turn on one stream
    ws = spark.alloc_cross_workspace(p)
    q2 = (q * 0.5).clone()
    want2 = spark.cross_attn(p, q2, k, v, **kw)
    graphs, outs = [], []
    for x in (q, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(spark.cross_attn(p, x, k, v, ws=ws, **kw))
        graphs.append(g)
    for _ in range(2):
        for o in outs:
            o.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want2)
    assert spark.get_status() == 0


# one block a row tile, a cluster of them, shares joined by a second launch; the same of the tensor-core kernel
@pytest.mark.parametrize("H,Nq,Nk", [(64, 3, 90), (4, 3, 700), (1, 1, 40000), (160, 300, 200), (2, 300, 5000)])
def test_cross_attention_nan_rows_stay_nan_and_alone(H, Nq, Nk):
    """A query row of NaN gives a row of NaN, not zeros, and no other row changes."""
    p, q, k, v, _ = inputs(1, H, H, Nq, Nk, 64)
    out, lse = spark.cross_attn(p, q, k, v, return_lse=True)
    q = q.clone()
    q[:, 0, Nq // 2] = float("nan")
    got, got_lse = spark.cross_attn(p, q, k, v, return_lse=True)
    assert got[:, 0, Nq // 2].isnan().all() and got_lse[:, 0, Nq // 2].isnan().all()
    got[:, 0, Nq // 2], got_lse[:, 0, Nq // 2] = out[:, 0, Nq // 2], lse[:, 0, Nq // 2]
    assert torch.equal(got, out) and torch.equal(got_lse, lse)


def test_cross_attention_mask_of_many_keys():
    """Masks whose packing takes several pieces a block, with an end inside a piece."""
    p, q, k, v, kw = inputs(2, 2, 1, 150, 140001, 64, mask="lengths mask")
    kw["key_len"][0], kw["key_len"][1] = 140001, 130000
    out, lse = spark.cross_attn(p, q, k, v, return_lse=True, **kw)
    assert spark.get_status() == 0
    ref = o64.Cross(q, k, v, **kw)
    bo, bl = ref.forward_bounds()
    o64.check(out, ref.out, bo, "out")
    o64.check(lse, ref.lse, bl, "lse")


# many rows of many heads: the tensor-core kernel (the same lengths at few heads are the few-row kernel's)
MANY = [
    (4, 40, 40, 129, 65, 128, "bf16", "mask"),
    (8, 40, 20, 200, 64, 64, "fp16", "none"),
    (2, 60, 60, 255, 127, 128, "fp16", "lengths"),
    (8, 48, 16, 333, 129, 64, "bf16", "lengths mask"),
    (1, 80, 80, 300, 257, 128, "bf16", "none"),
    (16, 30, 15, 257, 333, 128, "bf16", "empty"),
    (2, 200, 200, 150, 1, 128, "fp16", "none"),
    (3, 150, 150, 200, 2, 64, "bf16", "lengths"),
    (5, 70, 70, 131, 17, 128, "bf16", "mask"),
    (6, 32, 4, 100, 300, 64, "fp16", "mask"),
    (1, 3, 1, 400, 4000, 128, "fp16", "lengths mask"),
    (1, 12, 12, 2000, 640, 64, "bf16", "none"),
]


@pytest.mark.parametrize("c", MANY, ids=ids)
def test_cross_attention_many_rows(c):
    p = spark.cross_params(*c[:2], *c[3:6], heads_kv=c[2], dtype=c[6])
    assert spark.cross_workspace_size(p) >= 4 * c[0] * c[2] * c[4] * c[5]      # room for packed keys
    test_cross_attention(c)


def test_cross_attention_many_rows_lowest_values():
    """Keys of the type's lowest value (logits overflow to -inf), alone and beside others, in the tensor-core kernel."""
    for low in (0, 200):
        p, q, k, v, _ = inputs(1, 120, 120, 300, 300, 128)
        q, k = q.abs(), k.clone()
        k[:, :, low:] = torch.finfo(torch.bfloat16).min
        got, lse = spark.cross_attn(p, q, k, v, return_lse=True)
        assert spark.get_status() == 0
        if low == 0:
            assert (got == 0).all() and torch.isneginf(lse).all()
        else:
            want = o64.Cross(q, k[:, :, :low], v[:, :, :low])
            o64.check(got, want.out, want.forward_bounds()[0], "out")


def test_cross_attention_many_rows_layouts_streams_and_graphs():
    p, q, k, v, kw = inputs(4, 40, 20, 130, 99, 64, mask="lengths mask")
    want = spark.cross_attn(p, q, k, v, **kw)
    big = torch.full((4, 133, 42, 64), 7.0, dtype=q.dtype, device="cuda")
    view = big[:, 1:131, 1:41].transpose(1, 2)
    spark.cross_attn(p, q, k, v, out=view, **kw)
    assert torch.equal(view, want)
    big[:, 1:131, 1:41] = 7.0
    assert (big == 7.0).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = spark.cross_attn(p, q, k, v, **kw)
    s.synchronize()
    assert torch.equal(got, want)
    ws = spark.alloc_cross_workspace(p)
    outs, graphs = [], []
    for x in (q, (q * 0.5).clone()):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((x, spark.cross_attn(p, x, k, v, ws=ws, **kw)))
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for x, o in outs:
        assert torch.equal(o, spark.cross_attn(p, x, k, v, **kw))
    assert spark.get_status() == 0
