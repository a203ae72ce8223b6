"""Rotary positions with several axes, the per-head norm before them and their
gradient, against the formulas in 64 bits."""

import pytest
import torch

import block_sparse_attention_spark_b200 as spark
from tests import operators64 as o64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rand(gen, shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


# B, Hq, Hk, grid, d, dims, dtype, pairing, spectrum, norm of (q, k), positions given
CASES = [
    (1, 1, 0, (1, 1, 1), 64, (16, 24, 24), "bf16", "interleaved", "axis", (False, False), False),
    (1, 2, 2, (4, 16, 64), 64, (16, 24, 24), "bf16", "interleaved", "axis", (True, True), False),
    (2, 3, 1, (3, 5, 7), 128, (44, 42, 42), "bf16", "interleaved", "axis", (True, False), False),
    (1, 5, 5, (2, 9, 11), 128, (16, 56, 56), "fp16", "interleaved", "shared", (False, True), True),
    (2, 7, 3, (1, 13, 17), 128, (32, 32, 32), "fp16", "halves", "shared", (True, True), True),
    (1, 4, 4, (5, 3, 3), 64, (22, 20, 22), "bf16", "halves", "axis", (True, True), False),
    (3, 1, 2, (2, 2, 19), 64, (6, 2, 10), "fp32", "halves", "axis", (True, False), False),
    (1, 6, 2, (2, 7, 9), 128, (44, 42, 42), "fp32", "interleaved", "axis", (True, True), True),
    (1, 9, 9, (2, 8, 8), 128, (0, 64, 64), "bf16", "halves", "axis", (False, False), False),
    (1, 3, 3, (2, 8, 8), 64, (0, 0, 0), "bf16", "halves", "axis", (True, False), False),
    (1, 2, 1, (31, 1, 1), 64, (10, 0, 0), "fp32", "halves", "shared", (False, False), True),
]


def case(c, seed=3, projections=True):
    B, Hq, Hk, grid, d, dims, dtype, pairing, spectrum, norm, given = c
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, N = DT[dtype], grid[0] * grid[1] * grid[2]

    def tensor(H):
        return rand(g, (B, N, H, d), dt, 1.5).transpose(1, 2) if projections else rand(g, (B, H, N, d), dt, 1.5)

    q, k = tensor(Hq), tensor(Hk) if Hk else None
    wq = (1 + rand(g, (d,), dt, 0.3)).to(dt) if norm[0] else None
    wk = (1 + rand(g, (d,), dt, 0.3)).to(dt) if norm[1] and Hk else None
    pos = None
    where = o64.raster(grid, "cuda").unsqueeze(0)
    if given:
        pos = torch.randint(-50, 90000, (B, N, 3), generator=g, device="cuda").float()
        where = pos
    p = spark.rotary_params(B, Hq, N, d, dims, heads_k=Hk, grid=None if given else grid, dtype=dtype, pairing=pairing,
                            spectrum=spectrum, theta=10000.0, eps=1e-6)
    ang = o64.angles(dims, spectrum, 10000.0, where)
    return p, q, k, wq, wk, pos, ang, pairing


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_rotary(c):
    p, q, k, wq, wk, pos, ang, pairing = case(c)
    qo, ko = spark.rotary(p, q, k, positions=pos, q_weight=wq, k_weight=wk)
    assert qo.is_contiguous() and (ko is None) == (k is None)
    o64.check(qo, *o64.rotary(q, wq, ang, pairing, 1e-6), "q")
    if k is not None:
        o64.check(ko, *o64.rotary(k, wk, ang, pairing, 1e-6), "k")


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_rotary_gradient(c):
    p, q, k, wq, wk, pos, ang, pairing = case(c)
    g = torch.Generator(device="cuda").manual_seed(11)
    dqo = rand(g, q.shape, q.dtype)
    dko = None if k is None else rand(g, k.shape, k.dtype)
    dq, dk, dwq, dwk = spark.rotary_bwd(p, dqo, dko, q, k, positions=pos, q_weight=wq, k_weight=wk)
    assert dq.stride() == q.stride()
    for got, dy, x, w, dw in ((dq, dqo, q, wq, dwq),) + (() if k is None else ((dk, dko, k, wk, dwk),)):
        dx, b, dwx, bw = o64.rotary_bwd(dy, x, w, ang, pairing, 1e-6)
        o64.check(got, dx, b, "dx")
        assert (dw is None) == (w is None)
        if w is not None:
            o64.check(dw, dwx, bw, "dw")
    again = spark.rotary_bwd(p, dqo, dko, q, k, positions=pos, q_weight=wq, k_weight=wk)
    for a, b in zip((dq, dk, dwq, dwk), again):
        assert a is None or torch.equal(a, b)


def test_rotary_gradient_against_differences():
    """sum(g * rotary(x)) along a direction, by central differences of the 64-bit form's own 32-bit kernel calls."""
    c = (1, 2, 1, (2, 3, 5), 64, (16, 24, 24), "fp32", "interleaved", "axis", (True, True), False)
    p, q, k, wq, wk, pos, ang, pairing = case(c)
    g = torch.Generator(device="cuda").manual_seed(5)
    dqo, dko = rand(g, q.shape, q.dtype), rand(g, k.shape, k.dtype)
    vq, vk, vw = rand(g, q.shape, q.dtype), rand(g, k.shape, k.dtype), rand(g, (p.d,), q.dtype)

    def value(t):
        qo, ko = spark.rotary(p, q + t * vq, k + t * vk, q_weight=wq + t * vw, k_weight=wk)
        return float((qo.double() * dqo.double()).sum() + (ko.double() * dko.double()).sum())

    dq, dk, dwq, _ = spark.rotary_bwd(p, dqo, dko, q, k, q_weight=wq, k_weight=wk)
    want = float((dq.double() * vq.double()).sum() + (dk.double() * vk.double()).sum()
                 + (dwq.double() * vw.double()).sum())
    h = 2.0 ** -7
    got = (value(h) - value(-h)) / (2 * h)
    # values are sums of 11,520 terms of size ~1 with errors of 32 steps of 2^-24 each (random: sqrt of the count),
    # over 2h; the third derivative's h^2 / 6 adds less than 1e-3 of the norm of the terms
    size = float((dqo.double().square().sum() + dko.double().square().sum()).sqrt())
    assert abs(got - want) <= size * (32 * 2.0 ** -24 / h + 4 * h * h)


def test_rotary_values_past_the_rotated_ones_keep_infinities_to_themselves():
    c = (1, 1, 0, (2, 2, 2), 64, (4, 2, 4), "bf16", "interleaved", "axis", (False, False), False)
    p, q, *_ = case(c)
    q = q.clone()
    q[..., 30] = float("inf")
    qo, _ = spark.rotary(p, q)
    assert torch.isinf(qo[..., 30]).all() and torch.isfinite(qo[..., 31]).all()
    assert torch.equal(qo[..., 10:30], q[..., 10:30])


def test_rotary_in_place_strided_and_shared_rows():
    c = CASES[2]
    p, q, k, wq, wk, pos, ang, pairing = case(c)
    want, wantk = spark.rotary(p, q, k, q_weight=wq)
    q2, k2 = q.clone(), k.clone()
    spark.rotary(p, q2, k2, q_weight=wq, out=(q2, k2))
    assert torch.equal(q2, want) and torch.equal(k2, wantk)
    # the rows of a packed projection, and one item's rows for the whole batch
    B, Hq, Hk, N, d = p.B, p.Hq, p.Hk, p.N, p.d
    packed = torch.empty(B, N, Hq + 2 * Hk, d, dtype=q.dtype, device="cuda")
    packed[:, :, :Hq], packed[:, :, Hq:Hq + Hk] = q.transpose(1, 2), k.transpose(1, 2)
    a, b = spark.rotary(p, packed[:, :, :Hq].transpose(1, 2), packed[:, :, Hq:Hq + Hk].transpose(1, 2), q_weight=wq)
    assert torch.equal(a, want) and torch.equal(b, wantk)
    one = q[:1].expand(B, -1, -1, -1)
    a, _ = spark.rotary(p, one, k, q_weight=wq)
    assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[0])
    assert spark.get_status() == 0


def test_rotary_start_and_scale():
    B, H, grid, d, dims = 1, 2, (3, 4, 5), 64, (16, 24, 24)
    g = torch.Generator(device="cuda").manual_seed(0)
    q = rand(g, (B, H, 60, d), torch.float32)
    start, scale = (100.5, -3.0, 0.25), (0.5, 2.0, 1.0)
    p = spark.rotary_params(B, H, 60, d, dims, heads_k=0, grid=grid, dtype="fp32", start=start, scale=scale)
    qo, _ = spark.rotary(p, q)
    ang = o64.angles(dims, "axis", 10000.0, o64.raster(grid, "cuda").unsqueeze(0), start, scale)
    o64.check(qo, *o64.rotary(q, None, ang, "interleaved", 0.0), "q")


def test_rotary_on_another_stream_and_captured():
    p, q, k, wq, wk, pos, ang, pairing = case(CASES[1])
    want = spark.rotary(p, q, k, q_weight=wq, k_weight=wk)
    dqo, dko = q * 2, k * 3
    grads = spark.rotary_bwd(p, dqo, dko, q, k, q_weight=wq, k_weight=wk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = spark.rotary(p, q, k, q_weight=wq, k_weight=wk)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = spark.rotary(p, q, k, q_weight=wq, k_weight=wk)
        gg = spark.rotary_bwd(p, dqo, dko, q, k, q_weight=wq, k_weight=wk)
    for t in (*got, *gg):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, *gg), (*want, *grads)))
