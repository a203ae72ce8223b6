"""The longest calls, and calls at the same time as the rest of the library's."""

import pytest
import torch

import block_sparse_attention_spark_b200 as spark
from tests.test_gpu_cross import inputs
from tests.test_gpu_cross_bwd import gradient

pytestmark = pytest.mark.gpu

LONGEST = 1 << 22


def rows(t, a, b):
    return None if t is None else t[:, :, a:b]


def test_cross_attention_of_the_longest_queries():
    """4 M query tokens: each row as in a call on part of them, bit for bit; dk and dv the sum of the parts'."""
    p, q, k, v, kw = inputs(1, 1, 1, LONGEST, 77, 64)
    dout, out, lse, (dq, dk, dv) = gradient(p, q, k, v, kw)
    n = LONGEST // 4
    part = spark.cross_params(1, 1, n, 77, 64)
    sums = [torch.zeros_like(dk, dtype=torch.float64) for _ in range(2)]
    sizes = [torch.zeros_like(dk, dtype=torch.float64) for _ in range(2)]
    for a in range(0, LONGEST, n):
        got, got_lse = spark.cross_attn(part, rows(q, a, a + n), k, v, return_lse=True)
        assert torch.equal(got, rows(out, a, a + n)) and torch.equal(got_lse, rows(lse, a, a + n))
        got = spark.cross_attn_bwd(part, rows(q, a, a + n), k, v, rows(out, a, a + n), lse[:, :, a:a + n].contiguous(),
                                   rows(dout, a, a + n))
        assert torch.equal(got[0], rows(dq, a, a + n))
        for s, z, t in zip(sums, sizes, got[1:]):
            s += t.double()
            z += t.double().abs()
    for got, s, z in zip((dk, dv), sums, sizes):
        # each part and the whole rounded to bf16 by half a step; 32-bit sums of the same terms in other groups
        terms = 2.0 ** -24 * 2 ** 11 * (2 * LONGEST) ** 0.5
        assert ((got.double() - s).abs() <= 2.0 ** -8 * (z + s.abs()) + terms).all()
    assert spark.get_status() == 0


def test_rotary_of_the_longest_sequence():
    g = torch.Generator(device="cuda").manual_seed(6)
    q, dy = (torch.randn(1, 2, LONGEST, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = (1 + 0.2 * torch.randn(64, generator=g, device="cuda")).to(torch.bfloat16)
    t = torch.arange(LONGEST, device="cuda")
    pos = torch.stack([t // 16384, t // 128 % 128, t % 128], -1).float().unsqueeze(0)
    dims = (16, 24, 24)
    p = spark.rotary_params(1, 2, LONGEST, 64, dims, heads_k=0, grid=(256, 128, 128))
    out, _ = spark.rotary(p, q, q_weight=w)
    dq, _, dw, _ = spark.rotary_bwd(p, dy, None, q, q_weight=w)
    assert torch.equal(out, spark.rotary(p, q, positions=pos, q_weight=w)[0])
    n = LONGEST // 4
    part = spark.rotary_params(1, 2, n, 64, dims, heads_k=0)
    sums = torch.zeros(64, dtype=torch.float64, device="cuda")
    for a in range(0, LONGEST, n):
        at = pos[:, a:a + n].contiguous()
        assert torch.equal(spark.rotary(part, rows(q, a, a + n), positions=at, q_weight=w)[0], rows(out, a, a + n))
        got = spark.rotary_bwd(part, rows(dy, a, a + n), None, rows(q, a, a + n), positions=at, q_weight=w)
        assert torch.equal(got[0], rows(dq, a, a + n))
        sums += got[2].double()
    # 8 M terms of size about 1; a thread adds 2 * 4 M / (888 * 32) = 296 of them in 32 bits
    assert (dw.double() - sums).abs().max() <= 2 * 296 * 2.0 ** -24 * (2 * LONGEST) ** 0.5 * 4 + 2.0 ** -20


def test_with_the_block_sparse_pass_on_another_stream():
    """The pass and the operators at the same time, each with its own workspace: the results of each alone."""
    B, H, N, d = 1, 4, 8192, 128
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = (torch.randn(B, H, N, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    p = spark.params(B, H, N, d, topk_ratio=0.3)
    ws = spark.alloc_workspace(p)
    want = spark.forward(p, q, k, v, ws)
    c, cq, ck, cv, kw = inputs(2, 20, 10, 3000, 300, 64, mask="lengths mask")
    dout, out, lse, grads = gradient(c, cq, ck, cv, kw)
    few = inputs(1, 16, 16, 1, 4000, 128, dtype="fp16")
    few_out = spark.cross_attn(*few[:4])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[], [], []]
    for _ in range(3):
        with torch.cuda.stream(streams[0]):
            got[0].append(spark.forward(p, q, k, v, ws))
        with torch.cuda.stream(streams[1]):
            got[1].append((spark.cross_attn(c, cq, ck, cv, **kw), *spark.cross_attn_bwd(c, cq, ck, cv, out, lse, dout, **kw)))
        with torch.cuda.stream(streams[2]):
            got[2].append(spark.cross_attn(*few[:4]))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got[0])
    assert all(torch.equal(a, b) for ts in got[1] for a, b in zip(ts, (out, *grads)))
    assert all(torch.equal(t, few_out) for t in got[2])
    assert spark.get_status() == 0
