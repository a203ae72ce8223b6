"""Host-side checks of the rotary and cross attention entry points: what they
refuse, before anything is launched (no GPU needed, no call gets that far)."""

import ctypes

import pytest

import block_sparse_attention_spark_b200 as spark

FAKE = 1 << 20                                   # never dereferenced
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def R(**kw):
    base = dict(B=2, H=4, N=60, d=64, dims=(16, 24, 24), heads_k=2, grid=(3, 4, 5))
    base.update(kw)
    return spark.rotary_params(**base)


def C(**kw):
    base = dict(B=2, H=4, Nq=100, Nk=70, d=64, heads_kv=2)
    base.update(kw)
    return spark.cross_params(**base)


def view(B, H, N, d, data=FAKE, **kw):
    v = spark.View(data, H * N * d, N * d, d)
    for n, x in kw.items():
        setattr(v, n, x)
    return v


def test_struct_layouts():
    assert ctypes.sizeof(spark.RotaryParams) == 128 and spark.RotaryParams.theta.offset == 64
    assert ctypes.sizeof(spark.CrossParams) == 40 and spark.CrossParams.scale.offset == 32
    assert ctypes.sizeof(spark.View) == 32


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(heads_k=-1), INVALID), (dict(heads_k=0), OK),
    (dict(N=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(dims=(16, 24, 26)), INVALID),
    (dict(dims=(15, 24, 24)), INVALID), (dict(dims=(-2, 24, 24)), INVALID), (dict(dims=(0, 0, 0)), OK),
    (dict(theta=0.0), INVALID), (dict(theta=float("nan")), INVALID), (dict(eps=-1e-6), INVALID),
    (dict(scale=(1.0, float("inf"), 1.0)), INVALID), (dict(B=40000), UNSUPPORTED), (dict(N=(1 << 22) + 1), UNSUPPORTED),
])
def test_rotary_validate(kw, code):
    p = R(**kw)
    assert spark.rotary_validate(p) == code
    assert (spark.rotary_workspace_size(p) > 0) == (code == OK)


def test_rotary_bad_enums():
    for field, value in (("dtype", 3), ("pairing", 2), ("spectrum", -1), ("axes", 0), ("axes", 4)):
        p = R()
        setattr(p, field, value)
        assert spark.rotary_validate(p) == INVALID
    with pytest.raises(ValueError):
        spark.rotary_params(1, 1, 8, 64, (2, 2, 2, 2))
    with pytest.raises(ValueError):
        spark.rotary_params(1, 1, 8, 64, (2, 2), grid=(8,))


def test_rotary_refuses_without_launching():
    L, p = spark.lib(), R()
    q, k = view(2, 4, 60, 64), view(2, 2, 60, 64)

    def call(p=p, q=q, k=k, pos=None, wq=None, wk=None, qo=q, ko=k):
        return L.spark_rotary(p, q, k, pos, wq, wk, qo, ko, None)

    assert call(q=None) == INVALID and call(k=None) == INVALID and call(qo=None) == INVALID and call(ko=None) == INVALID
    assert call(q=view(2, 4, 60, 64, data=FAKE + 2)) == INVALID             # misaligned base
    assert call(q=view(2, 4, 60, 64, n=65)) == INVALID                      # token stride not a multiple of 16 bytes
    assert call(q=view(2, 4, 60, 64, n=32)) == INVALID                      # tokens that overlap
    assert call(q=view(2, 4, 60, 64, b=-64)) == INVALID
    assert call(qo=view(2, 4, 60, 64, b=0)) == INVALID                      # a written view that overlaps itself
    assert call(qo=view(2, 4, 60, 64, h=64)) == INVALID
    assert call(wq=FAKE + 8) == INVALID and call(pos=FAKE + 2) == INVALID
    assert call(p=R(grid=(3, 4, 6))) == INVALID and call(p=R(grid=None)) == INVALID     # no positions, no grid of N tokens
    assert call(p=R(dtype="fp32"), q=view(2, 4, 60, 64, n=66)) == INVALID


def test_rotary_gradient_refuses_without_launching():
    L, p = spark.lib(), R()
    q, k, n = view(2, 4, 60, 64), view(2, 2, 60, 64), spark.rotary_workspace_size(R())

    def call(p=p, gq=q, gk=k, q=q, k=k, wq=FAKE, wk=FAKE, dq=q, dk=k, dwq=FAKE, dwk=FAKE, ws=FAKE, size=n):
        return L.spark_rotary_bwd(p, gq, gk, q, k, None, wq, wk, dq, dk, dwq, dwk, ws, size, None)

    assert call(gq=None) == INVALID and call(gk=None) == INVALID and call(dq=None) == INVALID
    assert call(q=None) == INVALID and call(k=None) == INVALID              # a weight needs its rows
    assert call(dwq=None) == INVALID and call(dwk=None) == INVALID
    assert call(ws=None) == INVALID and call(ws=FAKE + 4) == INVALID and call(size=n - 1) == WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(B=0), INVALID), (dict(Nq=0), INVALID), (dict(Nk=0), INVALID), (dict(heads_kv=3), INVALID),
    (dict(heads_kv=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(dtype="fp32"), UNSUPPORTED), (dict(dtype="fp16"), OK),
    (dict(Nq=(1 << 22) + 1), UNSUPPORTED), (dict(B=20000), UNSUPPORTED), (dict(H=64, heads_kv=64, Nq=1 << 22, B=16), UNSUPPORTED),
    (dict(Nk=1 << 22), OK), (dict(Nq=1), OK),
])
def test_cross_validate(kw, code):
    p = C(**kw)
    assert spark.cross_validate(p) == code
    assert (spark.cross_workspace_size(p) > 0) == (code == OK)
    assert (spark.cross_workspace_size(p, True) > 0) == (code == OK and kw.get("dtype") != "fp16")


def test_cross_scale():
    p = C()
    for x in (-1.0, float("nan"), float("inf")):
        p.scale = x
        assert spark.cross_validate(p) == INVALID
    with pytest.raises(ValueError):
        C(scale=0.0)


def test_cross_refuses_without_launching():
    L = spark.lib()
    for Nq in (1, 100):
        p = C(Nq=Nq)
        q, k, n = view(2, 4, Nq, 64), view(2, 2, 70, 64), spark.cross_workspace_size(p)

        def call(p=p, q=q, k=k, v=k, kl=None, out=q, lse=None, ws=FAKE, size=n):
            return L.spark_cross_attn(p, q, k, v, kl, None, out, lse, ws, size, None)

        for name in ("q", "k", "v", "out"):
            assert call(**{name: None}) == INVALID
        assert call(k=view(2, 2, 70, 64, data=FAKE + 8)) == INVALID and call(k=view(2, 2, 70, 64, n=68)) == INVALID
        assert call(v=view(2, 2, 70, 64, n=0)) == INVALID
        assert call(out=view(2, 4, Nq, 64, h=0)) == INVALID
        assert call(kl=FAKE + 1) == INVALID and call(lse=FAKE + 2) == INVALID
        assert call(ws=None) == INVALID and call(size=n - 1) == WORKSPACE
        bad = C(Nq=Nq, dtype="fp32")
        assert call(p=bad) == UNSUPPORTED


def test_cross_gradient_refuses_without_launching():
    L, p = spark.lib(), C()
    q, k, n = view(2, 4, 100, 64), view(2, 2, 70, 64), spark.cross_workspace_size(C(), True)

    def call(p=p, q=q, k=k, v=k, out=q, lse=FAKE, dout=q, dq=q, dk=k, dv=k, ws=FAKE, size=n):
        return L.spark_cross_attn_bwd(p, q, k, v, out, lse, dout, None, None, dq, dk, dv, ws, size, None)

    for name in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "ws"):
        assert call(**{name: None}) == INVALID, name
    assert call(dk=view(2, 2, 70, 64, b=0)) == INVALID and call(size=n - 1) == WORKSPACE
    assert call(p=C(dtype="fp16")) == UNSUPPORTED


def test_forward_rotary_refuses_without_launching():
    L = spark.lib()
    p = spark.params(1, 2, 4096, 64)
    r = spark.rotary_params(1, 2, 4096, 64, (16, 24, 24), grid=(4, 16, 64))
    n = spark.forward_rotary_workspace_size(p)
    assert n >= spark.workspace_size(p) + 3 * 2 * 4096 * 64 * 2
    x = view(1, 2, 4096, 64)

    def call(p=p, r=r, q=x, v=x, out=FAKE, ws=FAKE, size=n):
        return L.spark_forward_rotary(p, r, q, x, v, None, None, None, out, None, ws, size, None)

    assert call(q=None) == INVALID and call(v=None) == INVALID and call(out=None) == INVALID
    assert call(ws=None) == INVALID and call(size=n - 1) == WORKSPACE
    assert call(p=spark.params(1, 2, 4100, 64)) == UNSUPPORTED
    for kw in (dict(heads_k=1), dict(dtype="fp16"), dict(grid=(4, 16, 63))):
        args = dict(B=1, H=2, N=4096, d=64, dims=(16, 24, 24), grid=(4, 16, 64))
        args.update(kw)
        assert call(r=spark.rotary_params(**args)) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch

    p, r = C(), R()
    q = torch.zeros(2, 4, 100, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        spark.cross_attn(p, q, q, q)
    with pytest.raises(TypeError):
        spark.rotary(r, torch.zeros(2, 4, 60, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        spark.rotary(r, None)
