"""Cases for the operators around the block-sparse attention of a video transformer layer:
rotary positions with several axes (with the per-head RMS norm before it) and cross attention to
an encoder's states, each with its gradient. Used to time them and to compare their outputs."""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


def _rotary(name, op, B, Hq, Hk, grid, d, dims, dtype, pairing, spectrum, norm, given):
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hk": Hk, "F": grid[0], "Hl": grid[1], "Wl": grid[2], "d": d,
            "dt": dims[0], "dh": dims[1], "dw": dims[2], "dtype": dtype, "pairing": pairing, "spectrum": spectrum,
            "norm": norm, "given": given}


def _cross(name, op, B, Hq, Hkv, Nq, Nk, d, dtype, mask):
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "d": d, "dtype": dtype, "mask": mask}


def listed():
    return [
        # the tiny workload's grid at its two heads: latency
        _rotary("rotary_tiny", "rotary", 1, 2, 2, (4, 16, 64), 64, (16, 24, 24), "bf16", "interleaved", "axis", False, False),
        # one layer of the reference clip: q and k of 40 heads out of the projections, normed per head
        _rotary("rotary_reference", "rotary", 1, 40, 40, (18, 48, 84), 128, (44, 42, 42), "bf16", "interleaved", "axis", True, False),
        # an odd image batch with shared key heads, positions given per token, half-split pairs, part of the head rotated
        _rotary("rotary_odd_halves", "rotary", 2, 24, 8, (1, 45, 79), 128, (32, 32, 32), "fp16", "halves", "shared", True, True),
        # gradient at the mid workload's grid, with the norm's weights
        _rotary("rotary_bwd_mid", "rotary_bwd", 2, 8, 8, (4, 48, 84), 128, (16, 56, 56), "bf16", "interleaved", "axis", True, False),
        # gradient in 32 bits, odd sizes, no norm
        _rotary("rotary_bwd_odd", "rotary_bwd", 3, 5, 1, (3, 17, 29), 64, (16, 24, 24), "fp32", "halves", "shared", False, True),
        # one query token per item over a padded encoder: the smallest call
        _cross("cross_one_token", "cross", 4, 16, 16, 1, 512, 128, "bf16", "lengths"),
        # one layer of the reference clip against the encoder's 512 states
        _cross("cross_reference", "cross", 1, 40, 40, 72576, 512, 128, "bf16", "none"),
        # an odd image batch, shared key heads, a mask with holes
        _cross("cross_odd_mask", "cross", 2, 24, 8, 3555, 333, 64, "fp16", "mask"),
        # a few latent queries gather a whole clip: long keys
        _cross("cross_long_keys", "cross", 1, 16, 4, 256, 72576, 128, "bf16", "none"),
        # gradients: an odd small one, the mid grid with padded prompts, the reference clip
        _cross("cross_bwd_odd", "cross_bwd", 3, 6, 2, 777, 99, 64, "bf16", "mask"),
        _cross("cross_bwd_mid", "cross_bwd", 2, 8, 8, 16128, 512, 128, "bf16", "lengths"),
        _cross("cross_bwd_reference", "cross_bwd", 1, 40, 40, 72576, 256, 128, "bf16", "none"),
    ]


def _between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "rotary_bwd", "cross", "cross", "cross", "cross_bwd", "cross_bwd"])
    if op.startswith("rotary"):
        d = rng.choice([64, 128])
        Hk = rng.choice([1, 2, 4, 5, 8, 10, 20])
        Hq = Hk * rng.choice([1, 1, 2, 3])
        B = rng.choice([1, 1, 2, 3])
        F, Hl, Wl = _between(rng, 1, 20), _between(rng, 1, 60), _between(rng, 1, 90)
        while B * (Hq + Hk) * F * Hl * Wl * d > 80 * 72576 * 128 // 2:
            F = max(1, F // 2)
            Hl = max(1, Hl - 3)
        step = rng.choice([1, 2])
        dims = [2 * step * rng.randint(1, d // 8 // step) for _ in range(3)]
        if rng.random() < 0.5:
            dims[2] = d - dims[0] - dims[1]
        return {"op": op, "B": B, "Hq": Hq, "Hk": Hk, "F": F, "Hl": Hl, "Wl": Wl, "d": d, "dt": dims[0], "dh": dims[1],
                "dw": dims[2], "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "pairing": rng.choice(["interleaved", "halves"]), "spectrum": rng.choice(["axis", "shared"]),
                "norm": rng.random() < 0.5, "given": rng.random() < 0.5}
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 10])
    Hq = Hkv * rng.choice([1, 1, 2, 3])
    B = rng.choice([1, 1, 2, 3])
    mask = rng.choice(["none", "lengths", "mask"])
    if op == "cross":
        kind = rng.choice(["few", "tokens", "long"])
        Nq = _between(rng, 1, 32) if kind == "few" else _between(rng, 33, 72576)
        Nk = _between(rng, 1024, 72576) if kind == "long" else _between(rng, 1, 1024)
    else:
        Nq, Nk = _between(rng, 16, 72576), _between(rng, 24, 1024)
    most = 40 * 72576 * 512 // 2 if op == "cross" else 40 * 72576 * 256 // 2
    while B * Hq * Nq * Nk > most:
        Nq = max(16, Nq // 2)
        Nk = max(24, Nk - Nk // 4)
    return {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "d": d,
            "dtype": rng.choice(["bf16", "fp16"]) if op == "cross" else "bf16", "mask": mask}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    s = {"case": case}
    B, d = case["B"], case["d"]
    if case["op"].startswith("rotary"):
        grid = (case["F"], case["Hl"], case["Wl"])
        N = grid[0] * grid[1] * grid[2]
        # the projections' results, [B, N, H, d]
        s["q"] = rand(B, N, case["Hq"], d, scale=1.7).transpose(1, 2)
        s["k"] = rand(B, N, case["Hk"], d, scale=0.8).transpose(1, 2)
        s["positions"] = None
        if case["given"]:
            # each item's own origin (a crop of a larger image, a later part of a clip)
            at = torch.randint(0, 2000, (B, 1, 3), generator=gen, device="cuda")
            s["positions"] = (_raster(grid) + at).float()
        s["wq"] = s["wk"] = None
        if case["norm"]:
            s["wq"], s["wk"] = (1 + 0.2 * torch.randn(2, d, generator=gen, device="cuda")).to(dtype).unbind(0)
        if case["op"] == "rotary_bwd":
            # the gradients come in the attention's layout, [B, H, N, d]
            s["dqo"], s["dko"] = rand(B, case["Hq"], N, d, scale=0.5), rand(B, case["Hk"], N, d, scale=0.5)
        return s
    Hq, Hkv, Nq, Nk = case["Hq"], case["Hkv"], case["Nq"], case["Nk"]
    s["q"] = rand(B, Nq, Hq, d, scale=1.3).transpose(1, 2)
    s["k"] = rand(B, Nk, Hkv, d).transpose(1, 2)
    s["v"] = rand(B, Nk, Hkv, d).transpose(1, 2)
    s["key_len"] = s["key_mask"] = None
    if case["mask"] == "lengths":
        s["key_len"] = torch.randint(max(1, Nk // 8), Nk + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    elif case["mask"] == "mask":
        keep = torch.rand(B, Nk, generator=gen, device="cuda") < 0.7
        keep[:, 0] = True
        s["key_mask"] = keep
    if case["op"] == "cross_bwd":
        s["dout"] = rand(B, Hq, Nq, d)
        s["out"], s["lse"] = _attend(s)
    return s


# ---------------------------------------------------------------- plain forms

def _raster(grid):
    """Positions of a grid's tokens in raster order, [N, 3]."""
    t = torch.arange(grid[0] * grid[1] * grid[2], device="cuda")
    x = t % grid[2]
    y = t // grid[2] % grid[1]
    return torch.stack([t // (grid[1] * grid[2]), y, x], dim=1)


def _turn(c, positions):
    """cos and sin of every token's angles, [B or 1, 1, N, R / 2]: angles in 64 bits."""
    p = (_raster((c["F"], c["Hl"], c["Wl"])).unsqueeze(0) if positions is None else positions).double()
    half = torch.tensor([c["dt"] // 2, c["dh"] // 2, c["dw"] // 2], device="cuda")
    axis = torch.repeat_interleave(torch.arange(3, device="cuda"), half)
    i = torch.arange(axis.numel(), device="cuda", dtype=torch.float64)
    if c["spectrum"] == "axis":
        first = torch.cumsum(half, 0) - half
        power = (i - first[axis]) / half[axis]
    else:
        power = i / axis.numel()
    angle = p[:, :, axis] * torch.pow(torch.tensor(10000.0, device="cuda", dtype=torch.float64), -power)
    return torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)


def _rotate(x, cos, sin, pairing):
    R = 2 * cos.shape[-1]
    if pairing == "interleaved":
        u, v = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([u * cos - v * sin, u * sin + v * cos], dim=-1).flatten(-2)
    else:
        u, v = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([u * cos - v * sin, u * sin + v * cos], dim=-1)
    return torch.cat([y, x[..., R:]], dim=-1)


def _plain_rotary(x, w, cos, sin, pairing):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    return _rotate(y, cos, sin, pairing).to(x.dtype).contiguous()


def _plain_rotary_bwd(dy, x, w, cos, sin, pairing):
    dn = _rotate(dy.float(), cos, -sin, pairing)
    if w is None:
        return dn.to(x.dtype), None
    x32 = x.float()
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + 1e-6)
    g = dn * w.float()
    dx = r * (g - x32 * (r * r * (x32 * g).mean(-1, keepdim=True)))
    dw = (dn * x32 * r).double().sum((0, 1, 2)).float()
    return dx.to(x.dtype), dw


def _kept(s):
    """[B, 1, 1, 1, Nk] truth values, or None."""
    if s["key_len"] is not None:
        keep = torch.arange(s["k"].shape[2], device="cuda") < s["key_len"].unsqueeze(1)
    elif s["key_mask"] is not None:
        keep = s["key_mask"]
    else:
        return None
    return keep[:, None, None, None, :]


def _grouped(s):
    """q as [B, Hkv, G, Nq, d], k and v as [B, Hkv, 1, Nk, d], in 32 bits, masked rows of k and v at zero."""
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    keep = _kept(s)
    if keep is not None:
        rows = keep[:, 0, 0, 0, None, :, None][:, 0]
        rows = rows.reshape(rows.shape[0], 1, -1, 1)
        k, v = torch.where(rows, k, 0.0), torch.where(rows, v, 0.0)
    q = q.unflatten(1, (k.shape[1], -1))
    return q, k.unsqueeze(2), v.unsqueeze(2), keep


def _attend(s):
    q, k, v, keep = _grouped(s)
    x = q @ k.transpose(-1, -2)
    x *= 1.0 / math.sqrt(q.shape[-1])
    if keep is not None:
        x.masked_fill_(~keep, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x @ v) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + m
    return out.flatten(1, 2).to(s["q"].dtype), lse.flatten(1, 2).squeeze(-1)


def _attend_bwd(s):
    q, k, v, keep = _grouped(s)
    scale = 1.0 / math.sqrt(q.shape[-1])
    dout, out = (s[n].float().unflatten(1, q.shape[1:3]) for n in ("dout", "out"))
    lse = s["lse"].unflatten(1, q.shape[1:3]).unsqueeze(-1)
    p = q @ k.transpose(-1, -2)
    p = p.mul_(scale).sub_(lse).exp_()
    if keep is not None:
        p.masked_fill_(~keep, 0.0)
    dv = (p.transpose(-1, -2) @ dout).sum(2)
    ds = dout @ v.transpose(-1, -2)
    ds = ds.sub_((dout * out).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = (ds @ k).flatten(1, 2)
    dk = (ds.transpose(-1, -2) @ q).sum(2)
    t = s["q"].dtype
    return dq.to(t), dk.to(t), dv.to(t)


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "rotary":
        cos, sin = _turn(c, s["positions"])
        return (_plain_rotary(s["q"], s["wq"], cos, sin, c["pairing"]),
                _plain_rotary(s["k"], s["wk"], cos, sin, c["pairing"]))
    if c["op"] == "rotary_bwd":
        cos, sin = _turn(c, s["positions"])
        dq, dwq = _plain_rotary_bwd(s["dqo"], s["q"], s["wq"], cos, sin, c["pairing"])
        dk, dwk = _plain_rotary_bwd(s["dko"], s["k"], s["wk"], cos, sin, c["pairing"])
        return dq, dk, dwq, dwk
    if c["op"] == "cross":
        return _attend(s)
    return _attend_bwd(s)


def _run_own(s, c):
    import block_sparse_attention_spark_b200 as spark

    if "params" not in s:  # made once by a user's program, as the workspace is
        if c["op"].startswith("rotary"):
            s["params"] = spark.rotary_params(
                c["B"], c["Hq"], c["F"] * c["Hl"] * c["Wl"], c["d"], (c["dt"], c["dh"], c["dw"]), heads_k=c["Hk"],
                grid=None if c["given"] else (c["F"], c["Hl"], c["Wl"]), dtype=c["dtype"], pairing=c["pairing"],
                spectrum=c["spectrum"], theta=10000.0, eps=1e-6)
            s["ws"] = spark.alloc_rotary_workspace(s["params"])
        else:
            s["params"] = spark.cross_params(c["B"], c["Hq"], c["Nq"], c["Nk"], c["d"], heads_kv=c["Hkv"], dtype=c["dtype"])
            s["ws"] = spark.alloc_cross_workspace(s["params"], bwd=c["op"] == "cross_bwd")
    p, ws = s["params"], s["ws"]
    if c["op"] == "rotary":
        return spark.rotary(p, s["q"], s["k"], positions=s["positions"], q_weight=s["wq"], k_weight=s["wk"])
    if c["op"] == "rotary_bwd":
        return spark.rotary_bwd(p, s["dqo"], s["dko"], s["q"], s["k"], positions=s["positions"], q_weight=s["wq"],
                                k_weight=s["wk"], ws=ws)
    if c["op"] == "cross":
        return spark.cross_attn(p, s["q"], s["k"], s["v"], ws=ws, key_len=s["key_len"], key_mask=s["key_mask"],
                                return_lse=True)
    return spark.cross_attn_bwd(p, s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], ws=ws, key_len=s["key_len"],
                                key_mask=s["key_mask"])


def work(case):
    c, size = case, SIZES[case["dtype"]]
    if c["op"].startswith("rotary"):
        tokens = c["B"] * c["F"] * c["Hl"] * c["Wl"]
        values = tokens * (c["Hq"] + c["Hk"]) * c["d"]
        passes = 2 if c["op"] == "rotary" or not c["norm"] else 3
        positions = 12 * tokens if c["given"] else 0
        return {"bytes": passes * values * size + positions, "flops": (6 if passes == 2 else 16) * values}
    B, Hq, Hkv, Nq, Nk, d = (c[n] for n in ("B", "Hq", "Hkv", "Nq", "Nk", "d"))
    # the keys that are kept, on average over what prepare draws
    kept = Nk * {"none": 1.0, "lengths": 0.5625, "mask": 0.7}[c["mask"]]
    rows, keys = B * Hq * Nq, B * Hkv * kept
    if c["op"] == "cross":
        return {"bytes": size * d * (2 * rows + 2 * keys) + 4 * rows, "flops": 4.0 * rows * kept * d}
    return {"bytes": size * d * (4 * rows + 2 * keys + 2 * B * Hkv * Nk) + 4 * rows, "flops": 10.0 * rows * kept * d}


# ---------------------------------------------------------------- the definition in 64 bits

def _spin(c, positions):
    """e^{i angle}, [B or 1, 1, N, R / 2]."""
    F, Hl, Wl = c["F"], c["Hl"], c["Wl"]
    if positions is None:
        f, y, x = torch.meshgrid(*(torch.arange(n, device="cuda", dtype=torch.float64) for n in (F, Hl, Wl)), indexing="ij")
        p = [a.reshape(1, -1, 1) for a in (f, y, x)]
    else:
        p = [positions[:, :, a:a + 1].double() for a in range(3)]
    R = c["dt"] + c["dh"] + c["dw"]
    angles, i = [], 0
    for a, n in enumerate((c["dt"], c["dh"], c["dw"])):
        powers = [2.0 * j / n if c["spectrum"] == "axis" else 2.0 * (i + j) / R for j in range(n // 2)]
        angles.append(p[a] * torch.tensor([10000.0 ** -e for e in powers], device="cuda", dtype=torch.float64))
        i += n // 2
    angle = torch.cat(angles, dim=-1).unsqueeze(1)
    return torch.polar(torch.ones_like(angle), angle)


def _times(x, z, pairing):
    """The first 2 * (pairs) values of each row as complex numbers, times z."""
    R = 2 * z.shape[-1]
    y = x.clone()
    if pairing == "interleaved":
        y[..., :R] = torch.view_as_real(torch.view_as_complex(x[..., :R].reshape(*x.shape[:-1], -1, 2).contiguous()) * z).flatten(-2)
    else:
        w = torch.complex(x[..., :R // 2], x[..., R // 2:R]) * z
        y[..., :R // 2], y[..., R // 2:R] = w.real, w.imag
    return y


def _exact_rotary_bwd(dy, x, w, z, pairing):
    dn = _times(dy.double(), z.conj(), pairing)
    if w is None:
        return dn, None
    x, w = x.double(), w.double()
    norm = torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)
    h = x / norm
    g = dn * w
    return (g - h * (g * h).sum(-1, keepdim=True) / x.shape[-1]) / norm, torch.einsum("bhnd,bhnd->d", dn, h)


def _exact_rotary(x, w, z, pairing):
    y = x.double()
    if w is not None:
        y = w.double() * y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + 1e-6)
    return _times(y, z, pairing)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rotary"):
        z = _spin(case, s["positions"])
        if case["op"] == "rotary":
            return (_exact_rotary(s["q"], s["wq"], z, case["pairing"]), _exact_rotary(s["k"], s["wk"], z, case["pairing"]))
        dq, dwq = _exact_rotary_bwd(s["dqo"], s["q"], s["wq"], z, case["pairing"])
        dk, dwk = _exact_rotary_bwd(s["dko"], s["k"], s["wk"], z, case["pairing"])
        return dq, dk, dwq, dwk
    Nk, scale = case["Nk"], case["d"] ** -0.5
    group = case["Hq"] // case["Hkv"]
    outs = [torch.zeros_like(s["q"], dtype=torch.float64, memory_format=torch.contiguous_format) for _ in range(2)]
    lse = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros(case["B"], case["Hkv"], Nk, case["d"], dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(case["B"]):
        keep = torch.ones(Nk, dtype=torch.bool, device="cuda")
        if s["key_len"] is not None:
            keep[int(s["key_len"][b]):] = False
        if s["key_mask"] is not None:
            keep = s["key_mask"][b]
        at = keep.nonzero().squeeze(1)
        for h in range(case["Hq"]):
            q, k, v = s["q"][b, h].double(), s["k"][b, h // group, at].double(), s["v"][b, h // group, at].double()
            x = scale * torch.mm(q, k.t())
            lse[b, h] = torch.logsumexp(x, dim=1)
            p = torch.exp(x - lse[b, h].unsqueeze(1))
            o = torch.mm(p, v)
            outs[0][b, h] = o
            if case["op"] == "cross_bwd":
                do = s["dout"][b, h].double()
                dv[b, h // group].index_add_(0, at, torch.mm(p.t(), do))
                ds = p * (torch.mm(do, v.t()) - (do * o).sum(1, keepdim=True))
                outs[1][b, h] = scale * torch.mm(ds, k)
                dk[b, h // group].index_add_(0, at, scale * torch.mm(ds.t(), q))
    if case["op"] == "cross":
        return outs[0], lse
    return outs[1], dk, dv
