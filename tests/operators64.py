"""Plain 64-bit forms of the operators around the attention (rotary positions,
cross attention, their gradients), with the error bounds of a kernel that
computes in 32 bits and rounds where its contract says so."""

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24


def angles(dims, spectrum, theta, positions, start=(0, 0, 0), scale=(1, 1, 1)):
    """[..., R/2] angles of positions [..., axes]."""
    R = sum(dims)
    cols, i = [], 0
    for a, n in enumerate(dims):
        for j in range(n // 2):
            f = theta ** (-2.0 * j / n) if spectrum == "axis" else theta ** (-2.0 * i / R)
            cols.append((start[a] + scale[a] * positions[..., a].double()) * f)
            i += 1
    return torch.stack(cols, -1) if cols else positions.new_zeros(*positions.shape[:-1], 0, dtype=torch.float64)


def raster(grid, device):
    ax = torch.meshgrid(*(torch.arange(n, device=device) for n in grid), indexing="ij")
    return torch.stack([a.reshape(-1) for a in ax], -1)


def pair_index(R, pairing, device):
    i = torch.arange(R // 2, device=device)
    return (2 * i, 2 * i + 1) if pairing == "interleaved" else (i, i + R // 2)


def turn(x, ang, pairing, sign=1.0):
    """x [B,H,N,d] float64, ang [B or 1, N, R/2]."""
    y = x.clone()
    iu, iv = pair_index(2 * ang.shape[-1], pairing, x.device)
    c, s = torch.cos(ang).unsqueeze(1), sign * torch.sin(ang).unsqueeze(1)
    u, v = x[..., iu], x[..., iv]
    y[..., iu], y[..., iv] = u * c - v * s, u * s + v * c
    return y


def pair_size(x, R, pairing):
    """|u| + |v| of each value's pair (its own size for a kept value)."""
    y = x.abs()
    iu, iv = pair_index(R, pairing, x.device)
    t = y[..., iu] + y[..., iv]
    y[..., iu], y[..., iv] = t, t
    return y


def rotary(x, w, ang, pairing, eps):
    """(result, bound) in 64 bits."""
    n = x.double()
    if w is not None:
        n = n * torch.rsqrt(n.square().mean(-1, keepdim=True) + eps) * w.double()
    y = turn(n, ang, pairing)
    # mean of squares and its root: at most 8 steps of 32 bits; two products; the angle rounded to 32 bits
    # (at most pi * 2^-24 of it), sincospi to 2 ulp, two products and a sum: below 32 steps of the pair's size
    bound = HALF[x.dtype] * y.abs() + 32 * U32 * pair_size(n, 2 * ang.shape[-1], pairing)
    if x.dtype == torch.float16:
        bound = bound + 2.0 ** -25               # half a step of the subnormals
    return y, bound


def rotary_bwd(dy, x, w, ang, pairing, eps):
    """(dx, bound, dw, bound)."""
    dn = turn(dy.double(), ang, pairing, -1.0)
    size = pair_size(dy.double(), 2 * ang.shape[-1], pairing)
    if w is None:
        bound = HALF[dy.dtype] * dn.abs() + 16 * U32 * size
        return dn, bound + (2.0 ** -25 if dy.dtype == torch.float16 else 0), None, None
    x, w = x.double(), w.double()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    g = dn * w
    t = (x * g).mean(-1, keepdim=True)
    dx = r * (g - x * r * r * t)
    # 16 steps for dn, 10 for r, 12 for the mean (a sum of d terms in a tree of eights), 3 r's and 4 products
    gb = size * w.abs()
    bound = HALF[dy.dtype] * dx.abs() + 64 * U32 * (r * (gb + x.abs() * r * r * (x.abs() * gb).mean(-1, keepdim=True)))
    dw = (dn * x * r).sum((0, 1, 2))
    # a thread adds at most 4096 rows here before 64-bit sums take over
    dwb = (64 + 4096) * U32 * (size * x.abs() * r).sum((0, 1, 2)) + 2.0 ** -24 * dw.abs()
    return dx, bound + (2.0 ** -25 if dy.dtype == torch.float16 else 0), dw, dwb


class Cross:
    """Cross attention of one call in 64 bits, with bounds for a kernel that rounds P (and dS) to the type."""

    def __init__(self, q, k, v, key_len=None, key_mask=None, scale=None):
        B, Hq, Nq, d = q.shape
        Hkv, Nk = k.shape[1], k.shape[2]
        self.dtype, self.G, self.d = q.dtype, Hq // Hkv, d
        self.scale = d ** -0.5 if scale is None else scale
        keep = torch.ones(B, Nk, dtype=torch.bool, device=q.device)
        if key_len is not None:
            keep &= torch.arange(Nk, device=q.device) < key_len.clamp(0, Nk).unsqueeze(1)
        if key_mask is not None:
            keep &= key_mask.bool()
        self.keep = keep[:, None, None, :]
        rows = keep[:, None, :, None]
        zero = torch.zeros((), dtype=torch.float64, device=q.device)
        self.q = q.double()
        self.k = torch.where(rows, k.double(), zero).repeat_interleave(self.G, 1)
        self.v = torch.where(rows, v.double(), zero).repeat_interleave(self.G, 1)
        x = self.scale * self.q @ self.k.transpose(-1, -2)
        x = x.masked_fill(~self.keep, -math.inf)
        self.lse = torch.logsumexp(x, -1)
        self.p = torch.where(self.keep, torch.exp(x - self.lse.unsqueeze(-1)), zero)
        self.p = torch.nan_to_num(self.p)
        self.out = self.p @ self.v
        # logits: d products summed in 32 bits, with one step per term and one for the scale
        size = self.scale * (self.q.abs().amax(-1) * self.k.abs().sum(-1).amax(-1, keepdim=True))
        self.es = ((d + 8) * U32 * size).unsqueeze(-1) + 2.0 ** -21      # and exp2 to 2^-22

    def forward_bounds(self):
        half = HALF[self.dtype]
        pv = self.p @ self.v.abs()
        out = half * (pv + self.out.abs()) + (3 * self.es + 64 * U32) * pv
        if self.dtype == torch.float16:
            out = out + 2.0 ** -25 * (1 + self.v.abs().sum(-2, keepdim=True))
        lse = self.es.squeeze(-1) + 64 * U32 * (1 + self.lse.abs().nan_to_num(0, 0, 0))
        return out, lse

    def backward(self, dout):
        """(dq, dk, dv) and their bounds."""
        half, do = HALF[self.dtype], dout.double()
        dp = do @ self.v.transpose(-1, -2)
        delta = (do * self.out).sum(-1, keepdim=True)
        ds = self.p * (dp - delta)
        dq = self.scale * ds @ self.k
        dk = self.scale * ds.transpose(-1, -2) @ self.q
        dv = self.p.transpose(-1, -2) @ do
        # dS: its own rounding; delta from the rounded out; dP and delta in 32 bits; P's relative error (lse and logits)
        dps = do.abs() @ self.v.abs().transpose(-1, -2)
        dds = (do * self.out).abs().sum(-1, keepdim=True)
        eds = half * ds.abs() + self.p * (half * dds + (self.d + 8) * U32 * (dps + dds)) \
            + (4 * self.es + 128 * U32 * (1 + self.lse.abs().nan_to_num(0, 0, 0)).unsqueeze(-1)) * self.p * (dps + dds)
        ep = (half + 4 * self.es + 128 * U32 * (1 + self.lse.abs().nan_to_num(0, 0, 0)).unsqueeze(-1)) * self.p
        n = self.q.shape[2] * self.G
        acc = 2.0 ** -24 * 64 + 2.0 ** -24 * math.sqrt(n)
        bq = half * dq.abs() + self.scale * (eds + acc * ds.abs()) @ self.k.abs()
        bk = self.scale * (eds + acc * ds.abs()).transpose(-1, -2) @ self.q.abs()
        bv = (ep + acc * self.p).transpose(-1, -2) @ do.abs()
        dk, dv, bk, bv = (t.unflatten(1, (-1, self.G)).sum(2) for t in (dk, dv, bk, bv))
        return (dq, dk, dv), (bq, half * dk.abs() + bk, half * dv.abs() + bv)


def check(got, want, bound, name):
    got = got.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), f"{name}: finite where it should not be, or the reverse"
    assert torch.equal(got[~fin], want[~fin]), name
    bad = (got - want).abs()[fin] > (bound.expand_as(want)[fin] + 1e-30)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} past the bound, worst "
                           f"{float(((got - want).abs()[fin] / (bound.expand_as(want)[fin] + 1e-30)).max()):.3g} bounds")
