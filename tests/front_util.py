"""Plain 64-bit forms of what stands between the projections and the mixers
(head norms with rotary positions, the short causal convolution) and their
gradients, written from the definitions, and how far fp32 arithmetic may be off.

A bound counts roundings of 2^-24 (fp32, half a step relative to the value)
along each path, against the sum of the magnitudes that enter, and at the end
the rounding to the output's type, torch.finfo(t).eps / 2 of the value."""
from __future__ import annotations

import math

import torch

D = 128
U = 2.0 ** -24
TINY = 1e-36    # fp32 results below this may be zero


def half_step(x, dtype):
    return torch.finfo(dtype).eps / 2 * x.abs()


def places(lens):
    """(sequence, position within it) of the packed tokens."""
    seq = torch.cat([torch.full((n,), i) for i, n in enumerate(lens)] + [torch.zeros(0)]).long()
    pos = torch.cat([torch.arange(n) for n in lens] + [torch.zeros(0)]).long()
    return seq, pos


# ---------------------------------------------------------------- rotary positions
def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """Radians a token of pair i < rot / 2."""
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" else base
        f = b ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            keep = min(1.0, max(0.0, (original_len * f / (2 * math.pi) - low) / (high - low)))
            f = f * keep + f / factor * (1 - keep)
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def pairs(rot, layout):
    """Elements of the pairs: (first, second), each [rot / 2]."""
    i = torch.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def turn(x, pos, freqs, layout, magnitude=1.0, sign=1.0):
    """x [T, h, 128] rotated by the positions [T], in 64 bits."""
    y = x.clone()
    rot = 2 * len(freqs)
    if rot == 0:
        return y
    a, b = pairs(rot, layout)
    ang = pos.double()[:, None, None] * freqs
    c, s = magnitude * torch.cos(ang), magnitude * torch.sin(ang) * sign
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def reach(x, rot, layout, magnitude):
    """What errors of a rotation scale with: m (|a| + |b|) of each pair, |x| of the rest."""
    y = x.abs()
    if rot == 0:
        return y
    a, b = pairs(rot, layout)
    both = magnitude * (y[..., a] + y[..., b])
    y[..., a] = both
    y[..., b] = both
    return y


def inv_norm(x, norm, eps):
    ss = (x * x).sum(-1, keepdim=True)
    return 1.0 / torch.sqrt((ss / D if norm == "rms" else ss) + eps)


def normed(x, norm, weight, eps):
    x = x.double()
    if norm != "none":
        x = x * inv_norm(x, norm, eps)
        if weight is not None:
            x = x * weight.double()
    return x


def rope_ref(x, pos, freqs, layout="half", magnitude=1.0, norm="none", weight=None, eps=1e-6):
    """(y, bound without the final rounding).

    fp32: r to 8 roundings (squares and a sum of 128 in 7 levels, halved by the
    root: 4; the root 2; the sum with eps, the division by 128 exact: 1), x r w 2,
    the magnitude 1, products and sum 2, cos and sin to 2 ulp (4 roundings)
    and an angle to 2^-25 half turns (1.6 of 2^-24): 19 in all, of |a| + |b|."""
    u = normed(x, norm, weight, eps)
    return turn(u, pos, freqs, layout, magnitude), 19 * U * reach(u, 2 * len(freqs), layout, magnitude) + TINY


def rope_bwd_ref(x, dy, pos, freqs, layout="half", magnitude=1.0, norm="none", weight=None, eps=1e-6, rows=64):
    """(dx, dw, their bounds without the final rounding).  rows: heads that one
    running sum of the weight's gradient takes, at most.

    du is off by 9 roundings of its reach, n by 10 of itself; the sum over a
    head by 8 more, so dx by 9 + 10 + 10 + 8 + 3 = 40 of r (|dn| + |n| sum |dn n|)."""
    du = turn(dy.double(), pos, freqs, layout, magnitude, -1.0)
    mass = reach(dy.double(), 2 * len(freqs), layout, magnitude)
    if norm == "none":
        return du, None, 9 * U * mass + TINY, None
    x = x.double()
    r = inv_norm(x, norm, eps)
    n = x * r
    dw = (du * n).sum((0, 1))
    bw = (9 + 10 + 2 + rows + 24) * U * (mass * n.abs()).sum((0, 1)) + TINY
    w = torch.ones(D, dtype=torch.float64) if weight is None else weight.double()
    dn, mn = du * w, mass * w.abs()
    k = 1.0 / D if norm == "rms" else 1.0
    dx = r * (dn - n * (dn * n).sum(-1, keepdim=True) * k)
    return dx, dw, 40 * U * r * (mn + n.abs() * (mn * n.abs()).sum(-1, keepdim=True) * k) + TINY, bw


# ---------------------------------------------------------------- the convolution
def padded(x, state, lens, W):
    """Per sequence the kept inputs and the tokens: a list of [W - 1 + n, C] in 64 bits."""
    out, at = [], 0
    for i, n in enumerate(lens):
        s = state[i].double() if state is not None else torch.zeros(W - 1, x.shape[1], dtype=torch.float64)
        out.append(torch.cat([s, x[at:at + n].double()]))
        at += n
    return out


class Conv:
    """Forward, gradients and bounds of one convolution; everything in 64 bits."""

    def __init__(self, x, weight, h_qk, bias=None, state=None, lens=None, silu=True, norm=True, eps=1e-6):
        self.T, self.C = x.shape
        self.W, self.h_qk, self.silu, self.norm, self.eps = weight.shape[1], h_qk, silu, norm, eps
        self.lens = [self.T] if lens is None else list(lens)
        self.w = weight.double()
        b = torch.zeros(self.C, dtype=torch.float64) if bias is None else bias.double()
        self.xs = padded(x, state, self.lens, self.W)
        W = self.W
        u, mag = [], []
        for xp, n in zip(self.xs, self.lens):
            u.append(sum((xp[j:j + n] * self.w[:, j] for j in range(W)), b.expand(n, -1)))
            mag.append(sum((xp[j:j + n].abs() * self.w[:, j].abs() for j in range(W)), b.abs().expand(n, -1)))
        self.u, mag = torch.cat(u), torch.cat(mag)
        self.eu = (W + 1) * U * mag                    # a rounding a tap
        self.last = torch.stack([xp[n:] for xp, n in zip(self.xs, self.lens)])
        s = torch.sigmoid(self.u) if silu else torch.ones_like(self.u)
        self.s = s
        y = (self.u * s).view(self.T, self.C // D, D)
        # the exponential to 2 + 1.173 |u| ulp (two roundings each), in a sigmoid times 1 - s; the sum and
        # the quotient 3 ulp, the product one: and the slope of u sigmoid(u) is at most 1.1
        self.ds = (2 * ((2 + 1.173 * self.u.abs()) * (1 - s) + 3) * U * s) if silu else torch.zeros_like(s)
        ey = ((1.1 if silu else 1.0) * self.eu + self.u.abs() * self.ds + 2 * U * (self.u * s).abs()).view(y.shape)
        self.y, self.ey = y, ey
        self.unit = torch.zeros(y.shape[1], dtype=torch.bool)
        if norm:
            self.unit[:2 * h_qk] = True
        r = 1.0 / torch.sqrt((y * y).sum(-1, keepdim=True) + eps)
        self.r = torch.where(self.unit[:, None], r, torch.ones_like(r))
        # r: half of what the sum is off by, relative to itself; its own arithmetic 8 roundings
        rel = (y.abs() * ey).sum(-1, keepdim=True) * self.r ** 2 + 8 * U
        self.rel = torch.where(self.unit[:, None], rel, torch.zeros_like(rel))
        out = y * self.r
        bound = self.r * ey + out.abs() * (self.rel + U) + TINY
        split = lambda t: (t[:, :h_qk], t[:, h_qk:2 * h_qk], t[:, 2 * h_qk:])  # noqa: E731
        self.out, self.bounds, self.n, self.en = split(out), split(bound), out, bound

    def backward(self, d_q, d_k, d_v, d_final=None, rows=64):
        """dx, d_weight, d_bias, d_state and their bounds."""
        W, C = self.W, self.C
        g = torch.cat([d_q, d_k, d_v], 1).double()
        m = self.unit[:, None]
        gn = (g * self.n).sum(-1, keepdim=True)
        mass = (g * self.n).abs().sum(-1, keepdim=True)
        dy = torch.where(m, self.r * (g - self.n * gn), g)
        size = self.r * (g.abs() + self.n.abs() * mass)
        edy = self.rel * size + self.r * (self.en * mass + self.n.abs() * (g.abs() * self.en).sum(-1, keepdim=True)) + 12 * U * size
        edy = torch.where(m, edy, torch.zeros_like(edy))
        dy, edy = dy.reshape(self.T, C), edy.reshape(self.T, C)
        if self.silu:
            slope = self.s + self.u * self.s * (1 - self.s)
            # the second derivative of u sigmoid(u) is at most 1/2
            eslope = 0.5 * self.eu + self.ds * (1 + self.u.abs()) + 4 * U * (1 + self.u.abs())
        else:
            slope, eslope = torch.ones_like(dy), torch.zeros_like(dy)
        du = dy * slope
        edu = edy * slope.abs() + dy.abs() * eslope + 2 * U * du.abs()
        dxs, exs = [torch.zeros_like(xp) for xp in self.xs], [torch.zeros_like(xp) for xp in self.xs]
        dw, ew = torch.zeros(C, W, dtype=torch.float64), torch.zeros(C, W, dtype=torch.float64)
        at = 0
        for i, n in enumerate(self.lens):
            part, epart = du[at:at + n], edu[at:at + n]
            at += n
            for j in range(W):
                dxs[i][j:j + n] += part * self.w[:, j]
                exs[i][j:j + n] += (epart + (W + 2) * U * part.abs()) * self.w[:, j].abs()
                xj = self.xs[i][j:j + n]
                dw[:, j] += (part * xj).sum(0)
                ew[:, j] += ((epart + (rows + 12) * U * part.abs()) * xj.abs()).sum(0)
            if d_final is not None:
                dxs[i][n:] += d_final[i].double()
                exs[i][n:] += U * d_final[i].double().abs()
        db = du.sum(0)
        eb = (edu + (rows + 12) * U * du.abs()).sum(0)
        head = lambda t: torch.stack([p[:W - 1] for p in t])  # noqa: E731
        tail = lambda t: torch.cat([p[W - 1:] for p in t])  # noqa: E731
        return (tail(dxs), dw, db, head(dxs)), (tail(exs) + TINY, ew + TINY, eb + TINY, head(exs) + TINY)


def check(name, got, want, bound, dtype=None):
    """got within bound plus its own rounding of want."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if not want.numel():
        return
    limit = bound * 1.01 + half_step(want, dtype or torch.float32) * 1.01
    err = ((got - want).abs() / limit)
    assert not got.isnan().any(), name
    assert err.max() <= 1, f"{name}: {err.max():.3f} of the bound"
