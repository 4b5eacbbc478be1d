"""Plain 64-bit forms of the 8-bit key/value cache's operators, written from
their definitions, and the bounds their results are held to."""
from __future__ import annotations

import math

import torch

PAGE, D = 64, 128
E_MIN, E_MAX = -40, 40


def e4m3(y: torch.Tensor) -> torch.Tensor:
    """Nearest e4m3 value, ties to even, saturating at 448; NaN for what is not finite."""
    f = torch.where(y.isfinite(), y, torch.zeros_like(y)).double()
    e = (torch.frexp(f)[1] - 1).clamp(min=-6).double()
    step = torch.pow(2.0, e - 3)
    r = (torch.round(f / step) * step).clamp(-448, 448)
    return torch.where(y.isfinite(), r, torch.full_like(r, math.nan))


def scale_exp(a: float) -> int:
    """Exponent of the smallest power of two s with a / s <= 448, within [E_MIN, E_MAX]."""
    if a == 0:
        return E_MIN
    e = math.frexp(a)[1] - 10
    while 448.0 * 2.0 ** e < a:
        e += 1
    return min(max(e, E_MIN), E_MAX)


class Batch:
    """Lengths, a shuffled page table and the values of a cache, on the CPU in 64 bits."""

    def __init__(self, q_lens, kv_lens, h_kv, seed=0, n_pages=None, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.q_lens, self.kv_lens, self.h_kv = g, list(q_lens), list(kv_lens), h_kv
        self.n = len(q_lens)
        pages = [-(-kv // PAGE) for kv in kv_lens]
        self.max_pages = max(1, max(pages))
        need = sum(pages)
        self.n_pages = n_pages or need + 2
        perm = torch.randperm(self.n_pages, generator=g)[:need].tolist() if self.n_pages < 1 << 20 else [
            self.n_pages - 1 - 7 * i for i in range(need)]
        self.table = torch.zeros(self.n, self.max_pages, dtype=torch.int32)
        at = 0
        for i, p in enumerate(pages):
            self.table[i, :p] = torch.tensor(perm[at:at + p], dtype=torch.int32)
            at += p
        self.T = sum(q_lens)
        self.cu = torch.tensor([0] + list(q_lens)).cumsum(0).to(torch.int32)
        self.lens = torch.tensor(kv_lens, dtype=torch.int32)
        self.spread = spread

    def randn(self, *s):
        return torch.randn(*s, generator=self.g)

    def fill(self, stale_nan=True):
        """Random codes and scales for every page in use: (codes as fp64 values, scales)."""
        out = []
        for _ in range(2):
            x = self.randn(self.n_pages, self.h_kv, PAGE, D) * torch.exp(self.spread * self.randn(self.n_pages, self.h_kv, 1, 1))
            s = torch.tensor([[2.0 ** scale_exp(float(a)) for a in row] for row in x.abs().amax((2, 3)).tolist()])
            c = e4m3(x / s[:, :, None, None]).float()
            out += [c, s]
        if stale_nan:  # rows after a sequence's end hold anything
            for i, kv in enumerate(self.kv_lens):
                if kv % PAGE:
                    page = int(self.table[i, kv // PAGE])
                    out[0][page, :, kv % PAGE:] = math.nan
                    out[2][page, :, kv % PAGE:] = math.nan
        self.k, self.ks, self.v, self.vs = out
        return out

    def tokens(self, which, i):
        """[kv, h_kv, 128] values of sequence i in 64 bits."""
        c, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        kv = self.kv_lens[i]
        pages = self.table[i, :-(-kv // PAGE)].long()
        x = c[pages].double() * s[pages].double()[..., None, None]
        return x.transpose(1, 2).reshape(-1, self.h_kv, D)[:kv]


def append_ref(b: Batch, k, v):
    """(codes, scale) of keys and values after the new tokens k, v [T, h_kv, 128]."""
    outs = []
    for x, c0, s0 in ((k, b.k, b.ks), (v, b.v, b.vs)):
        c, s, x = c0.double().clone(), s0.double().clone(), x.double()
        for i, (n, kv) in enumerate(zip(b.q_lens, b.kv_lens)):
            past = kv - n
            for slot in range(max(past, 0) // PAGE, -(-kv // PAGE)) if n else ():
                lo, hi = max(past - slot * PAGE, 0), min(kv - slot * PAGE, PAGE)
                if hi <= lo:
                    continue
                page = int(b.table[i, slot])
                t0 = int(b.cu[i]) + slot * PAGE + lo - past
                rows = x[t0:t0 + hi - lo].transpose(0, 1)
                for h in range(b.h_kv):
                    fin = rows[h][rows[h].isfinite()]
                    new = 2.0 ** scale_exp(float(fin.abs().max()) if fin.numel() else 0.0)
                    if lo:
                        old = float(s[page, h])
                        new = max(new, old)
                        c[page, h, :lo] = e4m3(c[page, h, :lo] * (old / new))
                    c[page, h, lo:hi] = e4m3(rows[h] / new)
                    s[page, h] = new
        outs += [c, s]
    return outs


def attn_ref(b: Batch, q, causal=True, window=0, scale=None):
    """out, lse in 64 bits, and per element / row the amounts rounding errors scale with:
    mass = sum_j w_j |v_j|, reach = scale max|q| max_j sum_d |k_j|, top = max_j |s_j|."""
    T, h_q = q.shape[:2]
    scale = scale or 1.0 / math.sqrt(D)
    o = torch.zeros(T, h_q, D, dtype=torch.float64)
    mass = torch.zeros_like(o)
    lse = torch.full((T, h_q), -math.inf, dtype=torch.float64)
    reach = torch.zeros(T, h_q, dtype=torch.float64)
    top = torch.zeros(T, h_q, dtype=torch.float64)
    for i, (n, kv) in enumerate(zip(b.q_lens, b.kv_lens)):
        if not n or not kv:
            continue
        K, V = b.tokens("k", i), b.tokens("v", i)
        p = torch.arange(kv - n, kv)
        key = torch.arange(kv)
        keep = torch.ones(n, kv, dtype=torch.bool)
        if causal:
            keep &= key[None, :] <= p[:, None]
        if window:
            keep &= key[None, :] > p[:, None] - window
        sl = slice(int(b.cu[i]), int(b.cu[i]) + n)
        for j in range(h_q):
            h = j * b.h_kv // h_q
            x = q[sl, j].double()
            s = (x @ K[:, h].T) * scale
            s = torch.where(keep, s, torch.full_like(s, -math.inf))
            z = torch.logsumexp(s, -1)
            w = torch.exp(s - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
            w = torch.where(keep, w, torch.zeros_like(w))
            v = V[:, h]
            o[sl, j] = torch.where(w[:, :, None] > 0, w[:, :, None] * v[None], torch.zeros(())).sum(1) if v.isnan().any() else w @ v
            mass[sl, j] = w @ v.abs().nan_to_num()
            lse[sl, j] = z
            reach[sl, j] = scale * x.abs().amax(-1) * K[:, h].abs().sum(-1).nan_to_num().max()
            top[sl, j] = torch.where(keep, s, torch.zeros_like(s)).abs().amax(-1)
    return o, lse, mass, reach, top


def half_ulp_bf16(x):
    return torch.pow(2.0, torch.frexp(x.abs().clamp(min=1e-30))[1].double() - 9)


def attn_bounds(o, mass, reach, top, dtype):
    """Bounds on |out - o| and |lse - ref|, from the arithmetic.

    bf16 calls: a query row enters as two e4m3 parts at 2^k, exact to 2^-10
    where the row's largest magnitude is in (224, 448]: 2^-17.8 of it, so a
    score is off by at most 2^-17.8 reach (+ fp32 sums of 128 terms, 2^-17 of
    sum |q k| in the worst order, taken as 2^-19 reach, and 2^-22 of |s| from
    the exponential's argument).  Weights enter the second product with two
    4-bit parts: 2^-8 relative at most.  Then one rounding to bf16.
    fp32 calls: sums of 128 terms, 2^-17 reach in the worst order; the softmax
    sums add up to 2^-16 of the mass over the tested lengths."""
    ds = 2.0 ** -17 * reach + 2.0 ** -20 * top + 2.0 ** -20
    if dtype == torch.bfloat16:
        return half_ulp_bf16(o) * 1.01 + (2.0 ** -8 * 1.25 + 2 * ds[..., None]) * mass + 1e-30, ds + 2.0 ** -16
    return (2.0 ** -16 + 2 * ds[..., None]) * mass + 1e-30, ds + 2.0 ** -18
