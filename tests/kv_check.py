"""Attention over the 8-bit cache against its 64-bit form, with what the
kernels drop of weights far below the largest in the bound."""
from __future__ import annotations

import math

import torch

from tests import kv_util as U

# What a kernel may drop of any weight, in units of the largest weight times
# value scale of the row, a value counted by its code.
#   few rows: P = 2^8 of the largest and hi + lo / 16 in e4m3; lo's subnormal
#     step is 2^-9, so half a step of P is 2^-14.
#   many rows: P = 2^3 of it or more, in fp16, whose subnormal step is 2^-24.
#   fp32: P = 2^14 of it, hi + lo in fp16.
FLOOR = {0: 2.0 ** -39, 1: 2.0 ** -22, 2: 2.0 ** -28}


def dropped(b: U.Batch, q, path, causal=True, window=0, scale=0.0):
    """[T, h_q, 128]: the sum over the attended keys of what may be dropped of each."""
    T, h_q = q.shape[:2]
    scale = scale or 1.0 / math.sqrt(U.D)
    out = torch.zeros(T, h_q, U.D, dtype=torch.float64)
    for i, (n, kv) in enumerate(zip(b.q_lens, b.kv_lens)):
        if not n or not kv:
            continue
        K = b.tokens("k", i)
        page = b.table[i, torch.arange(kv) // U.PAGE].long()
        codes, s = b.v[page, :, torch.arange(kv) % U.PAGE].double().nan_to_num().abs(), b.vs[page].double()
        p, key = torch.arange(kv - n, kv), torch.arange(kv)
        keep = torch.ones(n, kv, dtype=torch.bool)
        if causal:
            keep &= key[None, :] <= p[:, None]
        if window:
            keep &= key[None, :] > p[:, None] - window
        sl = slice(int(b.cu[i]), int(b.cu[i]) + n)
        for j in range(h_q):
            h = j * b.h_kv // h_q
            x = torch.where(keep, (q[sl, j].double() @ K[:, h].T) * scale, torch.full((), -math.inf, dtype=torch.float64))
            z = torch.logsumexp(x, -1)
            w = torch.where(keep, torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None]), torch.zeros(()).double())
            out[sl, j] = FLOOR[path] * (w * s[:, h]).nan_to_num().amax(-1)[:, None] * (keep.double() @ codes[:, h])
    return out


def check(gdn, b: U.Batch, h_q, plan, q=None, use_cu=True, dtype=torch.bfloat16):
    """Attention under `plan` (its masks and scale) within the bound.  Returns (out, lse)."""
    q = (b.randn(b.T, h_q, U.D) if q is None else q).to(dtype)
    dev = lambda c: c.float().to(torch.float8_e4m3fn).cuda()  # noqa: E731
    cache = gdn.KVCache(dev(b.k), dev(b.v), b.ks.float().cuda(), b.vs.float().cuda())
    out, lse = gdn.gdn_kv_attn(q.cuda(), cache, b.lens.cuda(), b.table.cuda(), b.cu.cuda() if use_cu else None, plan=plan)
    assert gdn.gdn_get_device_status(cache.status) == (0, 0)
    o, z, mass, reach, top = U.attn_ref(b, q, plan.causal, plan.window, plan.scale or None)
    if plan.scale < 0:
        reach = -reach
    bo, bz = U.attn_bounds(o, mass, reach, top, dtype)
    bo = bo + dropped(b, q, plan.raw.path, plan.causal, plan.window, plan.scale)
    got, got_z = out.double().cpu(), lse.double().cpu()
    empty = z == -math.inf
    assert torch.equal(got_z == -math.inf, empty) and (got[empty] == 0).all()
    assert not got.isnan().any()
    err = (got - o).abs() / bo
    assert err.max() <= 1, f"out: {err.max():.3f} of the bound"
    ez = ((got_z - z).abs() / bz)[~empty]
    assert ez.numel() == 0 or ez.max() <= 1, f"lse: {ez.max():.3f} of the bound"
    return out, lse
