"""Drawn calls of the operators between the projections and the mixers against
their 64-bit forms, and calls whose offsets pass 32 bits."""
from __future__ import annotations

import random

import pytest
import torch

from tests import front_util as F

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU, skipped there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_deltanet_linear_fwd_gb300 as gdn  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def draw_lens(r):
    return [0 if r.random() < 0.15 else int(2 ** r.uniform(0, 9)) for _ in range(r.choice([1, 1, 2, 5, 17]))] + [1]


def strided(r, t):
    """t on the GPU, half the time as a part of wider rows."""
    if r.random() < 0.5:
        return t.cuda()
    shape = list(t.shape)
    shape[1] += 3 if t.dim() == 3 else 136
    wide = torch.zeros(shape, dtype=t.dtype, device="cuda")
    part = wide[:, 1:1 + t.shape[1]] if t.dim() == 3 else wide[:, 64:64 + t.shape[1]]
    part.copy_(t)
    return part


@pytest.mark.parametrize("seed", range(16))
def test_rope(seed):
    r, g = random.Random(seed), torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    lens, dtype, layout, norm = draw_lens(r), r.choice([BF16, F32]), r.choice(["half", "interleaved"]), r.choice(["none", "rms", "unit"])
    rot, heads = 8 * r.randint(1, 16), [r.choice([1, 2, 3, 8, 25, 64]), r.choice([1, 2, 5, 8])]
    T, pos = sum(lens), F.places(lens)[1]
    pad = r.choice([0, 1, 6])   # tokens behind the last sequence
    xs = [rnd(T + pad, h, 128).to(dtype) for h in heads]
    ds = [rnd(T + pad, h, 128).to(dtype) for h in heads]
    ws = [1 + 0.3 * rnd(128) if norm != "none" and r.random() < 0.7 else None for _ in heads]
    mag = r.choice([1.0, 1.25])
    rope, f = gdn.gdn_rope_table(rot, layout=layout, base=5e5, magnitude=mag), F.frequencies(rot, 5e5)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    dev = [strided(r, x) for x in xs]
    outs = [strided(r, torch.full_like(x, 3.0)) for x in xs]
    how = dict(norm=norm, **{n + "_weight": None if w is None else w.cuda() for n, w in zip("qk", ws)})
    gdn.gdn_qk_rope(*dev, rope, None, cu, q_out=outs[0], k_out=outs[1], **how)
    grads = gdn.gdn_qk_rope_bwd(*dev, *[strided(r, d) for d in ds], rope, None, cu, **how)
    for i, (x, w) in enumerate(zip(xs, ws)):
        F.check("out", outs[i][:T], *F.rope_ref(x[:T], pos, f, layout, mag, norm, w), dtype)
        assert (outs[i][T:] == 3).all()
        dx, dw, bx, bw = F.rope_bwd_ref(x[:T], ds[i][:T], pos, f, layout, mag, norm, w)
        F.check("dx", grads[i][:T], dx, bx, dtype)
        if w is not None:
            F.check("dw", grads[2 + i], dw, bw)


@pytest.mark.parametrize("seed", range(16))
def test_conv(seed):
    r, g = random.Random(100 + seed), torch.Generator().manual_seed(100 + seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    lens, dtype, W = draw_lens(r), r.choice([BF16, F32]), r.choice([2, 3, 4])
    h_qk, h_v, silu, norm = r.choice([1, 2, 3]), r.choice([1, 2, 5, 8]), r.random() < 0.7, r.random() < 0.7
    T, C, n = sum(lens), (2 * h_qk + h_v) * 128, len(lens)
    pad = r.choice([0, 1, 6])
    x, w = rnd(T + pad, C).to(dtype), rnd(C, W) / 2
    bias = 0.3 * rnd(C) if r.random() < 0.5 else None
    state = rnd(n, W - 1, C).to(dtype) if r.random() < 0.5 else None
    d_final = rnd(n, W - 1, C).to(dtype) if r.random() < 0.5 else None
    d = [rnd(T + pad, h, 128).to(dtype) for h in (h_qk, h_qk, h_v)]
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    how = dict(activation="silu" if silu else "none", norm=norm)
    ref = F.Conv(x[:T], w, h_qk, bias, state, lens, silu, norm)
    gx = strided(r, x)
    outs = [torch.full_like(t, 3.0).cuda() for t in d]
    last = gdn.gdn_conv_fwd(gx, w.cuda(), h_qk, dev(bias), dev(state), cu, q=outs[0], k=outs[1], v=outs[2], **how)[3]
    for got, want, bound in zip(outs, ref.out, ref.bounds):
        F.check("out", got[:T], want, bound, dtype)
        assert (got[T:] == 3).all()
    assert torch.equal(last.double().cpu(), ref.last)
    dx = strided(r, torch.full_like(x, 3.0))
    got = gdn.gdn_conv_bwd(gx, w.cuda(), h_qk, *[t.cuda() for t in d], dev(bias), dev(state), dev(d_final), cu, dx=dx,
                           want_initial_state_grad=True, **how)
    want, bound = ref.backward(*[t[:T] for t in d], d_final)
    F.check("dx", dx[:T], want[0], bound[0], dtype)
    assert (dx[T:] == 3).all()
    F.check("dw", got[1], want[1], bound[1])
    if bias is not None:
        F.check("db", got[2], want[2], bound[2])
    F.check("d_state", got[3], want[3], bound[3], dtype)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_conv_of_many_short_sequences(W, dtype):
    """Hundreds of sequences of 0 to 9 tokens, runs of empty ones among them, states on both sides."""
    r, g = random.Random(W), torch.Generator().manual_seed(200 + W)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    lens = [r.choice([0, 1, 2, 3, 4, 4, 5, 8, 9]) for _ in range(150)] + [0] * 40 + [4] * 64 + [r.randint(0, 9) for _ in range(60)] + [0, 0]
    T, C, n = sum(lens), 512, len(lens)
    x, w, state, d_final = rnd(T, C).to(dtype), rnd(C, W) / 2, rnd(n, W - 1, C).to(dtype), rnd(n, W - 1, C).to(dtype)
    d = [rnd(T, h, 128).to(dtype) for h in (1, 1, 2)]
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    ref = F.Conv(x, w, 1, None, state, lens)
    q, k, v, last = gdn.gdn_conv_fwd(x.cuda(), w.cuda(), 1, None, state.cuda(), cu)
    for got, want, bound in zip((q, k, v), ref.out, ref.bounds):
        F.check("out", got, want, bound, dtype)
    assert torch.equal(last.double().cpu(), ref.last)
    got = gdn.gdn_conv_bwd(x.cuda(), w.cuda(), 1, *[t.cuda() for t in d], None, state.cuda(), d_final.cuda(), cu)
    want, bound = ref.backward(*d, d_final)
    F.check("dx", got[0], want[0], bound[0], dtype)
    F.check("dw", got[1], want[1], bound[1])
    F.check("d_state", got[3], want[3], bound[3], dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_heads(dtype):
    """More heads than tokens, and than a call has warps."""
    g = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, w = rnd(3, 5003, 128).to(dtype), rnd(3, 301, 128).to(dtype), 1 + 0.2 * rnd(128)
    rope, f, pos = gdn.gdn_rope_table(96), F.frequencies(96), torch.arange(3)
    dev = [t.cuda() for t in (q, k)]
    how = dict(norm="rms", q_weight=w.cuda(), k_weight=w.cuda())
    for got, x in zip(gdn.gdn_qk_rope(*dev, rope, **how), (q, k)):
        F.check("out", got, *F.rope_ref(x, pos, f, norm="rms", weight=w), dtype)
    grads = gdn.gdn_qk_rope_bwd(*dev, dev[0].flip(1), dev[1].flip(1), rope, **how)
    for i, x in enumerate((q, k)):
        dx, dw, bx, bw = F.rope_bwd_ref(x, x.flip(1), pos, f, norm="rms", weight=w)
        F.check("dx", grads[i], dx, bx, dtype)
        F.check("dw", grads[2 + i], dw, bw)
    h_qk, h_v, lens = 70, 131, [2, 5]
    x, taps = rnd(7, (2 * h_qk + h_v) * 128).to(dtype), rnd((2 * h_qk + h_v) * 128, 3) / 2
    d = [rnd(7, h, 128).to(dtype) for h in (h_qk, h_qk, h_v)]
    cu = torch.tensor([0, 2, 7], dtype=torch.int32, device="cuda")
    ref = F.Conv(x, taps, h_qk, lens=lens)
    out = gdn.gdn_conv_fwd(x.cuda(), taps.cuda(), h_qk, None, None, cu)
    for got, want, bound in zip(out, ref.out, ref.bounds):
        F.check("out", got, want, bound, dtype)
    got = gdn.gdn_conv_bwd(x.cuda(), taps.cuda(), h_qk, *[t.cuda() for t in d], None, None, None, cu)
    want, bound = ref.backward(*d)
    F.check("dx", got[0], want[0], bound[0], dtype)
    F.check("dw", got[1], want[1], bound[1])


def test_infinite_gradients_in_sums():
    """An infinity among what is summed is the sum, with its sign, as in one plain sum."""
    g = torch.Generator().manual_seed(7)
    q, d = torch.randn(40, 3, 128, generator=g), torch.randn(40, 3, 128, generator=g)
    d[17, 1, 3] = -torch.inf
    w = torch.ones(128)
    pos = F.places([40])[1]
    dw = gdn.gdn_qk_rope_bwd(q.cuda(), None, d.cuda(), None, gdn.gdn_rope_table(128), norm="rms", q_weight=w.cuda())[2].cpu()
    n, ang = F.normed(q, "rms", None, 1e-6)[17, 1], 17 * F.frequencies(128)[3]
    assert dw.isinf().nonzero().flatten().tolist() == [3, 67] and not dw.isnan().any()
    # du of the pair: cos (-inf) and sin inf
    assert (dw[3] < 0) == (torch.cos(ang) * n[3] > 0) and (dw[67] > 0) == (torch.sin(ang) * n[67] > 0) and pos[17] == 17
    x, taps, bias = torch.randn(40, 512, generator=g), torch.randn(512, 4, generator=g), torch.zeros(512)
    dv = torch.randn(40, 2, 128, generator=g)
    dv[9, 1, 5] = torch.inf
    zero = torch.zeros(40, 1, 128).cuda()
    db = gdn.gdn_conv_bwd(x.cuda(), taps.cuda(), 1, zero, zero, dv.cuda(), bias.cuda(), activation="none")[2].cpu()
    assert db.isinf().nonzero().flatten().tolist() == [389] and db[389] > 0 and not db.isnan().any()


# ---- more than 2^31 elements: the last tokens against a call on them alone, bit for bit ----
FAR, LAST = 2 ** 31 // 512 + 5000, 300


def far(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g, dtype=BF16)


def test_rope_past_32_bits():
    g = torch.Generator(device="cuda").manual_seed(1)
    q, w, rope = far(g, FAR, 4, 128), torch.rand(128, device="cuda", generator=g) + 0.5, gdn.gdn_rope_table(128)
    pos = torch.arange(FAR, dtype=torch.int32, device="cuda")
    out = gdn.gdn_qk_rope(q, None, rope, norm="rms", q_weight=w)[0]
    assert torch.equal(out[-LAST:], gdn.gdn_qk_rope(q[-LAST:], None, rope, pos[-LAST:], norm="rms", q_weight=w)[0])
    dx, _, dw, _ = gdn.gdn_qk_rope_bwd(q, None, out, None, rope, norm="rms", q_weight=w)
    small = gdn.gdn_qk_rope_bwd(q[-LAST:], None, out[-LAST:], None, rope, pos[-LAST:], norm="rms", q_weight=w)
    assert torch.equal(dx[-LAST:], small[0])
    # d_out is the output: du = x r w up to a bf16's rounding (2^-8) of what is turned, so dw = w sum (x r)^2,
    # whose sum over a head is 128; the roundings add up at random and are far below their bound
    want = (w.double() * FAR * 4 * 128).sum() / 128
    assert (dw.double().sum() / want - 1).abs() < 2.0 ** -8
    del q, out, dx
    torch.cuda.empty_cache()


def test_conv_past_32_bits():
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = far(g, FAR, 512), torch.randn(512, 4, device="cuda", generator=g) / 2
    outs = gdn.gdn_conv_fwd(x, w, 1)
    state = x[-LAST - 3:-LAST][None].contiguous()
    small = gdn.gdn_conv_fwd(x[-LAST:], w, 1, None, state)
    for a, b in zip(outs[:3], small):
        assert torch.equal(a[-LAST:], b)
    assert torch.equal(outs[3], small[3])
    dx, dw, _, _ = gdn.gdn_conv_bwd(x, w, 1, *outs[:3])
    # the first 3 of the last tokens get gradients from no earlier token: all of them have theirs whole
    assert torch.equal(dx[-LAST:], gdn.gdn_conv_bwd(x[-LAST:], w, 1, *[t[-LAST:].contiguous() for t in outs[:3]], None, state)[0])
    assert dw.isfinite().all() and (dw.abs().sum(1) > 0).all()
    del x, outs, dx
    torch.cuda.empty_cache()


def test_append_past_32_bits():
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens = FAR // 64 * 64 + 37
    qkv = far(g, tokens, 6, 128)        # 4 heads of queries, one of keys, one of values
    q, k, v = qkv.split([4, 1, 1], dim=1)
    pages = -(-tokens // 64)
    cache, rope = gdn.KVCache.empty(pages, 1), gdn.gdn_rope_table(128)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([tokens], dtype=torch.int32, device="cuda")
    out = gdn.gdn_kv_append_rope(cache, k, v, lens, table, rope=rope, norm="rms", q=q)
    n = 37 + 64
    few = gdn.KVCache.empty(pages, 1)
    small = gdn.gdn_kv_append_rope(few, k[-n:], v[-n:], lens, table, rope=rope, norm="rms", q=q[-n:])
    assert torch.equal(out[-n:], small)
    for name in ("k", "v"):
        assert torch.equal(getattr(cache, name)[-2:].view(torch.uint8)[..., :37, :], getattr(few, name)[-2:].view(torch.uint8)[..., :37, :])
        assert torch.equal(getattr(cache, name + "_scale")[-2:], getattr(few, name + "_scale")[-2:])
    assert gdn.gdn_get_device_status(cache.status) == (0, 0)
    del qkv, out
    torch.cuda.empty_cache()
