"""Host side of what stands between the projections and the mixers: the table
of frequencies, argument checks, and pins of the plain 64-bit forms (no GPU)."""
from __future__ import annotations

import ctypes
import math
import os
from decimal import Decimal, getcontext

import pytest
import torch

from tests import front_util as F

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 6


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_linear_fwd_gb300 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from gated_deltanet_linear_fwd_gb300 import build
        build.build()
    return _lib.load()


# ---------------------------------------------------------------- the table
def opts(**kw):
    from gated_deltanet_linear_fwd_gb300 import _lib as L
    d = dict(rot=128, scaling=0, base=10000.0, factor=1.0, original_len=0.0, low=1.0, high=32.0)
    d.update(kw)
    return L.gdn_rope_opts(*d.values())


def table(lib, **kw):
    o = opts(**kw)
    t = (ctypes.c_uint64 * (o.rot // 2))()
    assert lib.gdn_rope_table(o, t) == OK
    return [int(x) for x in t]


@pytest.mark.parametrize("kw", [dict(), dict(rot=64), dict(rot=8, base=500000.0), dict(rot=96, base=1.5), dict(scaling=1, factor=3.0),
                                dict(scaling=2, factor=8.0, rot=32), dict(scaling=3, factor=8.0, original_len=4096.0),
                                dict(scaling=3, factor=40.0, original_len=8192.0, low=1.0, high=4.0)])
def test_table(lib, kw):
    """The phase of far positions against the angle in 60 digits.  A frequency in
    fp64 is off by a few of 2^-53 of itself (the power, the products, 2 pi), so a
    position p by 8 p f 2^-53 radians, plus half a step of the table a token."""
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    t = table(lib, **kw)
    o = opts(**kw)
    for i in range(0, o.rot // 2, 3):
        base = Decimal(o.base)
        if o.scaling == 2:
            base *= Decimal(o.factor) ** (Decimal(o.rot) / Decimal(o.rot - 2))
        f = base ** (Decimal(-2 * i) / Decimal(o.rot))
        if o.scaling == 1:
            f /= Decimal(o.factor)
        if o.scaling == 3:
            r = Decimal(o.original_len) * f / (2 * pi)
            keep = min(Decimal(1), max(Decimal(0), (r - Decimal(o.low)) / (Decimal(o.high) - Decimal(o.low))))
            f = f * keep + f / Decimal(o.factor) * (1 - keep)
        for p in (1, 4097, 262143, 2 ** 31 - 1):
            phase = Decimal(p * t[i] % 2 ** 64) / Decimal(2 ** 64)
            want = (Decimal(p) * f / (2 * pi)) % 1
            off = abs(phase - want)
            off = min(off, 1 - off)
            assert off <= Decimal(p) * (8 * f / (2 * pi) * Decimal(2) ** -53 + Decimal(2) ** -65), (i, p)


@pytest.mark.parametrize("kw,expect", [
    (dict(rot=0), UNSUPPORTED), (dict(rot=130), UNSUPPORTED), (dict(rot=12), UNSUPPORTED), (dict(rot=-8), UNSUPPORTED),
    (dict(scaling=4), UNSUPPORTED), (dict(scaling=-1), UNSUPPORTED), (dict(base=1.0), INVALID), (dict(base=math.nan), INVALID),
    (dict(base=math.inf), INVALID), (dict(scaling=1, factor=0.5), INVALID), (dict(scaling=2, factor=math.inf), INVALID),
    (dict(scaling=3, factor=2.0), INVALID), (dict(scaling=3, factor=2.0, original_len=4096.0, low=4.0, high=4.0), INVALID),
    (dict(scaling=3, factor=2.0, original_len=math.nan), INVALID)])
def test_table_refuses(lib, kw, expect):
    t = (ctypes.c_uint64 * 80)()
    assert lib.gdn_rope_table(opts(**kw), t) == expect
    assert lib.gdn_rope_table(None, t) == INVALID and lib.gdn_rope_table(opts(), None) == INVALID


# ---------------------------------------------------------------- refusals of the C entries (nothing is followed)
def rope(**kw):
    from gated_deltanet_linear_fwd_gb300 import _lib as L
    d = dict(turns=4096, rot=128, layout=0, magnitude=0.0)
    d.update(kw)
    return L.gdn_rope(*d.values())


def rope_dims(**kw):
    from gated_deltanet_linear_fwd_gb300 import _lib as L
    d = dict(n_seqs=2, T=4, h_q=4, h_k=2, norm=1, eps=0.0, dtype=0, q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0,
             dq_stride=0, dk_stride=0)
    d.update(kw)
    return L.gdn_rope_dims(*d.values())


ROPE_BAD = [
    (dict(n_seqs=0), {}, INVALID), (dict(T=-1), {}, INVALID), (dict(T=3), {}, INVALID), (dict(h_q=-1), {}, INVALID),
    (dict(h_q=0, h_k=0), {}, INVALID), (dict(h_k=70000), {}, INVALID), (dict(norm=3), {}, UNSUPPORTED), (dict(norm=-1), {}, UNSUPPORTED),
    (dict(dtype=2), {}, UNSUPPORTED), (dict(eps=-1.0), {}, INVALID), (dict(eps=1e-30), {}, INVALID), (dict(eps=math.nan), {}, INVALID),
    (dict(eps=math.inf), {}, INVALID), (dict(q_stride=511), {}, INVALID), (dict(q_stride=516), {}, MISALIGNED),
    (dict(k_out_stride=-256), {}, INVALID), (dict(dk_stride=8), {}, INVALID), (dict(norm=0), {}, INVALID),
    ({}, dict(rot=4), UNSUPPORTED), ({}, dict(rot=136), UNSUPPORTED), ({}, dict(layout=2), UNSUPPORTED), ({}, dict(turns=None), INVALID),
    ({}, dict(turns=4104), MISALIGNED), ({}, dict(magnitude=math.nan), INVALID), ({}, dict(magnitude=-1.0), INVALID)]


@pytest.mark.parametrize("d,r,expect", ROPE_BAD)
def test_rope_refuses(lib, d, r, expect):
    assert lib.gdn_qk_rope(512, 1024, 64, 64, None, None, rope(**r), 2048, 4096, rope_dims(**d), None) == expect
    assert lib.gdn_qk_rope_bwd(512, 1024, 64, 64, None, None, rope(**r), 2048, 4096, 512, 512, 64, 64, rope_dims(**d), 256, 1 << 30,
                               None) == expect


def test_rope_refuses_pointers(lib):
    good = [512, 1024, 64, 64, None, None, rope(), 2048, 4096, rope_dims(), None]
    for i, bad, expect in ((0, None, INVALID), (1, None, INVALID), (7, None, INVALID), (8, None, INVALID), (9, None, INVALID),
                           (0, 520, MISALIGNED), (2, 68, MISALIGNED), (3, 72, MISALIGNED), (4, 6, MISALIGNED), (5, 2, MISALIGNED),
                           (7, 2056, MISALIGNED)):
        a = list(good)
        a[i] = bad
        assert lib.gdn_qk_rope(*a) == expect, i
    empty = list(good)
    empty[9] = rope_dims(T=0)
    assert lib.gdn_qk_rope(*empty) == OK
    n = ctypes.c_size_t(0)
    assert lib.gdn_qk_rope_bwd_workspace_bytes(n) == OK and n.value >= 128 * 4 and n.value % (128 * 4) == 0
    assert lib.gdn_qk_rope_bwd_workspace_bytes(None) == INVALID
    good = [512, 1024, 64, 64, None, None, rope(), 2048, 4096, 512, 512, 64, 64, rope_dims(), 256, n.value, None]
    for i, bad, expect in ((9, None, INVALID), (10, None, INVALID), (14, None, WORKSPACE), (15, n.value - 1, WORKSPACE),
                           (14, 264, MISALIGNED), (11, 68, MISALIGNED), (2, None, INVALID), (3, None, INVALID), (7, None, INVALID)):
        a = list(good)
        a[i] = bad
        assert lib.gdn_qk_rope_bwd(*a) == expect, i


def test_in_place_needs_the_same_rows(lib):
    """An output at its input's address with another token stride would overwrite rows that are yet to be read."""
    for kw in (dict(q_out_stride=1024), dict(q_stride=1024)):
        assert lib.gdn_qk_rope(512, 1024, 64, 64, None, None, rope(), 512, 4096, rope_dims(**kw), None) == INVALID
    assert lib.gdn_qk_rope(512, 1024, 64, 64, None, None, rope(), 2048, 1024, rope_dims(k_out_stride=2048), None) == INVALID
    for kw in (dict(q_out_stride=1024), dict(dq_stride=1024)):
        assert lib.gdn_qk_rope_bwd(512, 1024, 64, 64, None, None, rope(), 2048, 4096, 2048, 512, 64, 64, rope_dims(**kw), 256, 1 << 30,
                                   None) == INVALID
    assert lib.gdn_qk_rope_bwd(512, 1024, 64, 64, None, None, rope(), 2048, 4096, 512, 4096, 64, 64, rope_dims(dk_stride=2048), 256,
                               1 << 30, None) == INVALID
    for kw in (dict(q_stride=1024), dict(out_stride=1024)):
        assert lib.gdn_kv_append_rope(512, 1024, 64, 512, 64, 512, 64, 64, None, cache(), kv_dims(**kw), rope(), 1, 0.0, None) == INVALID


def kv_dims(**kw):
    from gated_deltanet_linear_fwd_gb300 import _lib as L
    d = dict(n_seqs=2, T=4, h_q=4, max_pages=3, causal=1, window=0, scale=0.0, dtype=0, q_stride=0, k_stride=0, v_stride=0,
             out_stride=0)
    d.update(kw)
    return L.gdn_kv_dims(*d.values())


def cache(**kw):
    from gated_deltanet_linear_fwd_gb300 import _lib as L
    d = dict(k=4096, v=8192, k_scale=64, v_scale=128, status=256, n_pages=5, h_kv=2, d=128)
    d.update(kw)
    return L.gdn_kv_cache(*d.values())


@pytest.mark.parametrize("at,bad,expect", [
    (0, None, INVALID), (1, None, INVALID), (6, None, INVALID), (7, None, INVALID), (9, None, INVALID), (10, None, INVALID),
    (0, 520, MISALIGNED), (2, 68, MISALIGNED), (3, 520, MISALIGNED), (4, 66, MISALIGNED), (5, 2056, MISALIGNED), (3, None, INVALID),
    (5, None, INVALID), (8, 2, MISALIGNED), (12, 5, UNSUPPORTED), (13, -1.0, INVALID), (12, 0, INVALID)])
def test_append_rope_refuses(lib, at, bad, expect):
    a = [512, 1024, 64, 512, 64, 2048, 64, 64, None, cache(), kv_dims(), rope(), 1, 0.0, None]
    a[at] = bad
    assert lib.gdn_kv_append_rope(*a) == expect


@pytest.mark.parametrize("d,c,r,expect", [
    (dict(T=3), {}, {}, INVALID), (dict(dtype=2), {}, {}, UNSUPPORTED), (dict(q_stride=8), {}, {}, INVALID),
    (dict(out_stride=516), {}, {}, MISALIGNED), (dict(h_q=0), {}, {}, INVALID), (dict(k_stride=100), {}, {}, INVALID),
    ({}, dict(d=64), {}, UNSUPPORTED), ({}, dict(v=8200), {}, MISALIGNED), ({}, dict(n_pages=0), {}, INVALID),
    ({}, {}, dict(rot=20), UNSUPPORTED), ({}, {}, dict(layout=7), UNSUPPORTED), ({}, {}, dict(turns=None), INVALID)])
def test_append_rope_refuses_dims(lib, d, c, r, expect):
    a = [512, 1024, 64, 512, 64, 2048, 64, 64, None, cache(**c), kv_dims(**d), rope(**r), 1, 0.0, None]
    assert lib.gdn_kv_append_rope(*a) == expect
    a[10] = kv_dims(T=0)
    a[9], a[11] = cache(), rope()
    assert lib.gdn_kv_append_rope(*a) == OK  # nothing to do


def conv_dims(**kw):
    from gated_deltanet_linear_fwd_gb300 import _lib as L
    d = dict(n_seqs=2, T=4, h_qk=1, h_v=2, width=4, activation=1, norm=1, eps=0.0, dtype=0, x_stride=0, dx_stride=0)
    d.update(kw)
    return L.gdn_conv_dims(*d.values())


CONV_BAD = [
    (dict(n_seqs=0), INVALID), (dict(T=-1), INVALID), (dict(h_qk=0), INVALID), (dict(h_v=0), INVALID),
    (dict(h_qk=20000), INVALID), (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED), (dict(activation=2), UNSUPPORTED),
    (dict(norm=2), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=1e-25), INVALID), (dict(dtype=3), UNSUPPORTED),
    (dict(x_stride=511), INVALID), (dict(x_stride=516), MISALIGNED), (dict(dx_stride=-512), INVALID),
    (dict(T=1 << 30, n_seqs=1, h_v=100), INVALID)]


@pytest.mark.parametrize("d,expect", CONV_BAD + [(dict(T=3), INVALID)])
def test_conv_refuses(lib, d, expect):
    assert lib.gdn_conv_fwd(512, 64, 64, None, None, 1024, 2048, 4096, 8192, conv_dims(**d), None) == expect
    assert lib.gdn_conv_bwd(512, 64, 64, None, None, 1024, 2048, 4096, None, 8192, 64, 64, None, conv_dims(**d), 256, 1 << 40,
                            None) == expect


@pytest.mark.parametrize("d,expect", CONV_BAD + [(dict(T=4), INVALID)])
def test_conv_step_refuses(lib, d, expect):
    assert lib.gdn_conv_step(512, 64, 64, 8192, 1024, 2048, 4096, conv_dims(**d), None) == expect


def test_conv_refuses_pointers(lib):
    n = ctypes.c_size_t(0)
    assert lib.gdn_conv_bwd_workspace_bytes(conv_dims(), n) == OK and n.value > 0
    assert lib.gdn_conv_bwd_workspace_bytes(conv_dims(), None) == INVALID
    assert lib.gdn_conv_bwd_workspace_bytes(None, n) == INVALID
    assert lib.gdn_conv_bwd_workspace_bytes(conv_dims(width=7), n) == UNSUPPORTED
    good = [512, 64, 64, 1 << 20, None, 1024, 2048, 4096, 1 << 21, conv_dims(), None]
    for i, bad, expect in ((0, None, INVALID), (1, None, INVALID), (5, None, INVALID), (6, None, INVALID), (7, None, INVALID),
                           (9, None, INVALID), (0, 520, MISALIGNED), (1, 72, MISALIGNED), (2, 68, MISALIGNED), (3, 1028, MISALIGNED),
                           (4, 2, MISALIGNED), (8, (1 << 20) + 512, INVALID)):
        a = list(good)
        a[i] = bad
        assert lib.gdn_conv_fwd(*a) == expect, i
    good = [512, 64, 64, 1 << 20, None, 1024, 2048, 4096, 1 << 21, 8192, 64, 64, 1 << 22, conv_dims(), 256, n.value, None]
    for i, bad, expect in ((0, None, INVALID), (5, None, INVALID), (9, None, INVALID), (9, 512, INVALID), (14, None, WORKSPACE),
                           (15, n.value - 1, WORKSPACE), (14, 260, MISALIGNED), (10, 68, MISALIGNED), (12, 1 << 21, INVALID),
                           (12, (1 << 20) + 16, INVALID)):
        a = list(good)
        a[i] = bad
        assert lib.gdn_conv_bwd(*a) == expect, i
    for i, bad, expect in ((0, None, INVALID), (1, None, INVALID), (3, None, INVALID), (4, None, INVALID), (3, 8200, MISALIGNED),
                           (6, 1025, MISALIGNED)):
        a = [512, 64, 64, 8192, 1024, 2048, 4096, conv_dims(T=2), None]
        a[i] = bad
        assert lib.gdn_conv_step(*a) == expect, i


@pytest.mark.parametrize("T", [0, 1, 63, 64, 65, 4097, 32768, 348160])
@pytest.mark.parametrize("h_qk,h_v,width", [(1, 1, 2), (2, 8, 4), (16, 16, 3)])
def test_conv_workspace_covers(lib, T, h_qk, h_v, width):
    """A row of W + 1 sums a channel for each group of 8 runs of 8 to 192 tokens, with and without the norm."""
    sizes = []
    for norm in (0, 1):
        n = ctypes.c_size_t(0)
        assert lib.gdn_conv_bwd_workspace_bytes(conv_dims(T=T, n_seqs=1, h_qk=h_qk, h_v=h_v, width=width, norm=norm), n) == OK
        sizes.append(n.value)
    row = (width + 1) * (2 * h_qk + h_v) * 128 * 4
    assert sizes[0] == sizes[1] and -(-T // (8 * 192)) * row <= sizes[0] <= -(-T // 64) * row


def test_python_refuses():
    import gated_deltanet_linear_fwd_gb300 as gdn
    q, k = torch.zeros(3, 2, 128), torch.zeros(3, 1, 128)
    for call in (lambda: gdn.gdn_qk_rope(q, k),                                       # not on a GPU
                 lambda: gdn.gdn_qk_rope(None, None),
                 lambda: gdn.gdn_qk_rope(q, torch.zeros(4, 1, 128)),
                 lambda: gdn.gdn_qk_rope(torch.zeros(3, 2, 64), None),
                 lambda: gdn.gdn_qk_rope_bwd(q, k, q, None),
                 lambda: gdn.gdn_rope_table(layout="both", device="cpu"),
                 lambda: gdn.gdn_rope_table(scaling="twice", device="cpu"),
                 lambda: gdn.Rope(torch.zeros(64)),
                 lambda: gdn.gdn_conv_fwd(torch.zeros(3, 512), torch.zeros(512, 4), 1),   # not on a GPU
                 lambda: gdn.gdn_conv_fwd(torch.zeros(512), torch.zeros(512, 4), 1),
                 lambda: gdn.gdn_conv_step(torch.zeros(1, 3, 512), torch.zeros(3, 3, 512), torch.zeros(512, 4), 1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(gdn.api.L.GDNError):
        gdn.gdn_rope_table(20, device="cpu")
    with pytest.raises(gdn.api.L.GDNError):
        gdn.gdn_conv_bwd_workspace_bytes(10, 1, 1, width=9)


def test_token_strides():
    """Views whose tokens are whole and evenly spaced give their stride, others are refused."""
    from gated_deltanet_linear_fwd_gb300.api import _spacing
    x = torch.zeros(6, 5, 128)
    assert _spacing("x", x[:, 1:3], 2) == 640 and _spacing("x", x[::2], 2) == 1280
    assert _spacing("x", x[:1, 1:3], 2) == 0
    b = torch.zeros(2, 3, 5, 128)
    assert _spacing("b", b[:, :, 2:], 2) == 640 and _spacing("b", b[:, ::3], 2) == 1920 and _spacing("b", b[:1, :, :1], 2) == 640
    c = torch.zeros(4, 640)
    assert _spacing("c", c[:, :512], 1) == 640 and _spacing("c", c.view(2, 2, 640)[:, :, :512], 1) == 640
    for bad, inner in ((x[:, ::2], 2), (x[:, :, ::2], 2), (x[:1, :2].expand(6, 2, 128), 2), (b[:, :2], 2), (c.T, 1), (c[:, ::2], 1),
                       (x.transpose(0, 1)[:, :2], 2)):
        with pytest.raises(ValueError):
            _spacing("bad", bad, inner)


# ---------------------------------------------------------------- pins of the plain forms
def test_rotation_is_by_relative_position():
    """Scores of rotated queries and keys depend on the distance alone, and the length stays."""
    g = torch.Generator().manual_seed(0)
    q, k = torch.randn(1, 1, 128, generator=g).double(), torch.randn(1, 1, 128, generator=g).double()
    f = F.frequencies(64)
    for layout in ("half", "interleaved"):
        score = lambda a, b: float((F.turn(q, torch.tensor([a]), f, layout) * F.turn(k, torch.tensor([b]), f, layout)).sum())  # noqa: E731
        assert abs(score(5, 3) - score(1005, 1003)) < 1e-9 and abs(score(5, 3) - score(5, 4)) > 1e-4
        assert torch.allclose(F.turn(q, torch.tensor([777]), f, layout).norm(), q.norm())
        assert torch.allclose(F.turn(F.turn(q, torch.tensor([9]), f, layout), torch.tensor([9]), f, layout, sign=-1.0), q)


@pytest.mark.parametrize("norm", ["none", "rms", "unit"])
@pytest.mark.parametrize("layout,rot", [("half", 128), ("interleaved", 16)])
def test_rope_gradient_against_differences(norm, layout, rot):
    g = torch.Generator().manual_seed(1)
    x, dy, d = (torch.randn(3, 2, 128, generator=g).double() for _ in range(3))
    w, dw_dir = torch.randn(128, generator=g).double(), torch.randn(128, generator=g).double()
    f, pos = F.frequencies(rot), torch.tensor([0, 5, 1000])
    if norm == "none":
        w = None
    loss = lambda x, w: float((F.rope_ref(x, pos, f, layout, 1.3, norm, w)[0] * dy).sum())  # noqa: E731
    dx, dw, *_ = F.rope_bwd_ref(x, dy, pos, f, layout, 1.3, norm, w)
    h = 1e-5
    assert abs((loss(x + h * d, w) - loss(x - h * d, w)) / (2 * h) - float((dx * d).sum())) < 1e-6
    if w is not None:
        assert abs((loss(x, w + h * dw_dir) - loss(x, w - h * dw_dir)) / (2 * h) - float((dw * dw_dir).sum())) < 1e-6


@pytest.mark.parametrize("W,silu,norm", [(2, True, True), (3, False, True), (4, True, False), (4, True, True)])
def test_conv_gradient_against_differences(W, silu, norm):
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g).double()  # noqa: E731
    lens = [1, 0, 6, 2]
    T, C, h = sum(lens), 3 * 128, 1e-5
    x, w, b, s = rnd(T, C), rnd(C, W), rnd(C), rnd(len(lens), W - 1, C)
    dq, dk, dv, df = rnd(T, 1, 128), rnd(T, 1, 128), rnd(T, 1, 128), rnd(len(lens), W - 1, C)

    def loss(x, w, b, s):
        c = F.Conv(x, w, 1, b, s, lens, silu, norm)
        return float(sum((o * d).sum() for o, d in zip(c.out, (dq, dk, dv))) + (c.last * df).sum())

    grads, _ = F.Conv(x, w, 1, b, s, lens, silu, norm).backward(dq, dk, dv, df)
    args = [x, w, b, s]
    for i, grad in enumerate(grads):
        d = rnd(*args[i].shape)
        up, down = ([a + sgn * h * d if j == i else a for j, a in enumerate(args)] for sgn in (1, -1))
        assert abs((loss(*up) - loss(*down)) / (2 * h) - float((grad * d).sum())) < 1e-5 * max(1.0, float((grad * d).abs().sum()) ** 0.5), i


def test_conv_is_torch_conv():
    """Against torch's own convolution, one sequence, no state."""
    g = torch.Generator().manual_seed(3)
    x, w, b = torch.randn(20, 384, generator=g).double(), torch.randn(384, 4, generator=g).double(), torch.randn(384, generator=g).double()
    u = torch.nn.functional.conv1d(x.T[None], w[:, None], b, padding=3, groups=384)[0, :, :20].T
    c = F.Conv(x, w, 1, b, norm=False)
    assert torch.allclose(torch.cat(c.out, 1).reshape(20, 384), torch.nn.functional.silu(u))
