"""Host side of the 8-bit key/value cache: planning, argument checks, and the
plain 64-bit forms' own pins (no GPU)."""
from __future__ import annotations

import ctypes
import math
import os

import pytest
import torch

from tests import kv_util as U


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_linear_fwd_gb300 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from gated_deltanet_linear_fwd_gb300 import build
        build.build()
    return _lib.load()


OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 6


def dims(**kw):
    from gated_deltanet_linear_fwd_gb300 import _lib as L
    d = dict(n_seqs=2, T=4, h_q=4, max_pages=3, causal=1, window=0, scale=0.0, dtype=0, q_stride=0, k_stride=0,
             v_stride=0, out_stride=0)
    d.update(kw)
    return L.gdn_kv_dims(*d.values())


def cache(**kw):
    from gated_deltanet_linear_fwd_gb300 import _lib as L
    d = dict(k=4096, v=8192, k_scale=64, v_scale=128, status=256, n_pages=5, h_kv=2, d=128)
    d.update(kw)
    return L.gdn_kv_cache(*d.values())


def plan(lib, h_kv=2, max_q=2, max_kv=0, sms=152, **kw):
    from gated_deltanet_linear_fwd_gb300 import _lib as L
    p = L.gdn_kv_plan_t()
    st = lib.gdn_kv_attn_plan(dims(**kw), h_kv, max_q, max_kv, sms, p)
    return st, p


BAD_COMMON = [
    (dict(n_seqs=0), {}, INVALID), (dict(T=-1), {}, INVALID), (dict(T=3), {}, INVALID), (dict(max_pages=0), {}, INVALID),
    (dict(dtype=2), {}, UNSUPPORTED), ({}, dict(d=64), UNSUPPORTED), ({}, dict(k=0), INVALID), ({}, dict(v_scale=0), INVALID),
    ({}, dict(status=0), INVALID), ({}, dict(k=4097), MISALIGNED), ({}, dict(v=8200), MISALIGNED),
    ({}, dict(k_scale=66), MISALIGNED), ({}, dict(n_pages=0), INVALID), ({}, dict(h_kv=0), INVALID),
    ({}, dict(n_pages=1 << 30, h_kv=4), INVALID)]


@pytest.mark.parametrize("d,c,expect", BAD_COMMON + [
    (dict(k_stride=255), {}, INVALID), (dict(v_stride=260), {}, MISALIGNED), (dict(k_stride=-256), {}, INVALID)])
def test_append_and_read_refuse(lib, d, c, expect):
    for fn in (lib.gdn_kv_append, lib.gdn_kv_read):
        assert fn(512, 1024, 64, 64, None, cache(**c), dims(**d), None) == expect


def test_append_refuses_pointers(lib):
    good = (512, 1024, 64, 64, None)
    for i, bad, expect in ((0, None, INVALID), (1, None, INVALID), (2, None, INVALID), (3, None, INVALID),
                           (0, 520, MISALIGNED), (1, 1025, MISALIGNED), (2, 65, MISALIGNED), (4, 2, MISALIGNED)):
        a = list(good)
        a[i] = bad
        assert lib.gdn_kv_append(*a, cache(), dims(), None) == expect
    assert lib.gdn_kv_append(*good, None, dims(), None) == INVALID
    assert lib.gdn_kv_append(*good, cache(), None, None) == INVALID
    assert lib.gdn_kv_append(*good, cache(), dims(T=0), None) == OK  # nothing to do


@pytest.mark.parametrize("kw,expect", [
    (dict(causal=2), UNSUPPORTED), (dict(window=-1), INVALID), (dict(h_q=1), INVALID), (dict(h_kv=0), INVALID),
    (dict(dtype=7), UNSUPPORTED), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID),
    (dict(n_seqs=0), INVALID), (dict(max_pages=0), INVALID), (dict(T=1 << 30, h_q=64, h_kv=1), INVALID)])
def test_plan_refuses(lib, kw, expect):
    st, _ = plan(lib, **kw)
    assert st == expect


def test_attn_refuses(lib):
    st, p = plan(lib, max_kv=100000, max_pages=2000)
    assert st == OK and p.workspace_bytes > 0 and p.n_ctas > 0
    call = lambda d, c=None, q=512, out=1024, lse=None, pl=p, ws=4096, size=None: lib.gdn_kv_attn(  # noqa: E731
        q, 64, 64, None, c or cache(), out, lse, d, pl, ws, p.workspace_bytes if size is None else size, None)
    good = dict(max_pages=2000)
    assert call(dims(**good), size=p.workspace_bytes - 1) == WORKSPACE
    assert call(dims(**good), ws=None) == WORKSPACE
    assert call(dims(**good), ws=4100) == MISALIGNED
    assert call(dims(**good), q=None) == INVALID
    assert call(dims(**good), out=1026) == MISALIGNED
    assert call(dims(**good), lse=3) == MISALIGNED
    assert call(dims(**good), pl=None) == INVALID
    assert call(dims(T=2, **good)) == INVALID        # another T than the plan's
    assert call(dims(dtype=1, **good)) == INVALID    # another type
    assert call(dims(h_q=8, **good)) == INVALID
    assert call(dims(**good), cache(h_kv=1)) == INVALID
    assert call(dims(q_stride=511, **good)) == INVALID
    assert call(dims(out_stride=516, **good)) == MISALIGNED
    assert call(dims(causal=3, **good)) == UNSUPPORTED
    assert call(dims(window=-5, **good)) == INVALID
    st, one = plan(lib, max_q=1, max_kv=100000, max_pages=2000)
    assert call(dims(**good), pl=one) == INVALID     # two tokens a sequence, a plan for one
    for d, c, expect in BAD_COMMON:
        assert call(dims(**{**good, **d}), cache(**c)) == expect


@pytest.mark.parametrize("T,n,h_q,h_kv,max_q,max_kv", [(1, 1, 8, 2, 1, 333), (256, 256, 8, 2, 1, 32768), (4, 4, 16, 2, 1, 262144),
                                                       (160, 32, 32, 8, 5, 8192), (2048, 1, 16, 2, 2048, 67584), (7, 3, 3, 2, 5, 100)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_plan_covers(lib, T, n, h_q, h_kv, max_q, max_kv, dtype):
    """Row tiles cover the rows, the workspace holds two parts a CTA, and its sections do not overlap."""
    st, p = plan(lib, h_kv=h_kv, max_q=max_q, max_kv=max_kv, T=T, n_seqs=n, h_q=h_q, max_pages=-(-max_kv // 64), dtype=dtype)
    assert st == OK
    group = -(-h_q // h_kv)
    assert p.rows * p.max_row_tiles >= max_q * group > p.rows * (p.max_row_tiles - 1)
    if p.n_ctas:
        assert p.off_ml - p.off_desc >= 16 * p.n_ctas
        assert p.off_o - p.off_ml >= 2 * p.n_ctas * p.rows * 8
        assert p.workspace_bytes - p.off_o >= 2 * p.n_ctas * p.rows * 512


def test_python_refuses():
    import gated_deltanet_linear_fwd_gb300 as gdn
    codes = torch.zeros(3, 2, 64, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(3, 2)
    with pytest.raises(ValueError):
        gdn.KVCache(codes.view(torch.uint8), codes, s, s)
    with pytest.raises(ValueError):
        gdn.KVCache(codes, codes, s[:, :1], s)
    with pytest.raises(ValueError):
        gdn.KVCache(codes[:, :, :32], codes, s, s)
    c = gdn.KVCache(codes, codes, s, s)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        gdn.gdn_kv_append(c, torch.zeros(1, 2, 128), torch.zeros(1, 2, 128), i32(1), i32(0).view(1, 1))  # not on a GPU
    with pytest.raises(ValueError):
        gdn.gdn_kv_read(c, i32(1).long(), i32(0).view(1, 1), T=1)


# ---------------------------------------------------------------- pins of the plain forms
def test_e4m3_matches_the_type():
    x = torch.cat([torch.randn(4000) * torch.exp(3 * torch.randn(4000)), torch.arange(-2048, 2048) * 2.0 ** -10]).double()
    assert torch.equal(U.e4m3(x), x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double())


def test_scale_rule():
    for a, e in ((448.0, 0), (448.1, 1), (1.75, -8), (1.7501, -7), (3.5, -7), (0.0, -40), (1e-30, -40), (1e30, 40)):
        assert U.scale_exp(a) == e


def test_reference_attention_is_softmax():
    """Against torch's own softmax on a dense causal case, and the mean of the values for zero queries."""
    b = U.Batch([30], [100], 1, seed=1)
    b.fill()
    q = b.randn(30, 1, 128)
    o, z, *_ = U.attn_ref(b, q)
    K, V = b.tokens("k", 0)[:, 0], b.tokens("v", 0)[:, 0]
    s = q[:, 0].double() @ K.T / math.sqrt(128) + torch.full((30, 100), -math.inf, dtype=torch.float64).triu(71)
    assert torch.allclose(o[:, 0], s.softmax(-1) @ V, atol=1e-12)
    o, z, *_ = U.attn_ref(b, 0 * q, causal=False)
    assert torch.allclose(o[3, 0], V.mean(0), atol=1e-12) and abs(float(z[0, 0]) - math.log(100)) < 1e-12
    o, z, *_ = U.attn_ref(b, q, window=1)
    assert torch.allclose(o[7, 0], V[77], atol=1e-12)
