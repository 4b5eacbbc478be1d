"""Refusals and edges of the 8-bit key/value cache's host side (no GPU)."""
from __future__ import annotations

import os
import re

import pytest
import torch

from tests.test_kv_host import INVALID, OK, WORKSPACE, cache, dims, lib, plan  # noqa: F401

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_fwd_gb300", "csrc")


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("max_kv", [0, 64, 100000])
def test_no_tokens(lib, dtype, max_kv):  # noqa: F811
    """A call without tokens plans, and does nothing."""
    st, p = plan(lib, max_q=0, max_kv=max_kv, T=0, max_pages=2000, dtype=dtype)
    assert st == OK and p.rows >= 8 and p.max_row_tiles == 1
    assert lib.gdn_kv_attn(None, 64, 64, None, cache(), None, None, dims(T=0, max_pages=2000, dtype=dtype), p, 4096,
                           p.workspace_bytes, None) == OK


# ---------------------------------------------------------------- the binding, with a library that only takes note of calls
class OnGpu(torch.Tensor):
    """A host tensor that says it lies on GPU 0."""
    is_cuda = True

    def get_device(self):
        return 0


class Calls:
    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        def call(*args):
            self.made.append((name, args))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    from gated_deltanet_linear_fwd_gb300 import _lib, api
    c = Calls()
    monkeypatch.setattr(_lib, "load", lambda: c)
    monkeypatch.setattr(api, "_raw_stream", lambda stream, t: 0)
    return c


def gpu(t):
    return t.as_subclass(OnGpu)


def batch(n=2, each=32, h_q=8, h_kv=2):
    """(cache, q, k, lens, table, offsets) as a user would have them on the GPU."""
    import gated_deltanet_linear_fwd_gb300 as gdn
    codes = lambda: gpu(torch.zeros(4, h_kv, 64, 128, dtype=torch.uint8).view(torch.float8_e4m3fn))  # noqa: E731
    c = gdn.KVCache(codes(), codes(), gpu(torch.ones(4, h_kv)), gpu(torch.ones(4, h_kv)))
    i32 = lambda *x: gpu(torch.tensor(x, dtype=torch.int32))  # noqa: E731
    T = n * each
    return (c, gpu(torch.zeros(T, h_q, 128, dtype=torch.bfloat16)), gpu(torch.zeros(T, h_kv, 128, dtype=torch.bfloat16)),
            i32(*[each] * n), i32(*range(2 * n)).view(n, 2), i32(*range(0, T + 1, each)))


def test_accepted(calls):
    import gated_deltanet_linear_fwd_gb300 as gdn
    c, q, k, lens, table, cu = batch()
    gdn.gdn_kv_append(c, k, k, lens, table, cu)
    gdn.gdn_kv_read(c, lens, table, cu, k_out=k, v_out=k)
    assert [name for name, _ in calls.made] == ["gdn_kv_append", "gdn_kv_read"]
    wide = gpu(torch.zeros(64, 12, 128, dtype=torch.bfloat16))
    gdn.gdn_kv_append(c, wide[:, 8:10], wide[:, 10:], lens, table, cu)
    dims = calls.made[-1][1][6]
    assert (dims.k_stride, dims.v_stride) == (12 * 128, 12 * 128)
    one = gpu(torch.zeros(1, 1, 128, dtype=torch.bfloat16)).expand(2, 2, 128)[:1]  # a single token has no stride
    with pytest.raises(ValueError):
        gdn.gdn_kv_append(c, one, one, lens, table)  # but its heads have


def overlapping(h):
    """[64, h, 128] views whose tokens share memory."""
    yield gpu(torch.zeros(1, h, 128, dtype=torch.bfloat16)).expand(64, h, 128)
    yield gpu(torch.zeros(64 * h * 128, dtype=torch.bfloat16)).as_strided((64, h, 128), (64, 128, 1))


@pytest.mark.parametrize("which", [0, 1])
def test_overlapping_tokens_refused(calls, which):
    """A token stride below heads * 128: 0 would read as "packed", past the end of the memory behind it."""
    import gated_deltanet_linear_fwd_gb300 as gdn
    c, q, k, lens, table, cu = batch()
    bad_k, bad_q = list(overlapping(2))[which], list(overlapping(8))[which]
    for call in (lambda: gdn.gdn_kv_append(c, bad_k, k, lens, table, cu), lambda: gdn.gdn_kv_append(c, k, bad_k, lens, table, cu),
                 lambda: gdn.gdn_kv_read(c, lens, table, cu, k_out=bad_k, v_out=k),
                 lambda: gdn.gdn_kv_read(c, lens, table, cu, k_out=k, v_out=bad_k),
                 lambda: gdn.gdn_kv_attn(bad_q, c, lens, table, cu), lambda: gdn.gdn_kv_attn(q, c, lens, table, cu, out=bad_q)):
        with pytest.raises(ValueError):
            call()
    assert not [name for name, _ in calls.made if name != "gdn_kv_attn_plan"]


def test_tensors_elsewhere_refused(calls):
    """Every tensor of a call lies on the cache's device, a GPU; a workspace is all there."""
    import gated_deltanet_linear_fwd_gb300 as gdn
    c, q, k, lens, table, cu = batch()
    host = lambda t: torch.Tensor.as_subclass(t, torch.Tensor)  # noqa: E731
    lse, ws = gpu(torch.zeros(64, 8)), gpu(torch.zeros(512, dtype=torch.uint8))
    good = dict(q=q, k=k, lens=lens, table=table, cu=cu, lse=lse, workspace=ws, out=q, k_out=k)

    def run(**kw):
        a = {**good, **kw}
        for fn in (lambda: gdn.gdn_kv_append(c, a["k"], a["k_out"], a["lens"], a["table"], a["cu"]),
                   lambda: gdn.gdn_kv_read(c, a["lens"], a["table"], a["cu"], k_out=a["k"], v_out=a["k_out"]),
                   lambda: gdn.gdn_kv_attn(a["q"], c, a["lens"], a["table"], a["cu"], out=a["out"], lse=a["lse"],
                                           workspace=a["workspace"])):
            calls.made.clear()
            try:
                fn()
                yield True
            except ValueError:
                assert not [name for name, _ in calls.made if name != "gdn_kv_attn_plan"]
                yield False

    assert list(run()) == [True] * 3
    for name, used in (("lens", (1, 1, 1)), ("table", (1, 1, 1)), ("cu", (1, 1, 1)), ("k", (1, 1, 0)), ("k_out", (1, 1, 0)),
                       ("q", (0, 0, 1)), ("out", (0, 0, 1)), ("lse", (0, 0, 1)), ("workspace", (0, 0, 1))):
        assert list(run(**{name: host(good[name])})) == [not u for u in used], name
    assert list(run(workspace=ws[:1].expand(512))) == [True, True, False]
    for i in range(4):  # a cache with one tensor on the host
        parts = [c.k, c.v, c.k_scale, c.v_scale]
        parts[i] = host(parts[i])
        with pytest.raises(ValueError):
            gdn.KVCache(*parts)
    c = gdn.KVCache(*map(host, (c.k, c.v, c.k_scale, c.v_scale)))
    assert list(run()) == [False] * 3


@pytest.mark.parametrize("name", ["gdn_kv_f32.cu", "gdn_kv_few.cu", "gdn_kv_many.cu"])
def test_waits_agree_by_warp(name):
    """Tensor-memory accesses are a whole warp's.  A bounded wait may give up in some lanes only, which no
    GPU test can bring about without a wait that runs out; so each one stands within kv_wait_warp."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    while "kv_wait_warp(" in text:
        at = text.index("kv_wait_warp(")
        end = at + len("kv_wait_warp(")
        depth = 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[end], 0)
            end += 1
        assert "kv_wait(" in text[at:end]
        text = text[:at] + text[end:]
    assert "kv_wait(" not in text


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T,n,h_q,h_kv,pages", [(64 * 2048, 64, 32, 8, 4096), (32768, 256, 8, 2, 4096), (1 << 20, 1024, 8, 2, 4096)])
def test_packed_batches_plan_without_a_bound(lib, dtype, T, n, h_q, h_kv, pages):  # noqa: F811
    """However the tokens spread over the sequences, they fill T group / rows row tiles, and one more a sequence
    that is not full: far fewer than every sequence with all the tokens."""
    st, p = plan(lib, h_kv=h_kv, max_q=0, T=T, n_seqs=n, h_q=h_q, max_pages=pages, dtype=dtype)
    assert st == OK
    assert p.max_q_len == T and p.rows * p.max_row_tiles >= T * h_q // h_kv  # one sequence may bring them all


def test_plan_still_refuses_too_many_units(lib):  # noqa: F811
    """2^31 units are not counted in 32 bits, whatever the bound says."""
    for max_q in (0, 1 << 20):
        st, _ = plan(lib, max_q=max_q, T=1 << 20, n_seqs=1, h_q=64, h_kv=64, max_pages=1 << 20)
        assert st == INVALID


@pytest.mark.parametrize("T,n,h_q,h_kv,kv,rows", [(256, 256, 8, 2, 32768, 8), (4, 4, 16, 2, 262144, 8), (160, 32, 32, 8, 8192, 24),
                                                  (90, 30, 8, 2, 4096, 16), (64, 8, 8, 2, 8192, 32)])
def test_small_batches_without_a_bound(lib, T, n, h_q, h_kv, kv, rows):  # noqa: F811
    """Generated and drafted tokens get the kernel for few rows, as with the bound."""
    for max_q in (0, T // n):
        st, p = plan(lib, h_kv=h_kv, max_q=max_q, T=T, n_seqs=n, h_q=h_q, max_pages=kv // 64)
        assert st == OK and (p.path, p.rows) == (1, rows)


def test_binding_gives_no_bound_for_offsets(calls):
    import gated_deltanet_linear_fwd_gb300 as gdn
    c, q, k, lens, table, cu = batch()
    for offsets, kw, bound in ((cu, {}, 0), (None, {}, 32), (cu, dict(max_q_len=40), 40)):
        gdn.gdn_kv_attn(q, c, lens, table, offsets, out=q, **kw)
        assert [args[2] for name, args in calls.made if name == "gdn_kv_attn_plan"][-1] == bound


def test_longest_lengths(lib):  # noqa: F811
    """A length is rounded up to a tile of 128 keys in 32 bits."""
    most = (2 ** 31 - 1 - 128) // 64
    for dtype in (0, 1):
        assert plan(lib, max_q=1, T=1, n_seqs=1, max_pages=most, dtype=dtype)[0] == OK
        for pages in (most + 1, (2 ** 31 - 1) // 64):
            assert plan(lib, max_q=1, T=1, n_seqs=1, max_pages=pages, dtype=dtype)[0] == INVALID
            st, p = plan(lib, max_q=1, T=1, n_seqs=1, max_pages=most, dtype=dtype)
            assert lib.gdn_kv_attn(512, 64, 64, None, cache(), 1024, None, dims(T=1, n_seqs=1, max_pages=pages, dtype=dtype),
                                   p, 4096, p.workspace_bytes, None) == INVALID


def test_table_wider_than_the_plans(lib):  # noqa: F811
    """The bound on units holds for the call's page table too, which may be wider than the one planned for."""
    kw = dict(T=1 << 18, n_seqs=1 << 12, h_q=64)
    st, p = plan(lib, h_kv=64, max_q=64, max_pages=1, **kw)
    assert st == OK
    assert plan(lib, h_kv=64, max_q=64, max_pages=1 << 16, **kw)[0] == INVALID
    calls = [lib.gdn_kv_attn(512, 64, 64, None, cache(h_kv=64), 1024, None, dims(max_pages=pages, **kw), p, None, 0, None)
             for pages in (1 << 16, 1 << 20)]
    assert calls == [INVALID, INVALID]
    assert p.n_ctas > 0 and lib.gdn_kv_attn(512, 64, 64, None, cache(h_kv=64), 1024, None, dims(max_pages=4, **kw), p, None, 0,
                                            None) == WORKSPACE  # accepted so far


@pytest.mark.parametrize("T,n,h_q,h_kv,max_q,max_kv,path,rows", [
    (1, 1, 8, 2, 1, 333, 1, 8), (256, 256, 8, 2, 1, 32768, 1, 8), (4, 4, 16, 2, 1, 262144, 1, 8), (160, 32, 32, 8, 5, 8192, 1, 24),
    (48, 16, 8, 2, 3, 4096, 1, 16), (64, 1, 8, 2, 64, 8192, 1, 32), (512, 1, 8, 2, 512, 512, 2, 256), (2048, 1, 16, 2, 2048, 67584, 2, 256),
    (32768, 1, 8, 2, 32768, 32768, 2, 256)])
def test_plan_chooses(lib, T, n, h_q, h_kv, max_q, max_kv, path, rows):  # noqa: F811
    """Kernel and row tile, on 152 SMs; fp32 has one of each."""
    for dtype, want in ((0, (path, rows)), (1, (0, 128))):
        st, p = plan(lib, h_kv=h_kv, max_q=max_q, max_kv=max_kv, T=T, n_seqs=n, h_q=h_q, max_pages=-(-max_kv // 64), dtype=dtype)
        assert st == OK and (p.path, p.rows) == want


@pytest.mark.parametrize("n,group,rows", [(2, 4, 8), (3, 3, 16), (1, 16, 16), (17, 1, 24), (5, 4, 24), (6, 4, 24), (5, 5, 32), (31, 1, 32), (8, 4, 32)])
@pytest.mark.parametrize("window", [0, 200])
def test_row_counts_get_their_row_tile(lib, n, group, rows, window):  # noqa: F811
    """What the GPU test of row counts runs on, whose calls give no bound."""
    st, p = plan(lib, h_kv=2, max_q=0, T=7 * n, n_seqs=7, h_q=2 * group, max_pages=94, window=window)
    assert st == OK and (p.path, p.rows) == (1, rows)
