"""Edges of the 8-bit key/value cache's calls on the GPU."""
from __future__ import annotations

import pytest
import torch

from tests import kv_util as U
from tests.test_gpu_kv import check_attn, gdn, status, to_cache  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("offsets", [False, True])
def test_no_tokens(gdn, dtype, offsets):  # noqa: F811
    """Sequences that bring no tokens: nothing is read or written."""
    b = U.Batch([0, 0], [70, 5], 2, seed=1)
    b.fill()
    cache = to_cache(gdn, b)
    lens, table, cu = b.lens.cuda(), b.table.cuda(), b.cu.cuda() if offsets else None
    none = torch.empty(0, 2, 128, dtype=dtype, device="cuda")
    before = cache.k.view(torch.uint8).clone()
    gdn.gdn_kv_append(cache, none, none, lens, table, cu)
    k, v = gdn.gdn_kv_read(cache, lens, table, cu, T=0, dtype=dtype)
    out, lse = gdn.gdn_kv_attn(torch.empty(0, 8, 128, dtype=dtype, device="cuda"), cache, lens, table, cu)
    assert k.shape == v.shape == (0, 2, 128) and out.shape == (0, 8, 128) and lse.shape == (0, 8)
    assert torch.equal(before, cache.k.view(torch.uint8)) and status(gdn, cache) == (0, 0)


@pytest.mark.parametrize("dtype,n,window", [(BF, 5, 2 ** 31 - 1), (F32, 5, 2 ** 31 - 1), (BF, 200, 2 ** 31 - 1), (BF, 200, 2 ** 31 - 60),
                                            (F32, 200, 2 ** 31 - 60), (BF, 40, 2 ** 31 - 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_widest_windows(gdn, dtype, n, window, causal):  # noqa: F811
    """A window that bounds nothing, with tokens before position 0: the same as no window."""
    b = U.Batch([n, n], [n // 2, 0], 2, seed=n)
    b.fill()
    cache, q = to_cache(gdn, b), b.randn(b.T, 8, 128).to(dtype).cuda()
    for sms in (152, 4):  # for 200 tokens on 4 SMs the kernel for many rows
        plans = [gdn.gdn_kv_attn_plan(T=b.T, n_seqs=2, h_q=8, h_kv=2, max_q_len=n, max_kv_len=n, dtype=dtype, causal=causal,
                                      window=w, sm_count=sms) for w in (0, window)]
        assert plans[0].raw.path == plans[1].raw.path == (0 if dtype == F32 else 2 if n * 4 > 32 and sms == 4 else 1)
        want, got = (gdn.gdn_kv_attn(q, cache, b.lens.cuda(), b.table.cuda(), plan=p) for p in plans)
        assert (want[1][n // 2 + n % 2:n] > -1e30).all()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert status(gdn, cache) == (0, 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q,kv,h_q,h_kv,window", [
    ([1] * 300, [1 + 37 * i % 500 for i in range(300)], 8, 2, 0),                        # as few as can be, all alike
    ([1] * 150 + [400] + [1] * 149, [1 + 11 * i % 300 for i in range(150)] + [500] + [9] * 149, 8, 2, 0),  # one brings most
    ([0, 3, 0, 0, 40, 1] * 30, [5, 3, 0, 0, 70, 130] * 30, 6, 3, 50),                    # many bring none
    ([5] * 64, [5 + 13 * i for i in range(64)], 8, 1, 0),
    ([0] * 70 + [2000] + [0] * 70, [3] * 70 + [2100] + [64] * 70, 4, 2, 0)])            # one brings all
def test_packed_batches_without_a_bound(gdn, q, kv, h_q, h_kv, window, dtype):  # noqa: F811
    """Offsets alone, no word on how many tokens a sequence brings at most."""
    b = U.Batch(q, kv, h_kv, seed=len(q) + h_q)
    b.fill()
    check_attn(gdn, b, h_q, dtype, window=window)
    # the same under a plan for runs of items, and one for whole ones
    for sms, longest in ((3, 20000), (5000, 64)):
        p = gdn.gdn_kv_attn_plan(T=b.T, n_seqs=b.n, h_q=h_q, h_kv=h_kv, max_kv_len=longest, window=window, dtype=dtype,
                                 sm_count=sms)
        check_attn(gdn, b, h_q, dtype, window=window, plan=p)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("runs", [False, True])
def test_bad_offsets_without_a_bound(gdn, dtype, runs):  # noqa: F811
    """Offsets that go back or leave the tokens, with more entries than a block looks at in one go: recorded,
    wherever they are, and the next call is clean."""
    n = 300
    b = U.Batch([2] * n, [2 + i % 90 for i in range(n)], 2, seed=3)
    b.fill()
    cache = to_cache(gdn, b)
    q = b.randn(b.T, 8, 128).to(dtype).cuda()
    p = gdn.gdn_kv_attn_plan(T=b.T, n_seqs=n, h_q=8, h_kv=2, max_kv_len=20000 if runs else 64, dtype=dtype,
                             sm_count=3 if runs else 5000)
    assert (p.raw.n_ctas > 0) == runs
    args = (q, cache, b.lens.cuda(), b.table.cuda())
    want = gdn.gdn_kv_attn(*args, b.cu.cuda(), plan=p)
    for at, value in ((0, -1), (1, 5), (7, 0), (150, b.T + 1), (150, 2 ** 31 - 1), (150, -2 ** 31), (299, 3), (300, b.T + 1), (300, 0)):
        cu = b.cu.clone()
        cu[at] = value
        gdn.gdn_kv_attn(*args, cu.cuda(), plan=p)
        assert status(gdn, cache) == (7, 7), (at, value)
        cache.status.zero_()
    cu = torch.arange(n + 1).flip(0).to(torch.int32)
    gdn.gdn_kv_attn(*args, cu.cuda(), plan=p)
    assert status(gdn, cache) == (7, 7)
    cache.status.zero_()
    cu = b.cu.clone()
    cu[:] = b.T  # nobody brings anything
    gdn.gdn_kv_attn(*args, cu.cuda(), plan=p)
    again = gdn.gdn_kv_attn(*args, b.cu.cuda(), plan=p)
    assert status(gdn, cache) == (0, 0)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tokens_of_no_sequence(gdn, dtype):  # noqa: F811
    """Tokens before the first offset and after the last one are left alone."""
    n = 300
    b = U.Batch([2] * n, [2 + i % 90 for i in range(n)], 2, seed=3)
    b.fill()
    cache, T = to_cache(gdn, b), b.T + 77
    q = torch.full((T, 8, 128), 3.0)
    q[50:50 + b.T] = b.randn(b.T, 8, 128)
    q = q.to(dtype)
    o, z, mass, reach, top = U.attn_ref(b, q[50:50 + b.T])
    bo, bz = U.attn_bounds(o, mass, reach, top, dtype)
    out, lse = torch.full_like(q, 7).cuda(), torch.full((T, 8), 7.0, device="cuda")
    gdn.gdn_kv_attn(q.cuda(), cache, b.lens.cuda(), b.table.cuda(), b.cu.cuda() + 50, out=out, lse=lse)
    assert (out[:50] == 7).all() and (out[50 + b.T:] == 7).all() and (lse[:50] == 7).all() and (lse[50 + b.T:] == 7).all()
    assert ((out[50:50 + b.T].double().cpu() - o).abs() <= bo).all() and ((lse[50:50 + b.T].double().cpu() - z).abs() <= bz).all()
    assert status(gdn, cache) == (0, 0)


@pytest.mark.parametrize("runs", [False, True])
def test_few_entries_of_many_units(gdn, runs):  # noqa: F811
    """A page table so wide that row tiles are found by search although there are few of them."""
    n, h = 40, 64
    b = U.Batch([256] + [0] * 10 + [1] * 29, [300] + [5] * 10 + [2 + 7 * i for i in range(29)], h, seed=1)
    b.fill()
    cache, q = to_cache(gdn, b), b.randn(b.T, h, 128)
    table = torch.zeros(n, 1 << 20, dtype=torch.int32, device="cuda")
    table[:, :b.max_pages] = b.table.cuda()
    p = gdn.gdn_kv_attn_plan(T=b.T, n_seqs=n, h_q=h, h_kv=h, max_q_len=256, max_kv_len=20000 if runs else 64, max_pages=1 << 20,
                             dtype=F32, sm_count=152 if runs else 100000)
    assert p.raw.max_row_tiles * n == 80 and (p.raw.n_ctas > 0) == runs
    out, lse = gdn.gdn_kv_attn(q.cuda(), cache, b.lens.cuda(), table, b.cu.cuda(), plan=p)
    o, z, mass, reach, top = U.attn_ref(b, q)
    bo, bz = U.attn_bounds(o, mass, reach, top, F32)
    assert ((out.double().cpu() - o).abs() <= bo).all() and ((lse.double().cpu() - z).abs() <= bz).all()
    cu = b.cu.clone()
    cu[20] = 0
    gdn.gdn_kv_attn(q.cuda(), cache, b.lens.cuda(), table, cu.cuda(), plan=p)
    assert status(gdn, cache) == (7, 7)
