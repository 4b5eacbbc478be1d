"""The many-rows attention kernel over the 8-bit cache, on calls whose plan is
checked to take it: items that follow one another in a CTA, and contents that
only this kernel treats in its own way."""
from __future__ import annotations

import dataclasses
import math

import pytest
import torch

from tests import kv_util as U
from tests.kv_check import check, dropped
from tests.test_gpu_kv import check_attn, gdn, status, to_cache  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def many_plan(gdn, b, h_q, ctas, **kw):  # noqa: F811
    """A plan for many rows, without a window one whose CTAs take runs of items (sized for longer sequences than there are)."""
    p = gdn.gdn_kv_attn_plan(T=b.T, n_seqs=b.n, h_q=h_q, h_kv=b.h_kv, max_q_len=max(b.q_lens), max_kv_len=20000,
                             sm_count=ctas, **kw)
    assert (p.raw.path, p.raw.rows, p.raw.n_ctas) == (2, 256, 0 if kw.get("window") else ctas)
    return p


@pytest.mark.parametrize("q,kv,h_q,h_kv", [
    ([300] * 3, [700, 300, 411], 8, 4),      # 600 rows: a last row tile of 88, one query tile, a warp without rows
    ([300, 37, 90], [300, 60, 222], 7, 3),   # heads that do not divide: rows without a query in every warp
    ([130] * 4, [130, 900, 131, 150], 16, 8)])
@pytest.mark.parametrize("ctas", [1, 3, 7])
def test_items_in_turn(gdn, q, kv, h_q, h_kv, ctas):  # noqa: F811
    """Several items a CTA, every head with its own keys and queries: a warp that is done with an item early
    writes its next queries while others still hand out their output."""
    b = U.Batch(q, kv, h_kv, seed=ctas + h_q)
    b.fill()
    x = b.randn(b.T, h_q, 128)
    plan = many_plan(gdn, b, h_q, ctas)
    first = check_attn(gdn, b, h_q, BF, q=x, plan=plan)
    cache, lens, table, cu = to_cache(gdn, b), b.lens.cuda(), b.table.cuda(), b.cu.cuda()
    for _ in range(20):
        out, lse = gdn.gdn_kv_attn(x.to(BF).cuda(), cache, lens, table, cu, plan=plan)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert status(gdn, cache) == (0, 0)


@pytest.mark.parametrize("what", [float("inf"), -float("inf"), float("nan")])
def test_bad_queries_without_keys(gdn, what):  # noqa: F811
    """Queries that are not finite are NaN where they have a key, and zeros like any other where they have none."""
    b = U.Batch([200, 150], [60, 400], 2, seed=5)  # the first sequence's first 140 tokens lie before position 0
    b.fill()
    q = b.randn(b.T, 8, 128)
    q[::3, :, 5] = what
    cache = to_cache(gdn, b)
    plan = many_plan(gdn, b, 8, 5)
    out, lse = gdn.gdn_kv_attn(q.to(BF).cuda(), cache, b.lens.cuda(), b.table.cuda(), b.cu.cuda(), plan=plan)
    assert (out[:140] == 0).all() and (lse[:140] == -float("inf")).all()
    bad = torch.zeros(b.T, dtype=torch.bool)
    bad[::3] = True
    bad[:140] = False
    assert torch.equal(out.isnan().all(-1).cpu(), bad[:, None].expand(-1, 8))
    assert torch.equal(out.isnan().any(-1).cpu(), bad[:, None].expand(-1, 8))
    assert torch.equal(lse.isnan().cpu(), bad[:, None].expand(-1, 8))


@pytest.mark.parametrize("tiny", [0.0, 1e-30])
@pytest.mark.parametrize("window", [0, 100])
def test_zero_queries_over_zero_keys(gdn, tiny, window):  # noqa: F811
    """Every key weighs the same, whatever scale a page of zeros has (2^-40, the least there is)."""
    b = U.Batch([200, 300], [200, 700], 2, seed=3)
    b.fill()
    for i in (0, 1):
        pages = b.table[i, :3 if i else 2].long()  # of the second sequence, the first keys only
        b.k[pages], b.ks[pages] = 0.0, 2.0 ** -40
    q = b.randn(b.T, 8, 128)
    q[:250] = tiny
    check_attn(gdn, b, 8, BF, q=q, window=window, plan=many_plan(gdn, b, 8, 5, window=window))


def test_zero_prompt(gdn):  # noqa: F811
    """A prompt of zeros through append and attention, as a warm-up sends it, under the call's own plan."""
    n = 512
    b = U.Batch([n], [n], 2, seed=1)
    b.fill(stale_nan=False)
    b.v, b.vs = b.randn(b.n_pages, 2, 64, 128).to(torch.float8_e4m3fn).float(), torch.ones(b.n_pages, 2)
    assert gdn.gdn_kv_attn_plan(T=n, n_seqs=1, h_q=8, h_kv=2, max_pages=b.max_pages).raw.path == 2
    cache, lens, table = to_cache(gdn, b), b.lens.cuda(), b.table.cuda()
    zero = torch.zeros(n, 2, 128, dtype=BF, device="cuda")
    gdn.gdn_kv_append(cache, zero, zero, lens, table)
    assert (cache.k_scale[b.table[0].long()] == 2.0 ** -40).all()
    out, lse = gdn.gdn_kv_attn(torch.zeros(n, 8, 128, dtype=BF, device="cuda"), cache, lens, table)
    assert (out == 0).all()
    want = torch.log(torch.arange(1, n + 1, dtype=torch.float64))[:, None].cuda()
    assert (lse.double() - want).abs().max() <= 2.0 ** -16


# ---------------------------------------------------------------- contents, lengths and layouts, on this kernel for certain
def plan_of(gdn, b, h_q, runs, window=0, **kw):  # noqa: F811
    """Whole items, or runs of items on five CTAs; sized for more than a window leaves."""
    p = gdn.gdn_kv_attn_plan(T=b.T, n_seqs=b.n, h_q=h_q, h_kv=b.h_kv, max_q_len=max(b.q_lens),
                             max_kv_len=20000 if runs else max(b.kv_lens), sm_count=5, **kw)
    assert p.raw.path == 2 and (p.raw.n_ctas > 0) == runs
    return dataclasses.replace(p, window=window)


@pytest.mark.parametrize("runs", [False, True])
@pytest.mark.parametrize("n,window", [(200, 0), (300, 33), (100, 150)])
def test_nan_outside_masks(gdn, n, window, runs):  # noqa: F811
    """Keys and values that no row may use, NaN in both, change nothing; rows that may use one are NaN."""
    b = U.Batch([n], [450], 2, seed=n)
    b.fill()

    def poison(pos, keys=True):
        page = int(b.table[0, pos // 64])
        if keys:
            b.k[page, :, pos % 64] = math.nan
        b.v[page, :, pos % 64, 5] = math.nan  # one element of the value
    if window:
        poison(450 - n - window)  # the last position outside every window
        poison(0)
        seen = None
    else:
        seen = 430
        poison(seen, keys=False)  # the last 20 rows see it
    q = b.randn(b.T, 4, 128).to(BF)
    cache = to_cache(gdn, b)
    out, lse = gdn.gdn_kv_attn(q.cuda(), cache, b.lens.cuda(), b.table.cuda(), plan=plan_of(gdn, b, 4, runs, window))
    o, z, mass, reach, top = U.attn_ref(b, q, True, window)
    bo, bz = U.attn_bounds(o, mass, reach, top, BF)
    bo = bo + dropped(b, q, 2, True, window)
    rows = slice(0, n if seen is None else seen - (450 - n))
    assert not out[rows].isnan().any() and not lse[rows].isnan().any()
    assert ((out.double().cpu() - o).abs() <= bo)[rows].all() and ((lse.double().cpu() - z).abs() <= bz)[rows].all()
    if seen is not None:
        assert out[seen - (450 - n):, :, 5].isnan().all()


@pytest.mark.parametrize("runs", [False, True])
def test_nan_keys_attended(gdn, runs):  # noqa: F811
    """A NaN key makes the rows that attend to it NaN, in tiles with masks and without; the others stay."""
    b = U.Batch([200], [600], 2, seed=7)
    b.fill()
    for pos in (450, 590):
        b.k[int(b.table[0, pos // 64]), 1, pos % 64] = math.nan
    q = b.randn(b.T, 4, 128).to(BF)
    out, lse = gdn.gdn_kv_attn(q.cuda(), to_cache(gdn, b), b.lens.cuda(), b.table.cuda(), plan=plan_of(gdn, b, 4, runs))
    bad = torch.zeros(200, 4, dtype=torch.bool)
    bad[450 - 400:, 2:] = True  # the second key/value head's query heads
    assert torch.equal(out.isnan().any(-1).cpu(), bad) and torch.equal(out.isnan().all(-1).cpu(), bad)
    assert torch.equal(lse.isnan().cpu(), bad)


@pytest.mark.parametrize("runs", [False, True])
def test_scales_far_apart(gdn, runs):  # noqa: F811
    """Pages whose scales differ by many powers of two, pages of zeros among them."""
    b = U.Batch([150], [700], 1, seed=150)
    b.fill()
    e = torch.tensor([0, -40, 12, -9, 3, -20, 20, -3, 0, 1, -1, 5])[: len(b.table[0])].double()
    for slot, x in enumerate(e.tolist()):
        b.vs[b.table[0, slot].long()] *= 2.0 ** max(min(x, 20.0), -20.0)
        b.ks[b.table[0, slot].long()] *= 2.0 ** max(min(x / 8, 2.0), -20.0)
    b.v[b.table[0, 1].long()] = 0.0
    b.vs[b.table[0, 1].long()] = 2.0 ** -40
    b.ks = torch.pow(2.0, torch.round(torch.log2(b.ks)))
    check(gdn, b, 4, plan_of(gdn, b, 4, runs))


@pytest.mark.parametrize("runs", [False, True])
def test_sharp_and_flat(gdn, runs):  # noqa: F811
    """Scores from far below to far above the others, rows of zeros and of tiny queries, a negative scale."""
    b = U.Batch([1, 200, 40], [500, 500, 500], 2, seed=9, spread=0.2)
    b.fill()
    q = b.randn(b.T, 4, 128)
    q[0] *= 200.0
    q[1:10] = 0.0
    q[20:60] *= 1e-20
    q[60:70] *= 1e-37
    q[150:170] *= 1e4
    check(gdn, b, 4, plan_of(gdn, b, 4, runs), q=q)
    for scale in (0.5, -0.5):
        check(gdn, b, 4, plan_of(gdn, b, 4, runs, scale=scale))


@pytest.mark.parametrize("runs", [False, True])
def test_weights_far_below_the_largest(gdn, runs):  # noqa: F811
    """The largest weight's value is zero, and the others, 2^-15 of it, make the output: the weights are fp16 at
    2^3 of the largest, with all eleven bits from 2^-17 of it on, and the output's rounding is one of nine."""
    n, kv = 100, 1000
    b = U.Batch([n], [kv], 1, seed=n)
    pages = b.table[0].long()
    b.k, b.ks = torch.zeros(b.n_pages, 1, 64, 128), torch.ones(b.n_pages, 1)
    b.v, b.vs = torch.zeros(b.n_pages, 1, 64, 128), torch.ones(b.n_pages, 1)
    b.v[pages] = 1.0
    b.v[pages[0], 0, 0] = 0.0
    b.k[pages[0], 0, 0, 0] = 1.0
    q = torch.zeros(n, 4, 128)
    q[..., 0] = 1.0
    scale = 15 * math.log(2.0)
    out, _ = gdn.gdn_kv_attn(q.to(BF).cuda(), to_cache(gdn, b), b.lens.cuda(), b.table.cuda(),
                             plan=plan_of(gdn, b, 4, runs, scale=scale))
    w = (kv - n + torch.arange(n)).double() * 2.0 ** -15
    want = (w / (1 + w))[:, None, None]
    assert ((out.double().cpu() - want).abs() / want).max() <= 2.0 ** -11 + 2.0 ** -9 + 2.0 ** -12


@pytest.mark.parametrize("runs", [False, True])
def test_strided(gdn, runs):  # noqa: F811
    b = U.Batch([1, 4, 90], [100, 4, 300], 2, seed=21)
    b.fill()
    wide = b.randn(b.T, 11, 128).to(BF).cuda()
    into = torch.full((b.T, 9, 128), 7.0, dtype=BF, device="cuda")
    args = (to_cache(gdn, b), b.lens.cuda(), b.table.cuda(), b.cu.cuda())
    plan = plan_of(gdn, b, 6, runs)
    out, lse = gdn.gdn_kv_attn(wide[:, 2:8], *args, plan=plan, out=into[:, 1:7])
    packed, lse2 = check(gdn, b, 6, plan, q=wide[:, 2:8].cpu())
    assert torch.equal(out, packed) and torch.equal(lse, lse2)
    assert (into[:, 0] == 7).all() and (into[:, 7:] == 7).all()


def test_pool_past_32_bits(gdn):  # noqa: F811
    """Pages whose codes lie past 2^31 and 2^32 bytes of the pool."""
    b = U.Batch([150], [400], 2, seed=2)
    b.fill(stale_nan=False)
    pool = 300_000  # 2 heads: 4.9 GB of keys
    cache = gdn.KVCache.empty(pool, 2)
    table = torch.tensor([[pool - 1 - 11 * i for i in range(b.max_pages)]], dtype=torch.int32)
    for i in range(b.max_pages):
        src, dst = int(b.table[0, i]), int(table[0, i])
        cache.k.view(torch.uint8)[dst] = b.k[src].to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        cache.v.view(torch.uint8)[dst] = b.v[src].to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        cache.k_scale[dst], cache.v_scale[dst] = b.ks[src].cuda(), b.vs[src].cuda()
    q = b.randn(150, 4, 128)
    plan = plan_of(gdn, b, 4, True)
    want = check(gdn, b, 4, plan, q=q, use_cu=False)
    got = gdn.gdn_kv_attn(q.to(BF).cuda(), cache, b.lens.cuda(), table.cuda(), plan=plan)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("runs", [False, True])
def test_graph_replay_with_growing_lengths(gdn, runs):  # noqa: F811
    """A captured append + attention, replayed while the lengths grow on the device, gives what eager calls give."""
    n = 140
    b = U.Batch([n, n], [900, 900], 2, seed=6)
    b.fill(stale_nan=False)
    table = b.table.cuda()
    lens = torch.tensor([n + 60, n], dtype=torch.int32, device="cuda")
    q, k, v = (b.randn(2 * n, h, 128).to(BF).cuda() for h in (8, 2, 2))
    plan = plan_of(gdn, b, 8, runs)
    ws = torch.empty(max(256, plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    cache, eager = to_cache(gdn, b), to_cache(gdn, b)
    out, lse = torch.empty_like(q), torch.empty(2 * n, 8, device="cuda")
    torch.cuda.synchronize()
    gdn.gdn_kv_append(cache, k, v, lens, table)
    gdn.gdn_kv_attn(q, cache, lens, table, plan=plan, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_kv_append(cache, k, v, lens, table)
        gdn.gdn_kv_attn(q, cache, lens, table, plan=plan, out=out, lse=lse, workspace=ws)
    for step in range(3):
        g.replay()
        gdn.gdn_kv_append(eager, k, v, lens, table)
        o2, z2 = gdn.gdn_kv_attn(q, eager, lens, table, plan=plan)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, z2)
        lens += n
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape).to(x.dtype))
    assert status(gdn, cache) == (0, 0)
