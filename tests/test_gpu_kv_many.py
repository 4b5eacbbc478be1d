"""The many-rows attention kernel over the 8-bit cache, on calls whose plan is
checked to take it: items that follow one another in a CTA, and contents that
only this kernel treats in its own way."""
from __future__ import annotations

import pytest
import torch

from tests import kv_util as U
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
