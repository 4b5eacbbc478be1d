"""The few-rows attention kernel over the 8-bit cache at each of its row tiles, over ordinary lengths, on calls
whose plan is checked to take it."""
from __future__ import annotations

import dataclasses

import pytest

from tests import kv_util as U
from tests.kv_check import check
from tests.test_gpu_kv import gdn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("runs", [False, True])
@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("rows,n,h_q,h_kv", [(8, 1, 8, 2), (8, 2, 8, 2), (8, 1, 7, 3), (16, 3, 8, 2), (16, 1, 16, 1), (24, 5, 8, 2),
                                             (24, 6, 4, 1), (24, 8, 7, 3), (32, 8, 8, 2), (32, 10, 7, 3), (32, 1, 32, 1)])
def test_row_tiles(gdn, rows, n, h_q, h_kv, window, runs):  # noqa: F811
    """Several sequences, their heads' keys and values all different, lengths from a few keys to forty tiles."""
    b = U.Batch([n] * 9, [n, 70, 128, 129, 300, 511, 1100, 2500, 5000], h_kv, seed=rows + n)
    b.fill()
    p = gdn.gdn_kv_attn_plan(T=b.T, n_seqs=9, h_q=h_q, h_kv=h_kv, max_q_len=n, max_kv_len=20000 if runs else 64, sm_count=11)
    assert (p.raw.path, p.raw.rows) == (1, rows) and (p.raw.n_ctas > 0) == runs
    check(gdn, b, h_q, dataclasses.replace(p, window=window))  # sized for more than a window leaves


@pytest.mark.parametrize("n,h_q,h_kv", [(40, 8, 2), (9, 40, 1), (30, 7, 3)])
def test_several_row_tiles(gdn, n, h_q, h_kv):  # noqa: F811
    """Small calls of more than 32 rows, in tiles of 32."""
    b = U.Batch([n, 1, n - 7], [n, 700, 1500], h_kv, seed=n)
    b.fill()
    p = gdn.gdn_kv_attn_plan(T=b.T, n_seqs=3, h_q=h_q, h_kv=h_kv, max_q_len=n, max_kv_len=1500, sm_count=152)
    assert (p.raw.path, p.raw.rows) == (1, 32) and p.raw.max_row_tiles > 1
    check(gdn, b, h_q, p)
