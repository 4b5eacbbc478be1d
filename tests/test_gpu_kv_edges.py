"""Edges of the 8-bit key/value cache's calls on the GPU."""
from __future__ import annotations

import pytest
import torch

from tests import kv_util as U
from tests.test_gpu_kv import gdn, status, to_cache  # noqa: F401

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
