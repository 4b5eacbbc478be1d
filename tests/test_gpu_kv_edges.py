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
