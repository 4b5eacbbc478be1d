"""Refusals and edges of the 8-bit key/value cache's host side (no GPU)."""
from __future__ import annotations

import pytest

from tests.test_kv_host import INVALID, OK, cache, dims, lib, plan  # noqa: F401


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("max_kv", [0, 64, 100000])
def test_no_tokens(lib, dtype, max_kv):  # noqa: F811
    """A call without tokens plans, and does nothing."""
    st, p = plan(lib, max_q=0, max_kv=max_kv, T=0, max_pages=2000, dtype=dtype)
    assert st == OK and p.rows >= 8 and p.max_row_tiles == 1
    assert lib.gdn_kv_attn(None, 64, 64, None, cache(), None, None, dims(T=0, max_pages=2000, dtype=dtype), p, 4096,
                           p.workspace_bytes, None) == OK
