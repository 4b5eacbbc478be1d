"""Calls at the ends of what the operators between the projections and the mixers
take, refused on the host (no GPU)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from tests.test_front_host import INVALID, OK, cache, conv_dims, kv_dims, lib, rope, rope_dims  # noqa: F401


@pytest.mark.parametrize("eps", [1.1e20, 1e36, 3e38])
def test_eps_beside_which_a_large_sum_is_not_alone(lib, eps):  # noqa: F811
    """Squares past fp32's range are summed of scaled elements and without eps, so eps has to be nothing beside 3e38 / 128."""
    assert lib.gdn_qk_rope(512, 1024, 64, 64, None, None, rope(), 2048, 4096, rope_dims(eps=eps), None) == INVALID
    assert lib.gdn_qk_rope_bwd(512, 1024, 64, 64, None, None, rope(), 2048, 4096, 512, 512, 64, 64, rope_dims(eps=eps), 256, 1 << 30,
                               None) == INVALID
    assert lib.gdn_kv_append_rope(512, 1024, 64, 512, 64, 2048, 64, 64, None, cache(), kv_dims(), rope(), 1, eps, None) == INVALID
    assert lib.gdn_conv_fwd(512, 64, 64, None, None, 1024, 2048, 4096, 8192, conv_dims(eps=eps), None) == INVALID
    assert lib.gdn_conv_bwd(512, 64, 64, None, None, 1024, 2048, 4096, None, 8192, 64, 64, None, conv_dims(eps=eps), 256, 1 << 40,
                            None) == INVALID
    assert lib.gdn_conv_step(512, 64, 64, 8192, 1024, 2048, 4096, conv_dims(T=2, eps=eps), None) == INVALID


@pytest.mark.parametrize("eps", [0.0, 1e-20, 1.0, 1e20])
def test_eps_that_is_taken(lib, eps):  # noqa: F811
    assert lib.gdn_qk_rope(None, None, 64, 64, None, None, rope(), None, None, rope_dims(T=0, eps=eps), None) == OK
    n = ctypes.c_size_t(0)
    assert lib.gdn_conv_bwd_workspace_bytes(conv_dims(eps=eps), n) == OK


def test_append_of_more_tokens_than_its_warps_are_counted(lib):  # noqa: F811
    """With offsets and up to 8 tokens a sequence a warp a token, head, and keys or values: their number stays below 2^31."""
    for T, n_seqs, h_kv in ((1 << 29, 1 << 26, 7), (1 << 28, 1 << 25, 4), (1 << 30, 1 << 27, 3)):
        many, offsets = kv_dims(T=T, n_seqs=n_seqs, h_q=1), 64
        assert 2 * (T // 64 + 2 * n_seqs) * h_kv < 2 ** 31 <= 2 * T * h_kv
        a = [512, 1024, 64, None, None, None, 64, 64, offsets, cache(h_kv=h_kv), many, rope(), 1, 0.0, None]
        assert lib.gdn_kv_append_rope(*a) == INVALID


def test_an_output_without_its_input():
    """It would come back as it was, as if it were the result."""
    import gated_deltanet_linear_fwd_gb300 as gdn
    x, y = torch.zeros(3, 2, 128), torch.ones(3, 2, 128)
    for call in (lambda: gdn.gdn_qk_rope(None, x, q_out=y), lambda: gdn.gdn_qk_rope(x, None, k_out=y),
                 lambda: gdn.gdn_qk_rope_bwd(None, x, None, x, d_q=y), lambda: gdn.gdn_qk_rope_bwd(x, None, x, None, d_k=y)):
        with pytest.raises(ValueError, match="go with"):
            call()
