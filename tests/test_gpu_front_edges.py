"""The operators between the projections and the mixers where fp32 ends: heads
near its largest numbers, and sums over millions of tokens."""
from __future__ import annotations

import pytest
import torch

from tests import front_util as F

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU, skipped there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_deltanet_linear_fwd_gb300 as gdn  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("norm", ["rms", "unit"])
def test_gradients_of_the_largest_heads(norm):
    """r is below fp32's normal numbers there, its product with a large gradient is not: as good as of other heads.

    One element of dy is not zero and nothing turns, so its dx is r dn but for 1 / 128: r is good to 8 roundings
    (F.rope_ref), the fused product and r's one each.  The others are r n sum(dn n) k, of 10, 10 + 8 + 1, 8 and 2."""
    g = torch.Generator().manual_seed(1)
    T = 96
    x = (torch.randn(T, 2, 128, generator=g).sign() * torch.logspace(37.0, 38.5, T)[:, None, None]).contiguous()
    dy = torch.zeros(T, 2, 128)
    at = torch.randint(0, 128, (T, 2, 1), generator=g)
    dy.scatter_(2, at, 1e12 * (1 + torch.rand(T, 2, 1, generator=g)))
    got = gdn.gdn_qk_rope_bwd(x.cuda(), None, dy.cuda(), None, norm=norm)[0]
    want = F.rope_bwd_ref(x, dy, torch.arange(T), F.frequencies(0), norm=norm)[0]
    r = F.inv_norm(x.double(), norm, 1e-6)
    n, k = x.double() * r, 1 / 128 if norm == "rms" else 1.0
    F.check("dx", got, want, F.U * r * (10 * dy.double() + 39 * n.abs() * (dy.double() * n.abs()).sum(-1, keepdim=True) * k))
