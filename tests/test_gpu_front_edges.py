"""The operators between the projections and the mixers where fp32 ends: heads
near its largest numbers, and sums over millions of tokens; long fp32 appends."""
from __future__ import annotations

import pytest
import torch

from tests import front_util as F

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU, skipped there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_deltanet_linear_fwd_gb300 as gdn  # noqa: E402
from tests.test_gpu_kv_rope import Case  # noqa: E402

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


def test_large_gradients_of_large_heads():
    """r is large beside the scale there: dx is far within fp32's range, as is each product on the way."""
    x, dy = torch.full((3, 1, 128), 1.65e18), torch.zeros(3, 1, 128)     # squares' sum 3.5e38
    dy[:, 0, 7] = torch.tensor([1e37, -2e37, 1e36])
    got = gdn.gdn_qk_rope_bwd(x.cuda(), None, dy.cuda(), None, norm="rms")[0]
    want, _, bound, _ = F.rope_bwd_ref(x, dy, torch.arange(3), F.frequencies(0), norm="rms")
    F.check("dx", got, want, bound)


def test_large_gradients_of_large_heads_before_the_delta_rule():
    """The same behind the convolution's unit norm, whose taps are one of the token itself."""
    x, w = torch.full((3, 384), 1.65e18), torch.zeros(384, 2)
    w[:, 1] = 1
    d = [torch.zeros(3, 1, 128) for _ in range(3)]
    d[0][:, 0, 7] = d[1][:, 0, 9] = torch.tensor([3e37, -9e37, 1e36])
    got = gdn.gdn_conv_bwd(x.cuda(), w.cuda(), 1, *[t.cuda() for t in d], activation="none")[0]
    want, bound = F.Conv(x, w, 1, silu=False).backward(*d)
    F.check("dx", got, want[0], bound[0])


def in_pieces(T, f, step=1 << 17):
    return sum(f(slice(i, min(i + step, T))) for i in range(0, T, step))


# Heads of a lane that one fp32 number sums, and the half-warps of a CTA, whose sums are then added up in fp32 too;
# the CTAs' are added in pairs of fp32.
ROPE_ROWS = 256 + 16


@pytest.mark.parametrize("dtype,rows", [(F32, 700), (BF16, 700), (BF16, 5500)])
def test_rope_weights_gradients_of_many_tokens(dtype, rows):
    """Every element against 64 bits, `rows` heads a lane.  Of the first 64 elements all terms are equal, where the
    roundings of a running sum do not cancel: with numbers of 2^12 it drops half a term's last 12 bits each time."""
    T = rows * (2 * 152) * 16 // 4
    g = torch.Generator("cuda").manual_seed(2)
    x = [torch.randint(0, 2, (T, h, 128), device="cuda", generator=g, dtype=torch.int8).mul_(2).sub_(1).to(dtype) for h in (3, 1)]
    d = [torch.randn(T, h, 128, device="cuda", generator=g, dtype=dtype) for h in (3, 1)]
    for a, b in zip(x, d):
        b[..., :64] = a[..., :64]
    magnitude = 1 + 0.45 * 2.0 ** -12     # du n of the first 64, but for r
    rope = gdn.gdn_rope_table(128, magnitude=magnitude)
    w = torch.ones(128, device="cuda")
    grads = gdn.gdn_qk_rope_bwd(*x, *d, rope, torch.zeros(T, dtype=torch.int32, device="cuda"), norm="rms", q_weight=w, k_weight=w)
    factor = float(torch.tensor(magnitude, dtype=F32)) / (1 + 1e-6) ** 0.5
    for a, b, got in zip(x, d, grads[2:]):
        want = factor * in_pieces(T, lambda s: (a[s].double() * b[s].double()).sum((0, 1)))
        mass = factor * in_pieces(T, lambda s: b[s].abs().sum((0, 1), dtype=torch.float64))
        # du to 9 roundings (of one element alone: cos 1, sin 0), n to 10 and 2 for the product and the end
        F.check("dw", got, want.cpu(), ((9 + 10 + 2 + ROPE_ROWS) * F.U * mass).cpu())


def test_conv_weights_gradients_of_many_tokens():
    """Every tap and bias against 64 bits, where dx_t and the products are plain: no activation, no norm."""
    T, W = 2 ** 22 + 77, 4
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(T, 384, device="cuda", generator=g, dtype=BF16)
    d = [torch.randn(T, 1, 128, device="cuda", generator=g, dtype=BF16) for _ in range(3)]
    d[2] += 1    # sums that grow
    w, b = torch.randn(384, W, device="cuda", generator=g), torch.zeros(384, device="cuda")
    _, dw, db, _ = gdn.gdn_conv_bwd(x, w, 1, *d, b, activation="none", norm=False)
    # a running sum takes 192 tokens, then 8 warps'; the CTAs' are added in pairs of fp32; a product, and the end
    roundings = (192 + 8 + 2) * F.U
    for i, du in enumerate(d):
        xc, du = x[:, 128 * i:128 * i + 128], du[:, 0]
        want = in_pieces(T, lambda s: du[s].sum(0, dtype=torch.float64))
        F.check("db", db[128 * i:128 * i + 128], want.cpu(), roundings * in_pieces(T, lambda s: du[s].abs().sum(0, dtype=torch.float64)).cpu())
        for j in range(W):
            late = W - 1 - j     # du_t meets x_{t - late}
            a, c = xc[:T - late], du[late:]
            want = in_pieces(T - late, lambda s: (a[s].double() * c[s].double()).sum(0))
            mass = in_pieces(T - late, lambda s: (a[s].double() * c[s].double()).abs().sum(0))
            F.check("dw", dw[128 * i:128 * i + 128, j], want.cpu(), (roundings * mass).cpu())


@pytest.mark.parametrize("h_q,h_kv", [(8, 2), (2, 4)])
def test_long_append_of_fp32(h_q, h_kv):
    """More queries' heads than the resident warps take one of, pages beside them, behind earlier tokens."""
    c = Case([2900, 1, 333], [2900, 70, 1000], h_q, h_kv, F32, seed=4)
    c.check(c.call())
