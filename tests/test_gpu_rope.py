"""Head norms and rotary positions on the GPU against their 64-bit forms: every
layout, norm and type, odd sizes, strides, far positions, values at the ends
of the range, and the gradients."""
from __future__ import annotations

import math

import pytest
import torch

from tests import front_util as F

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU, skipped there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_deltanet_linear_fwd_gb300 as gdn  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def rand(g, *s, spread=0.4):
    return torch.randn(*s, generator=g) * torch.exp(spread * torch.randn(*s[-2:], generator=g))


def fused(parts, dtype):
    """The tensors [T, h, 128] as views of one [T, sum h, 128] on the GPU."""
    x = torch.cat(parts, 1).to(dtype).cuda()
    return list(x.split([p.shape[1] for p in parts], dim=1))


class Case:
    def __init__(self, lens, h_q, h_k, dtype=BF16, layout="half", rot=128, norm="rms", weights=True, where="cu", strided=True,
                 eps=0.0, seed=0, **scaling):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.T, self.dtype, self.layout, self.rot, self.norm = lens, sum(lens), dtype, layout, rot, norm
        self.q, self.k = rand(g, self.T, h_q, 128).to(dtype), rand(g, self.T, h_k, 128).to(dtype)
        self.dq, self.dk = rand(g, self.T, h_q, 128).to(dtype), rand(g, self.T, h_k, 128).to(dtype)
        self.qw = 1 + 0.3 * torch.randn(128, generator=g) if weights and norm != "none" else None
        self.kw = 1 + 0.3 * torch.randn(128, generator=g) if weights and norm != "none" else None
        self.eps = eps or 1e-6
        self.mag = scaling.pop("magnitude", 1.0)
        self.freqs = F.frequencies(rot, **scaling)
        self.rope = gdn.gdn_rope_table(rot, layout=layout, magnitude=self.mag, **scaling)
        self.positions = self.cu = None
        self.pos = F.places(lens)[1]
        if where == "positions":
            self.pos = torch.randint(-2 ** 20, 2 ** 20, (self.T,), generator=g)
            self.positions = self.pos.to(torch.int32).cuda()
        elif len(lens) > 1:
            self.cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
        if strided:
            self.gq, self.gk, _ = fused([self.q, self.k, self.k], dtype)
        else:
            self.gq, self.gk = self.q.cuda(), self.k.cuda()
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.how = dict(norm=norm, q_weight=dev(self.qw), k_weight=dev(self.kw), eps=eps)

    def want(self, x, w):
        return F.rope_ref(x, self.pos, self.freqs, self.layout, self.mag, self.norm, w, self.eps)

    def forward(self, **kw):
        return gdn.gdn_qk_rope(self.gq, self.gk, self.rope, self.positions, self.cu, **self.how, **kw)

    def check_forward(self, outs):
        for name, got, x, w in (("q", outs[0], self.q, self.qw), ("k", outs[1], self.k, self.kw)):
            F.check(name, got, *self.want(x, w), self.dtype)

    def backward(self, **kw):
        return gdn.gdn_qk_rope_bwd(self.gq, self.gk, self.dq.cuda(), self.dk.cuda(), self.rope, self.positions, self.cu, **self.how,
                                   **kw)

    def check_backward(self, grads):
        for name, got, got_w, x, dy, w in (("q", grads[0], grads[2], self.q, self.dq, self.qw),
                                           ("k", grads[1], grads[3], self.k, self.dk, self.kw)):
            dx, dw, bx, bw = F.rope_bwd_ref(x, dy, self.pos, self.freqs, self.layout, self.mag, self.norm, w, self.eps)
            F.check("d" + name, got, dx, bx, self.dtype)
            if w is None:
                assert got_w is None
            else:
                F.check("d" + name + "_weight", got_w, dw, bw)


CASES = [
    dict(lens=[1], h_q=1, h_k=1), dict(lens=[1], h_q=8, h_k=2, where="positions"), dict(lens=[7], h_q=3, h_k=2, dtype=F32, strided=False),
    dict(lens=[333], h_q=8, h_k=2), dict(lens=[64, 1, 0, 130, 17], h_q=5, h_k=5, layout="interleaved", rot=64),
    dict(lens=[40, 41], h_q=16, h_k=1, norm="unit", dtype=F32), dict(lens=[100], h_q=2, h_k=2, norm="none", layout="interleaved"),
    dict(lens=[0, 0, 90, 0], h_q=4, h_k=3, rot=8, norm="unit", weights=False), dict(lens=[257], h_q=1, h_k=1, rot=16, dtype=F32, norm="none"),
    dict(lens=[200], h_q=32, h_k=8, rot=96, where="positions"), dict(lens=[50] * 9, h_q=7, h_k=1, layout="interleaved", rot=24, dtype=F32),
    dict(lens=[700], h_q=8, h_k=2, scaling="parts", factor=8.0, original_len=4096.0, magnitude=1.2079, where="positions"),
    dict(lens=[61], h_q=4, h_k=4, scaling="ntk", factor=4.0, rot=32, where="positions", dtype=F32),
    dict(lens=[61], h_q=4, h_k=4, scaling="linear", factor=2.0, layout="interleaved", eps=1e-2, strided=False),
    dict(lens=[4109], h_q=3, h_k=2, rot=40, norm="rms", weights=False)]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward(i):
    c = Case(**CASES[i], seed=i)
    outs = c.forward()
    assert all(o.is_contiguous() for o in outs)
    c.check_forward(outs)


@pytest.mark.parametrize("i", range(len(CASES)))
def test_backward(i):
    c = Case(**CASES[i], seed=100 + i)
    c.check_backward(c.backward())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_into_given_tensors(dtype):
    """Outputs in place of the inputs, and as parts of a wider tensor whose rest stays."""
    c = Case([45, 3], 4, 2, dtype, seed=7)
    wide = torch.full((48, 9, 128), 7.0, dtype=dtype, device="cuda")
    c.check_forward(c.forward(q_out=wide[:, 1:5], k_out=wide[:, 6:8]))
    assert (wide[:, [0, 5, 8]] == 7).all()
    rest = c.gk.clone()
    again = c.forward(q_out=c.gq)
    assert again[0] is c.gq and torch.equal(c.gk, rest)
    c.check_forward(again)
    c = Case([45, 3], 4, 2, dtype, seed=8)
    d_qk = fused([c.dq, c.dk], dtype)
    grads = gdn.gdn_qk_rope_bwd(c.gq, c.gk, *d_qk, c.rope, c.positions, c.cu, **c.how, d_q=d_qk[0], d_k=d_qk[1])
    c.check_backward(grads)


def test_batch_of_rows():
    """[B, T, h, 128]: each row from position 0; a single-token row; rows of a wider batch."""
    g = torch.Generator().manual_seed(3)
    rope, f = gdn.gdn_rope_table(128), F.frequencies(128)
    for B, T in ((3, 5), (4, 1), (1, 9)):
        x = torch.randn(B, T, 6, 128, generator=g)
        dev = x.cuda()
        q, k = gdn.gdn_qk_rope(dev[:, :, :4], dev[:, :, 4:], rope)
        assert q.shape == (B, T, 4, 128)
        pos = torch.arange(T).repeat(B)
        F.check("q", q.flatten(0, 1), *F.rope_ref(x[:, :, :4].flatten(0, 1), pos, f))
        F.check("k", k.flatten(0, 1), *F.rope_ref(x[:, :, 4:].flatten(0, 1), pos, f))


def test_one_side():
    c = Case([20], 4, 2, seed=9)
    q, none = gdn.gdn_qk_rope(c.gq, None, c.rope, norm="rms", q_weight=c.how["q_weight"])
    assert none is None and torch.equal(q, c.forward()[0])
    none, k = gdn.gdn_qk_rope(None, c.gk, c.rope, norm="rms", k_weight=c.how["k_weight"])
    assert none is None and torch.equal(k, c.forward()[1])
    got = gdn.gdn_qk_rope_bwd(None, c.gk, None, c.dk.cuda(), c.rope, norm="rms", k_weight=c.how["k_weight"])
    want = c.backward()
    assert got[0] is None and got[2] is None and torch.equal(got[1], want[1])
    c.check_backward((want[0], got[1], want[2], got[3]))   # a call of other heads adds up in another order


def test_norm_alone():
    """Without a rotation: the norm, and with no norm either a copy."""
    c = Case([33], 2, 2, F32, seed=10)
    q, _ = gdn.gdn_qk_rope(c.gq, c.gk, norm="rms", q_weight=c.how["q_weight"], k_weight=c.how["k_weight"])
    F.check("q", q, F.normed(c.q, "rms", c.qw, 1e-6), 10 * F.U * F.normed(c.q, "rms", c.qw, 1e-6).abs())
    assert torch.equal(gdn.gdn_qk_rope(c.gq, None)[0], c.gq)


@pytest.mark.parametrize("positions", [[2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, -1, 0, 10 ** 9, 262143, 16777217]])
def test_far_positions(positions):
    """Angles keep fp32's precision at any position: the bound has no term in it."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(len(positions), 2, 128, generator=g)
    p = torch.tensor(positions)
    for layout in ("half", "interleaved"):
        q, _ = gdn.gdn_qk_rope(x.cuda(), None, gdn.gdn_rope_table(128, layout=layout), p.to(torch.int32).cuda())
        want, bound = F.rope_ref(x, p, F.frequencies(128), layout)
        # the 64-bit form's own angle, p f, is off by up to 4 of 2^-53 of itself: 2^31 radians by 2^-20
        F.check("q", q, want, bound + 4 * p.abs().double()[:, None, None] * 2.0 ** -53 * F.reach(x.double(), 128, layout, 1.0))


@pytest.mark.parametrize("norm", ["rms", "unit"])
def test_ends_of_the_range(norm):
    """Heads of zeros, of the largest finite values, of values whose squares underflow, and not finite ones."""
    rope, f = gdn.gdn_rope_table(128), F.frequencies(128)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(1, 6, 128, generator=g)
    x[0, 0] = 0
    x[0, 1] *= 1e38 / 5
    x[0, 2] = 3.3e38
    x[0, 3] *= 1e-30
    x[0, 4] *= 1e-3
    x[0, 5] = 0
    x[0, 5, 3] = 2.0 ** 70
    pos = torch.tensor([12345])
    q, _ = gdn.gdn_qk_rope(x.cuda(), None, rope, pos.to(torch.int32).cuda(), norm=norm)
    want, bound = F.rope_ref(x, pos, f, norm=norm)
    F.check("q", q, want, bound)
    assert (q[0, 0] == 0).all()
    # gradients of the ordinary and the large ones: dx of large heads is below fp32's normal numbers
    dy = torch.randn(1, 6, 128, generator=g)
    dx = gdn.gdn_qk_rope_bwd(x.cuda(), None, dy.cuda(), None, rope, pos.to(torch.int32).cuda(), norm=norm)[0]
    want, _, bound, _ = F.rope_bwd_ref(x, dy, pos, f, norm=norm)
    F.check("dx", dx, want, bound + 1e-37)
    # an infinity makes NaN of its pair, NaN of the head
    y = torch.randn(1, 3, 128, generator=g)
    y[0, 0, 5] = math.inf
    y[0, 1, 9] = math.nan
    q, _ = gdn.gdn_qk_rope(y.cuda(), None, rope, pos.to(torch.int32).cuda(), norm=norm)
    bad = q[0, 0].isnan().cpu()
    assert bad[5] and bad[69] and bad.sum() == 2 and (q[0, 0].cpu()[~bad] == 0).all()
    assert q[0, 1].isnan().all()
    F.check("q", q[:, 2:], *F.rope_ref(y[:, 2:], pos, f, norm=norm))


def test_tokens_outside_every_sequence():
    """A padded batch: what lies before the first and behind the last sequence stays, and does not count."""
    c = Case([5, 0, 30], 3, 2, F32, seed=11)
    pad = lambda t: torch.cat([torch.full((4, *t.shape[1:]), math.nan), t, torch.full((6, *t.shape[1:]), math.nan)]).cuda()  # noqa: E731
    cu = c.cu + 4
    q_out, k_out = torch.full((45, 3, 128), 5.0, device="cuda"), torch.full((45, 2, 128), 5.0, device="cuda")
    q, k = gdn.gdn_qk_rope(pad(c.q), pad(c.k), c.rope, None, cu, **c.how, q_out=q_out, k_out=k_out)
    c.check_forward((q[4:39], k[4:39]))
    for t in (q, k):
        assert (t[:4] == 5).all() and (t[39:] == 5).all()
    q_out.fill_(5)
    k_out.fill_(5)
    grads = gdn.gdn_qk_rope_bwd(pad(c.q), pad(c.k), pad(c.dq), pad(c.dk), c.rope, None, cu, **c.how, d_q=q_out, d_k=k_out)
    c.check_backward((grads[0][4:39], grads[1][4:39], *grads[2:]))
    for t in grads[:2]:
        assert (t[:4] == 5).all() and (t[39:] == 5).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_the_rest_of_a_head_stays_apart(layout):
    """What is not finite in the part that does not turn stays in its element, and in the other's pair."""
    g = torch.Generator().manual_seed(20)
    x = torch.randn(1, 2, 128, generator=g)
    x[0, 0, [40, 101]] = math.inf
    x[0, 1, 3] = math.nan
    q, _ = gdn.gdn_qk_rope(x.cuda(), None, gdn.gdn_rope_table(32, layout=layout), torch.tensor([77], dtype=torch.int32, device="cuda"))
    assert q[0, 0].isfinite().logical_not().nonzero().flatten().tolist() == [40, 101]
    assert q[0, 1].isfinite().logical_not().nonzero().flatten().tolist() == ([3, 19] if layout == "half" else [2, 3])


def test_no_tokens():
    c = Case([3], 2, 2, seed=12)
    q, k = gdn.gdn_qk_rope(c.gq[:0], c.gk[:0], c.rope, **c.how)
    assert q.shape == (0, 2, 128) and k.shape == (0, 2, 128)
    grads = gdn.gdn_qk_rope_bwd(c.gq[:0], c.gk[:0], c.dq[:0].cuda(), c.dk[:0].cuda(), c.rope, **c.how)
    assert grads[0].shape == (0, 2, 128) and (grads[2] == 0).all() and (grads[3] == 0).all()


def test_gradients_against_differences():
    """The GPU's gradients along a direction against differences of the 64-bit forward."""
    c = Case([20, 12], 3, 2, F32, norm="rms", where="cu", seed=13)
    grads = c.backward()
    g = torch.Generator().manual_seed(14)
    for x, w, dy, dx, dw in ((c.q, c.qw, c.dq, grads[0], grads[2]), (c.k, c.kw, c.dk, grads[1], grads[3])):
        d, e = torch.randn(x.shape, generator=g).double(), torch.randn(128, generator=g).double()
        loss = lambda t: float((c.want(x.double() + t * d, w.double() + t * e)[0] * dy.double()).sum())  # noqa: E731
        h = 1e-5
        slope = (loss(h) - loss(-h)) / (2 * h)
        parts = (dx.double().cpu() * d).sum() + (dw.double().cpu() * e).sum()
        size = (dx.double().cpu() * d).abs().sum() + (dw.double().cpu() * e).abs().sum()
        # fp32 gradients to 2^-17 of what is summed; differences to h^2 and 2^-53 / h of the loss's terms
        assert abs(slope - float(parts)) <= float(size) * 2.0 ** -17 + 1e-4


def test_repeats_bit_for_bit():
    c = Case([5000], 8, 2, seed=15)
    one, two = c.backward(), c.backward(workspace=torch.full((gdn.gdn_qk_rope_bwd_workspace_bytes(),), 255, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_refusals():
    c = Case([8], 2, 2, seed=16)
    other = torch.zeros(8, 2, 128, device="cuda", dtype=F32)
    for bad in (dict(q_out=other), dict(k_out=c.gk[:4]), dict(q_out=torch.zeros(8, 2, 128, dtype=BF16)), dict(norm="both"),
                dict(q_weight=torch.ones(64, device="cuda")), dict(q_weight=torch.ones(128, device="cuda", dtype=BF16)),
                dict(k_weight=torch.ones(128))):
        with pytest.raises(ValueError):
            gdn.gdn_qk_rope(c.gq, c.gk, c.rope, **{**c.how, **bad})
    for positions in (torch.zeros(8, device="cuda"), torch.zeros(7, dtype=torch.int32, device="cuda"), torch.zeros(8, dtype=torch.int32)):
        with pytest.raises(ValueError):
            gdn.gdn_qk_rope(c.gq, c.gk, c.rope, positions)
    with pytest.raises(ValueError):
        gdn.gdn_qk_rope(c.gq, c.gk, gdn.gdn_rope_table(128, device="cpu"))
    with pytest.raises(gdn.api.L.GDNError):
        gdn.gdn_qk_rope(c.gq, c.gk, c.rope, q_weight=c.how["q_weight"])   # a weight without a norm
    with pytest.raises(ValueError):
        gdn.gdn_qk_rope(c.gq.view(2, 4, 2, 128) if c.gq.is_contiguous() else c.gq.clone().view(2, 4, 2, 128), None, c.rope, None,
                        torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda"))
    with pytest.raises(gdn.api.L.GDNError):
        gdn.gdn_qk_rope_bwd(c.gq, c.gk, c.dq.cuda(), c.dk.cuda(), c.rope, **c.how,
                            workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
