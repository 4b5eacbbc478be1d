"""The short causal convolution on the GPU against its 64-bit form: forward,
gradients and single tokens, every width and type, runs and sequences that end
anywhere, states on both sides."""
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


class Case:
    def __init__(self, lens, h_qk=1, h_v=2, dtype=BF16, width=4, bias=False, state=False, silu=True, norm=True, pad=0, seed=0,
                 size=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.h_qk, self.h_v, self.dtype, self.width = list(lens), h_qk, h_v, dtype, width
        self.T, self.C, n = sum(lens), (2 * h_qk + h_v) * 128, len(lens)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.x = (size * rnd(self.T, self.C)).to(dtype)
        self.w = rnd(self.C, width) / math.sqrt(width)
        self.b = 0.3 * rnd(self.C) if bias else None
        self.state = rnd(n, width - 1, self.C).to(dtype) if state else None
        self.d = [rnd(self.T, h, 128).to(dtype) for h in (h_qk, h_qk, h_v)]
        self.d_final = rnd(n, width - 1, self.C).to(dtype) if state else None
        self.silu, self.norm = silu, norm
        self.cu = torch.tensor([0] + self.lens).cumsum(0).to(torch.int32).cuda() if n > 1 else None
        wide = torch.cat([self.x, torch.full((self.T, pad), math.nan, dtype=dtype)], 1).cuda()
        self.gx = wide[:, :self.C]
        self.how = dict(activation="silu" if silu else "none", norm=norm)
        self.ref = F.Conv(self.x, self.w, h_qk, self.b, self.state, self.lens, silu, norm)

    def dev(self, t):
        return None if t is None else t.cuda()

    def forward(self, **kw):
        return gdn.gdn_conv_fwd(self.gx, self.w.cuda(), self.h_qk, self.dev(self.b), self.dev(self.state), self.cu, **self.how, **kw)

    def check_forward(self, outs):
        for name, got, want, bound in zip("qkv", outs, self.ref.out, self.ref.bounds):
            F.check(name, got, want, bound, self.dtype)
        assert torch.equal(outs[3].double().cpu(), self.ref.last)

    def backward(self, **kw):
        return gdn.gdn_conv_bwd(self.gx, self.w.cuda(), self.h_qk, *[t.cuda() for t in self.d], self.dev(self.b), self.dev(self.state),
                                self.dev(self.d_final), self.cu, **self.how, **kw)

    def check_backward(self, grads, state_too=None):
        want, bound = self.ref.backward(*self.d, self.d_final)
        for i, (name, dt) in enumerate((("dx", self.dtype), ("d_weight", F32), ("d_bias", F32), ("d_state", self.dtype))):
            if (i == 2 and self.b is None) or (i == 3 and not (self.state is not None if state_too is None else state_too)):
                assert grads[i] is None
            else:
                F.check(name, grads[i], want[i], bound[i], dt)


CASES = [
    dict(lens=[1]), dict(lens=[2], state=True), dict(lens=[3], dtype=F32, width=2), dict(lens=[4], bias=True, width=3, state=True),
    dict(lens=[63]), dict(lens=[64], state=True), dict(lens=[65], dtype=F32, state=True), dict(lens=[700], h_qk=2, h_v=3, pad=16),
    dict(lens=[1, 2, 3, 4, 5, 6, 7, 8, 9], state=True, dtype=F32), dict(lens=[0, 5, 0, 0, 64, 1, 0], state=True),
    dict(lens=[1] * 40, state=True, width=3), dict(lens=[1] * 40, width=4), dict(lens=[2] * 33, width=4, state=True, bias=True, dtype=F32),
    dict(lens=[200, 1, 61, 8, 8, 8], h_qk=2, h_v=4, silu=False), dict(lens=[150, 3], norm=False, bias=True, pad=8),
    dict(lens=[31, 33], silu=False, norm=False, width=2, dtype=F32, state=True), dict(lens=[513], h_qk=3, h_v=1, width=2),
    dict(lens=[0, 0], state=True), dict(lens=[300, 500], size=20.0), dict(lens=[128], size=1e-3, dtype=F32),
    dict(lens=[2500, 100, 1], h_qk=4, h_v=8, state=True)]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward(i):
    c = Case(**CASES[i], seed=i)
    c.check_forward(c.forward())


@pytest.mark.parametrize("i", range(len(CASES)))
def test_backward(i):
    c = Case(**CASES[i], seed=200 + i)
    c.check_backward(c.backward())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_steps_continue_the_prompt(dtype, width):
    """Single tokens after a prompt: the outputs and states of one longer prompt, bit for bit."""
    c = Case([37, 1, 2, 9], 1, 2, dtype, width, bias=True, seed=width)
    whole = c.forward()
    begin = [0, 37, 38, 40]
    steps = [5, 0, 1, 3]
    first = [n - s for n, s in zip(c.lens, steps)]
    keep = torch.cat([torch.arange(b, b + f) for b, f in zip(begin, first)])
    cu = torch.tensor([0] + first).cumsum(0).to(torch.int32).cuda()
    q, k, v, state = gdn.gdn_conv_fwd(c.gx[keep], c.w.cuda(), c.h_qk, c.b.cuda(), None, cu)
    for got, want in zip((q, k, v), whole):
        assert torch.equal(got, want[keep.cuda()])
    for t in range(max(steps)):
        live = [i for i in range(4) if t < steps[i]]
        at = torch.tensor([begin[i] + first[i] + t for i in live]).cuda()
        s = state[live].contiguous()
        got = gdn.gdn_conv_step(c.gx[at], s, c.w.cuda(), c.h_qk, c.b.cuda())
        state[live] = s
        for g, want in zip(got, whole):
            assert torch.equal(g, want[at])
    assert torch.equal(state, whole[3])


@pytest.mark.parametrize("kw", [dict(), dict(dtype=F32, width=3, bias=True), dict(silu=False, norm=False, width=2), dict(h_qk=16, h_v=16)])
@pytest.mark.parametrize("n", [1, 5, 300])
def test_step(n, kw):
    c = Case([1] * n, **{**dict(h_qk=2, h_v=3), **kw}, state=True, pad=24, seed=n)
    state = c.state.cuda()
    outs = gdn.gdn_conv_step(c.gx, state, c.w.cuda(), c.h_qk, c.dev(c.b), **c.how)
    c.check_forward((*outs, state))


def test_pieces_of_a_prompt():
    """A long sequence in pieces through the kept state, the last shorter than the taps."""
    c = Case([411], 2, 2, seed=5)
    whole = c.forward()
    state, outs = None, []
    for a, b in ((0, 100), (100, 101), (101, 409), (409, 411)):
        *qkv, state = gdn.gdn_conv_fwd(c.gx[a:b], c.w.cuda(), c.h_qk, None, state)
        outs.append(qkv)
    for i in range(3):
        assert torch.equal(torch.cat([o[i] for o in outs]), whole[i])
    assert torch.equal(state, whole[3])


def test_batch_of_rows():
    """[B, T, C], also as part of a wider projection, against rows one by one."""
    g = torch.Generator().manual_seed(6)
    wide = torch.randn(3, 50, 512 + 64, generator=g).bfloat16().cuda()
    x, w = wide[..., :512], torch.randn(512, 4, generator=g).cuda()
    q, k, v, s = gdn.gdn_conv_fwd(x, w, 1)
    assert q.shape == (3, 50, 1, 128) and v.shape == (3, 50, 2, 128) and s.shape == (3, 3, 512)
    d = [torch.randn(t.shape, generator=g).bfloat16().cuda() for t in (q, k, v)]
    dx, dw, none, none_too = gdn.gdn_conv_bwd(x, w, 1, *d)
    assert none is None and none_too is None and dx.shape == x.shape
    for b in range(3):
        one = gdn.gdn_conv_fwd(x[b], w, 1)
        assert all(torch.equal(got[b], want) for got, want in zip((q, k, v), one)) and torch.equal(s[b], one[3][0])
        assert torch.equal(gdn.gdn_conv_bwd(x[b], w, 1, *[t[b] for t in d])[0], dx[b])


def test_gradient_of_a_state_of_zeros():
    c = Case([5, 2, 0, 70], dtype=F32, seed=9)
    c.check_backward(c.backward(want_initial_state_grad=True), True)
    assert c.backward(want_initial_state_grad=False)[3] is None


def test_given_outputs():
    """Outputs in given tensors; dx as part of a wider gradient whose rest stays; no final state."""
    c = Case([90, 7], 1, 1, seed=10)
    bufs = [torch.empty(97, 1, 128, dtype=BF16, device="cuda") for _ in range(3)]
    outs = c.forward(q=bufs[0], k=bufs[1], v=bufs[2], output_final_state=False)
    assert outs[3] is None and all(a is b for a, b in zip(outs, bufs))
    for name, got, want, bound in zip("qkv", outs, c.ref.out, c.ref.bounds):
        F.check(name, got, want, bound, BF16)
    wide = torch.full((97, 384 + 8), 3.0, dtype=BF16, device="cuda")
    c.check_backward(c.backward(dx=wide[:, :384]))
    assert (wide[:, 384:] == 3).all()


def test_tokens_outside_every_sequence():
    """A padded batch: rows before the first and behind the last sequence stay, and do not count."""
    c = Case([5, 0, 70, 2], dtype=F32, state=True, bias=True, seed=11)
    pad = lambda t: torch.cat([torch.full((3, *t.shape[1:]), math.nan), t, torch.full((66, *t.shape[1:]), math.nan)]).cuda()  # noqa: E731
    cu, T = c.cu + 3, 77 + 69
    bufs = [torch.full((T, h, 128), 9.0, device="cuda") for h in (1, 1, 2)]
    outs = gdn.gdn_conv_fwd(pad(c.x), c.w.cuda(), 1, c.b.cuda(), c.state.cuda(), cu, q=bufs[0], k=bufs[1], v=bufs[2])
    c.check_forward((*[t[3:80] for t in outs[:3]], outs[3]))
    dx = torch.full((T, c.C), 9.0, device="cuda")
    grads = gdn.gdn_conv_bwd(pad(c.x), c.w.cuda(), 1, *[pad(t) for t in c.d], c.b.cuda(), c.state.cuda(), c.d_final.cuda(), cu, dx=dx)
    c.check_backward((grads[0][3:80], *grads[1:]))
    for t in (*bufs, dx):
        assert (t[:3] == 9).all() and (t[80:] == 9).all()


def test_offsets_that_make_no_sense_stay_inside():
    """Offsets that go back or leave the batch: outputs undefined, nothing around the buffers written."""
    c = Case([64, 64], dtype=BF16, state=True, seed=12)
    for offsets in ([0, 200, 128], [0, 90, 50], [-5, 64, 128], [128, 64, 0], [0, 2 ** 31 - 1, -2 ** 31]):
        cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        guard = [torch.full((128 + 8, h, 128), 2.0, dtype=BF16, device="cuda") for h in (1, 1, 2)]
        state = torch.full((4, 3, c.C), 2.0, dtype=BF16, device="cuda")
        gdn.gdn_conv_fwd(c.gx, c.w.cuda(), 1, None, c.state.cuda(), cu, q=guard[0][4:132], k=guard[1][4:132], v=guard[2][4:132],
                         final_state=state[1:3])
        dx = torch.full((128 + 8, c.C), 2.0, dtype=BF16, device="cuda")
        gdn.gdn_conv_bwd(c.gx, c.w.cuda(), 1, *[t.cuda() for t in c.d], None, c.state.cuda(), c.d_final.cuda(), cu, dx=dx[4:132])
        torch.cuda.synchronize()
        for t in (*guard, dx):
            assert (t[:4] == 2).all() and (t[132:] == 2).all()
        assert (state[0] == 2).all() and (state[3] == 2).all()


@pytest.mark.parametrize("norm", [True, False])
def test_ends_of_the_range(norm):
    """Zeros, values whose squares pass fp32's range, and what is not finite stays in its channel or head."""
    c = Case([40], 1, 1, F32, norm=norm, bias=False, seed=13)
    x = c.x.clone()
    x[:10] = 0
    x[20:] *= 1e25
    ref = F.Conv(x, c.w, 1, None, None, [40], True, norm)
    outs = gdn.gdn_conv_fwd(x.cuda(), c.w.cuda(), 1, **c.how)
    for name, got, want, bound in zip("qkv", outs, ref.out, ref.bounds):
        F.check(name, got, want, bound)
    assert all((t[:7] == 0).all() for t in outs[:3])
    x = c.x.clone()
    x[8, 130] = math.nan
    x[9, 256 + 5] = math.inf
    q, k, v, _ = (t.cpu() for t in gdn.gdn_conv_fwd(x.cuda(), c.w.cuda(), 1, **c.how))
    assert not q.isnan().any() and not k[:8].isnan().any() and not k[12:].isnan().any()
    assert (k[8:12].isnan().all() if norm else k[8:12, 0, 2].isnan().all() and k[8:12].isnan().sum() == 4)
    assert v.isfinite().logical_not().nonzero()[:, 2].unique().tolist() == [5]


def test_gradients_against_differences():
    """The GPU's gradients along a direction against differences of the 64-bit forward."""
    c = Case([30, 2, 9], 1, 2, F32, bias=True, state=True, seed=14)
    g = torch.Generator().manual_seed(15)
    args = [c.x, c.w, c.b, c.state]
    dirs = [torch.randn(a.shape, generator=g).double() for a in args]

    def loss(t):
        x, w, b, s = (a.double() + t * d for a, d in zip(args, dirs))
        r = F.Conv(x, w, 1, b, s, c.lens)
        return float(sum((o * d.double()).sum() for o, d in zip(r.out, c.d)) + (r.last * c.d_final.double()).sum())

    terms = [got.double().cpu() * d for got, d in zip(c.backward(), dirs)]
    h = 1e-5
    slope = (loss(h) - loss(-h)) / (2 * h)
    # fp32 gradients to 2^-15 of what is summed (a sigmoid's slope is good to some 50 roundings); differences to h^2
    assert abs(slope - float(sum(t.sum() for t in terms))) <= float(sum(t.abs().sum() for t in terms)) * 2.0 ** -15 + 1e-3


def test_repeats_bit_for_bit():
    c = Case([3000, 50], 2, 2, bias=True, seed=16)
    size = gdn.gdn_conv_bwd_workspace_bytes(c.T, 2, 2, n_seqs=2)
    one, two = c.backward(), c.backward(workspace=torch.full((size,), 255, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(one[:3], two[:3]))


def test_refusals():
    c = Case([8], 1, 1, state=True, seed=17)
    w = c.w.cuda()
    for call in (lambda: gdn.gdn_conv_fwd(c.gx, w, 2), lambda: gdn.gdn_conv_fwd(c.gx, w[:, :2], 1),
                 lambda: gdn.gdn_conv_fwd(c.gx, w.bfloat16(), 1), lambda: gdn.gdn_conv_fwd(c.gx, w, 1, torch.zeros(3, device="cuda")),
                 lambda: gdn.gdn_conv_fwd(c.gx, w, 1, None, c.state.float().cuda()),
                 lambda: gdn.gdn_conv_fwd(c.gx, w, 1, None, None, torch.tensor([0, 8], device="cuda")),
                 lambda: gdn.gdn_conv_fwd(c.gx, w, 1, q=torch.empty(8, 1, 128, device="cuda")),
                 lambda: gdn.gdn_conv_fwd(c.gx, w, 1, activation="relu"),
                 lambda: gdn.gdn_conv_bwd(c.gx, w, 1, c.d[0].cuda(), c.d[1].cuda(), c.d[0].float().cuda()),
                 lambda: gdn.gdn_conv_step(c.gx, c.state.cuda(), w, 1), lambda: gdn.gdn_conv_step(c.gx, None, w, 1)):
        with pytest.raises(ValueError):
            call()
    s = c.state.cuda()
    with pytest.raises(gdn.api.L.GDNError):
        gdn.gdn_conv_fwd(c.gx, w, 1, None, s, final_state=s)      # the states may not overlap
    with pytest.raises(gdn.api.L.GDNError):
        gdn.gdn_conv_bwd(c.gx, w, 1, *[t.cuda() for t in c.d], dx=c.gx)
