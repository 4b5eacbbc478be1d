"""The append that normalises and rotates keys on the way, and the queries beside
them, against the 64-bit forms of both halves."""
from __future__ import annotations

import math

import pytest
import torch

from tests import front_util as F
from tests import kv_util as K

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU, skipped there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_deltanet_linear_fwd_gb300 as gdn  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class Case:
    def __init__(self, q_lens, kv_lens, h_q, h_kv, dtype=BF16, layout="half", rot=128, norm="rms", weights=True, strided=True, seed=0,
                 use_cu=True, **scaling):
        self.b = b = K.Batch(q_lens, kv_lens, h_kv, seed=seed, spread=0.5)
        b.fill(stale_nan=False)
        self.h_q, self.dtype, self.layout, self.rot, self.norm = h_q, dtype, layout, rot, norm
        grow = lambda *s: b.randn(*s) * torch.exp(0.5 * b.randn(s[0], s[1], 1))  # noqa: E731
        self.q, self.k, self.v = (grow(b.T, h, 128).to(dtype) for h in (h_q, h_kv, h_kv))
        self.qw = 1 + 0.3 * b.randn(128) if weights and norm != "none" else None
        self.kw = 1 + 0.3 * b.randn(128) if weights and norm != "none" else None
        self.mag = scaling.pop("magnitude", 1.0)
        self.freqs = F.frequencies(rot, **scaling)
        self.rope = gdn.gdn_rope_table(rot, layout=layout, magnitude=self.mag, **scaling)
        self.pos = torch.cat([torch.arange(kv - n, kv) for n, kv in zip(q_lens, kv_lens)])
        code = lambda c: c.float().to(torch.float8_e4m3fn).cuda()  # noqa: E731
        self.cache = gdn.KVCache(code(b.k), code(b.v), b.ks.float().cuda(), b.vs.float().cuda())
        if strided:
            x = torch.cat([self.q, self.k, self.v], 1).cuda()
            self.gq, self.gk, self.gv = x.split([h_q, h_kv, h_kv], dim=1)
        else:
            self.gq, self.gk, self.gv = self.q.cuda(), self.k.cuda(), self.v.cuda()
        self.cu = b.cu.cuda() if use_cu else None
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.how = dict(rope=self.rope, norm=norm, k_weight=dev(self.kw))
        self.q_how = dict(q=self.gq, q_weight=dev(self.qw))

    def call(self, **kw):
        return gdn.gdn_kv_append_rope(self.cache, self.gk, self.gv, self.b.lens.cuda(), self.b.table.cuda(), self.cu,
                                      **{**self.how, **self.q_how, **kw})

    def check(self, q_out):
        """Scales are equal, codes too but where a key is as near to the middle between
        two codes as fp32 may move it; rows that no token is in stay as they were."""
        assert gdn.gdn_get_device_status(self.cache.status) == (0, 0)
        want_q, bq = F.rope_ref(self.q, self.pos, self.freqs, self.layout, self.mag, self.norm, self.qw)
        if q_out is not None:
            F.check("q", q_out, want_q, bq, self.dtype)
        k64, bk = F.rope_ref(self.k, self.pos, self.freqs, self.layout, self.mag, self.norm, self.kw)
        # A key's cosine and sine are products of two rotations', cos a cos b - sin a sin b: each factor to
        # 4 + 1.6 roundings, as there the one, and two more for product and sum: 8 of them beside its 19.
        bk = bk * (27 / 19)
        ck, sk, cv, sv = K.append_ref(self.b, k64, self.v)
        assert torch.equal(self.cache.v_scale.double().cpu(), sv)
        assert torch.equal(self.cache.v.float().double().cpu(), cv)
        got_s = self.cache.k_scale.double().cpu()
        assert torch.equal(got_s, sk)
        got = self.cache.k.float().double().cpu()
        lo, *_ = K.append_ref(self.b, k64 - bk, self.v)[:1]
        hi, *_ = K.append_ref(self.b, k64 + bk, self.v)[:1]
        ok = (got == ck) | (got == lo) | (got == hi)
        assert ok.all()
        assert (got != ck).float().mean() < 1e-3


CASES = [
    dict(q_lens=[1], kv_lens=[1], h_q=4, h_kv=2), dict(q_lens=[1], kv_lens=[64], h_q=4, h_kv=2), dict(q_lens=[1], kv_lens=[65], h_q=1, h_kv=1),
    dict(q_lens=[1, 1, 1, 1], kv_lens=[5, 64, 129, 1000], h_q=8, h_kv=2, use_cu=False),
    dict(q_lens=[1, 1, 1, 1], kv_lens=[5, 64, 129, 1000], h_q=3, h_kv=3, dtype=F32, use_cu=False, layout="interleaved"),
    dict(q_lens=[200], kv_lens=[200], h_q=4, h_kv=2), dict(q_lens=[130, 0, 7, 64], kv_lens=[130, 77, 100, 128], h_q=6, h_kv=2),
    dict(q_lens=[63, 65, 1], kv_lens=[127, 65, 333], h_q=2, h_kv=1, dtype=F32, rot=64, layout="interleaved", norm="unit"),
    dict(q_lens=[100], kv_lens=[5000], h_q=8, h_kv=4, norm="none", rot=32, strided=False),
    dict(q_lens=[40, 3], kv_lens=[41, 900], h_q=8, h_kv=8, weights=False, scaling="parts", factor=8.0, original_len=512.0, magnitude=1.2),
    dict(q_lens=[5] * 6, kv_lens=[5, 66, 64, 69, 300, 128], h_q=4, h_kv=1, use_cu=False, dtype=F32, rot=8),
    dict(q_lens=[1] * 70, kv_lens=list(range(1, 71)), h_q=2, h_kv=2, use_cu=False),
    dict(q_lens=[1] * 70, kv_lens=list(range(1, 71)), h_q=5, h_kv=1, use_cu=True)]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_append(i):
    c = Case(**CASES[i], seed=i)
    c.check(c.call())


@pytest.mark.parametrize("i", [2, 5, 8])
def test_without_queries(i):
    c = Case(**CASES[i], seed=50 + i)
    assert c.call(q=None, q_weight=None) is None
    c.check(None)


def test_queries_in_place():
    c = Case([33, 70], [33, 500], 4, 2, seed=60)
    k, v = c.gk.clone(), c.gv.clone()
    out = c.call(q_out=c.gq)
    assert out is c.gq and torch.equal(c.gk, k) and torch.equal(c.gv, v)
    c.check(out)


def test_nothing_turned_is_the_append():
    """Without norm and rotation: gdn_kv_append bit for bit, and queries copied."""
    for use_cu in (True, False):
        a, b = (Case([1] * 5, [1, 64, 65, 200, 130], 4, 2, norm="none", seed=61, use_cu=use_cu) for _ in range(2))
        out = a.call(rope=None)
        gdn.gdn_kv_append(b.cache, b.gk, b.gv, b.b.lens.cuda(), b.b.table.cuda(), b.cu)
        assert torch.equal(out, a.gq)
        for name in ("k", "v", "k_scale", "v_scale"):
            x, y = getattr(a.cache, name), getattr(b.cache, name)
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("grow", [False, True])
def test_token_by_token(dtype, grow):
    """Tokens one at a time over page ends, scales growing or not: each against the form on the cache before it."""
    c = Case([1, 1], [60, 127], 4, 2, dtype, seed=62, use_cu=False, norm="none" if grow else "rms")
    for t in range(8):
        lens = [60 + t, 127 + t]
        n = Case([1, 1], lens, 4, 2, dtype, seed=63 + t, use_cu=False, norm="none" if grow else "rms")
        n.b.table, n.b.n_pages = c.b.table, c.b.n_pages
        if t == 0:
            cache = n.cache
            pages = torch.zeros(2, 4, dtype=torch.int32)
            pages[0, :3], pages[1, :4] = torch.tensor([0, 1, 2]), torch.tensor([3, 4, 5, 6])
            pool = 7
            g = torch.Generator().manual_seed(0)
            codes = K.e4m3(torch.randn(pool, 2, 64, 128, generator=g) * 100).float()
            cache = gdn.KVCache(codes.to(torch.float8_e4m3fn).cuda(), codes.to(torch.float8_e4m3fn).cuda(),
                                torch.full((pool, 2), 2.0 ** -8, device="cuda"), torch.full((pool, 2), 2.0 ** -8, device="cuda"))
        n.b.table, n.b.n_pages = pages, pool
        if grow:
            n.gk, n.k = n.gk * 2.0 ** t, n.k * 2.0 ** t
        n.b.k, n.b.ks = cache.k.float().cpu(), cache.k_scale.cpu()
        n.b.v, n.b.vs = cache.v.float().cpu(), cache.v_scale.cpu()
        n.cache = cache
        n.check(n.call())


@pytest.mark.parametrize("n", [2, 3, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_tokens_each(n, dtype):
    """The same number of new tokens in every sequence, whole, across page ends, in an idle slot, with earlier rows that stay
    or follow a scale that grows."""
    kv = [n, n + 1, 63 + n, 64, 65 + n // 2, 64 + n, 128, 129, 300]
    for norm, size in (("rms", 1.0), ("none", 40.0), ("none", 1e-3)):
        c = Case([n] * len(kv), kv, 3, 2, dtype, seed=80 + n, use_cu=False, norm=norm, layout="interleaved" if n % 2 else "half", rot=96)
        c.k, c.v = (c.k.float() * size).to(dtype), (c.v.float() * size).to(dtype)
        c.gk, c.gv = c.k.cuda(), c.v.cuda()
        c.check(c.call())
    c = Case([n] * 3, [70, n, n], 2, 1, dtype, seed=81, use_cu=False)
    lens = torch.tensor([70, n - 1, 0], dtype=torch.int32, device="cuda")  # a token before position 0; an idle slot
    before = c.cache.k.clone()
    c.call(q=None, q_weight=None)
    whole = c.cache.k.view(torch.uint8).clone()
    c.cache.k.copy_(before)
    gdn.gdn_kv_append_rope(c.cache, c.gk, c.gv, lens, c.b.table.cuda(), **c.how)
    one, idle = int(c.b.table[1, 0]), int(c.b.table[2, 0])
    got = c.cache.k.view(torch.uint8)
    assert torch.equal(got[idle], before.view(torch.uint8)[idle]) and torch.equal(got[one, :, n:], whole[one, :, n:])
    assert gdn.gdn_get_device_status(c.cache.status) == (0, 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mean", [4, 8])
def test_few_tokens_with_offsets(dtype, mean):
    """Mostly single tokens, a few long pieces over several pages among them, empty sequences, tokens behind the last one."""
    q = [1, 0, 2, 70, 1, 1, 5, 0, 1, 9, 1] + [1] * 20 + [0, 3, 17, 64, 0]
    q += [1] * max(0, -((mean * len(q) - sum(q) - 3) // (mean - 1)))
    kv = [max(n, 1) + (37 * i) % 200 for i, n in enumerate(q)]
    kv[3], kv[-1] = 70, 65
    assert sum(q) + 3 <= mean * len(q)
    for norm, size, layout in (("rms", 1.0, "half"), ("unit", 1.0, "interleaved"), ("none", 50.0, "half")):
        c = Case(q, kv, 3, 2, dtype, seed=90 + mean, norm=norm, layout=layout, weights=norm == "rms")
        c.k = (c.k.float() * size).to(dtype)
        pad = lambda t: torch.cat([t, torch.full((3, *t.shape[1:]), math.nan, dtype=t.dtype)]).cuda()  # noqa: E731
        c.gk, c.gv = pad(c.k), pad(c.v)
        out = torch.full((c.b.T + 3, 3, 128), 6.0, dtype=dtype, device="cuda")
        c.call(q=pad(c.q), q_out=out)
        assert (out[c.b.T:] == 6).all()
        c.check(out[:c.b.T])
    lens = c.b.lens.clone()
    lens[1] = -5   # a sequence without tokens
    gdn.gdn_kv_append_rope(c.cache, c.gk, c.gv, lens.cuda(), c.b.table.cuda(), c.cu, **c.how)
    assert gdn.gdn_get_device_status(c.cache.status) == (7, 7)
    for bad in ([0] * len(q) + [sum(q)], [0, 5, 3] + c.b.cu.tolist()[3:], [0] + [2 ** 30] * len(q), [-4] + c.b.cu.tolist()[1:]):
        c.cache.status.zero_()   # offsets that leave the call or go back: no access leaves the buffers
        gdn.gdn_kv_append_rope(c.cache, c.gk, c.gv, c.b.lens.cuda(), c.b.table.cuda(),
                               torch.tensor(bad, dtype=torch.int32, device="cuda"), **c.how)
        torch.cuda.synchronize()


@pytest.mark.parametrize("use_cu", [True, False])
def test_not_finite_keys(use_cu):
    """They become NaN codes (their whole head under a norm, but for an infinity's) and do not count in the scale."""
    c = Case([3], [3], 2, 2, F32, norm="none", seed=70, use_cu=use_cu)
    c.k[0, 0, 5] = math.inf
    c.k[1, 1, 100] = math.nan
    c.gk = c.k.cuda()
    c.call(q=None)
    codes = c.cache.k.float().cpu()[int(c.b.table[0, 0])]
    assert codes[0, 0].isnan().nonzero().flatten().tolist() == [5, 69] and codes[1, 1].isnan().nonzero().flatten().tolist() == [36, 100]
    fin = torch.where(c.k.isfinite(), c.k, torch.zeros_like(c.k))
    turned = F.turn(fin.double(), c.pos, c.freqs, "half")
    turned[0, 0, [5, 69]] = 0
    turned[1, 1, [36, 100]] = 0
    for h in range(2):
        assert float(c.cache.k_scale[int(c.b.table[0, 0]), h]) == 2.0 ** K.scale_exp(float(turned[:, h].abs().max()))
    c = Case([2], [2], 2, 1, F32, norm="rms", weights=False, seed=71, use_cu=use_cu)
    c.k[0, 0, 5] = math.nan
    c.gk = c.k.cuda()
    c.call(q=None)
    codes = c.cache.k.float().cpu()[int(c.b.table[0, 0])]
    assert codes[0, 0].isnan().all() and not codes[0, 1].isnan().any()


def test_idle_slots_and_bad_lengths():
    """kv_lens[i] < n_i stores nothing of the tokens before position 0; lengths and pages out of bounds are reported."""
    c = Case([1, 1, 1], [30, 1, 2], 2, 1, seed=72, use_cu=False)
    before = [t.clone() for t in (c.cache.k.view(torch.uint8), c.cache.k_scale)]
    lens = torch.tensor([30, 0, 2], dtype=torch.int32, device="cuda")
    gdn.gdn_kv_append_rope(c.cache, c.gk, c.gv, lens, c.b.table.cuda(), **c.how, **c.q_how)
    assert gdn.gdn_get_device_status(c.cache.status) == (0, 0)
    idle = int(c.b.table[1, 0])
    assert torch.equal(c.cache.k.view(torch.uint8)[idle], before[0][idle]) and c.cache.k_scale[idle] == before[1][idle]
    for bad_lens, table, detail in (([30, 10 ** 6, 2], c.b.table, 7), ([30, -1, 2], c.b.table, 7), ([30, 1, 2], c.b.table + 1000, 8)):
        c.cache.status.zero_()
        gdn.gdn_kv_append_rope(c.cache, c.gk, c.gv, torch.tensor(bad_lens, dtype=torch.int32, device="cuda"), table.cuda(), **c.how,
                               **c.q_how)
        assert gdn.gdn_get_device_status(c.cache.status) == (7, detail)


def test_queries_behind_the_last_sequence():
    c = Case([3, 4], [3, 100], 4, 2, seed=73)
    pad = lambda t: torch.cat([t, torch.full((5, *t.shape[1:]), math.nan, dtype=t.dtype)]).cuda()  # noqa: E731
    out = torch.full((12, 4, 128), 6.0, dtype=BF16, device="cuda")
    c.gk, c.gv = pad(c.k), pad(c.v)
    c.call(q=pad(c.q), q_out=out)
    assert (out[7:] == 6).all()
    c.check(out[:7])


def test_refusals():
    c = Case([4], [4], 2, 1, seed=74)
    for bad in (dict(q=c.gq[:2]), dict(q=c.gq.float()), dict(q_out=c.gq.float()), dict(q=None, q_out=c.gq, q_weight=None), dict(norm="max"),
                dict(k_weight=torch.ones(128)), dict(rope=gdn.gdn_rope_table(128, device="cpu"))):
        with pytest.raises(ValueError):
            c.call(**bad)
    with pytest.raises(gdn.api.L.GDNError):
        c.call(norm="none")       # weights without a norm
    with pytest.raises(gdn.api.L.GDNError):
        c.call(eps=-1.0)
