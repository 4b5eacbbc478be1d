"""The 8-bit key/value cache on the GPU: append, read and attention against
plain 64-bit forms, where lengths, masks, strides and contents can go wrong."""
from __future__ import annotations

import math

import pytest
import torch

from tests import kv_util as U

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_linear_fwd_gb300 as g
    return g


def to_cache(gdn, b):
    dev = lambda c: c.float().to(torch.float8_e4m3fn).cuda()  # noqa: E731
    return gdn.KVCache(dev(b.k), dev(b.v), b.ks.float().cuda(), b.vs.float().cuda())


def status(gdn, cache):
    return gdn.gdn_get_device_status(cache.status)


def same(a, ref):
    """Equal values, NaN where the reference has NaN."""
    a, ref = a.double().cpu(), ref.double()
    return torch.equal(a.isnan(), ref.isnan()) and torch.equal(a.nan_to_num(), ref.nan_to_num())


# ---------------------------------------------------------------- append
APPEND = {
    "one_token_new_page": ([1], [1], 1),
    "one_token_mid_page": ([1, 1, 1, 1], [2, 64, 65, 130], 2),
    "idle_and_empty": ([1, 1, 1], [0, 5, 0], 2),
    "pieces": ([70, 0, 1, 200, 3], [70, 9, 77, 333, 66], 3),
    "page_exact": ([64, 128], [64, 192], 1),
    "cut_at_zero": ([10, 80], [4, 66], 2),
    "many": ([1 + i % 3 for i in range(300)], [3 + 7 * i % 200 for i in range(300)], 2),
}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", list(APPEND))
def test_append(gdn, name, dtype):
    q, kv, h = APPEND[name]
    b = U.Batch(q, kv, h, seed=len(name))
    b.fill(stale_nan=False)
    k, v = (b.randn(b.T, h, 128).mul(2.0 ** (3 * i)).to(dtype) for i in (-1, 1))
    cache = to_cache(gdn, b)
    gdn.gdn_kv_append(cache, k.cuda(), v.cuda(), b.lens.cuda(), b.table.cuda(), b.cu.cuda())
    ref = U.append_ref(b, k, v)
    for got, want in zip((cache.k, cache.k_scale, cache.v, cache.v_scale), ref):
        assert same(got.float(), want)
    assert status(gdn, cache) == (0, 0)
    if min(q) == max(q):  # the same without offsets
        other = to_cache(gdn, b)
        gdn.gdn_kv_append(other, k.cuda(), v.cuda(), b.lens.cuda(), b.table.cuda())
        assert torch.equal(other.k.view(torch.uint8), cache.k.view(torch.uint8))
        assert torch.equal(other.v_scale, cache.v_scale)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_values(gdn, dtype):
    """Scale edges: zeros, the largest a at each power of two, subnormal codes, saturation, inf and NaN."""
    rows = [torch.zeros(128), torch.full((128,), 448.0), torch.full((128,), 449.0 if dtype == F32 else 450.0),
            torch.linspace(-448, 448, 128), 2.0 ** torch.linspace(-60, -30, 128), 2.0 ** torch.linspace(30, 60, 128),
            torch.full((128,), 1e-45), torch.tensor([math.inf, -math.inf, math.nan, 1.0] * 32),
            torch.full((128,), math.nan), torch.tensor([3.5 * 2.0 ** -7, -1.75] * 64), torch.arange(128) * 2.0 ** -9,
            (torch.arange(128) + 0.5) * 2.0 ** -9]
    n = len(rows)
    b = U.Batch([1] * n, [1] * n, 1)
    b.fill(stale_nan=False)
    k = torch.stack(rows).view(n, 1, 128).to(dtype)
    cache = to_cache(gdn, b)
    gdn.gdn_kv_append(cache, k.cuda(), (2 * k).cuda(), b.lens.cuda(), b.table.cuda())
    ref = U.append_ref(b, k, 2 * k)
    for got, want in zip((cache.k, cache.k_scale, cache.v, cache.v_scale), ref):
        assert same(got.float(), want)


def test_append_token_by_token(gdn):
    """Writing token by token with growing magnitudes re-encodes earlier codes; the values stay those of one scale."""
    n = 150
    b = U.Batch([n], [n], 2, seed=3)
    b.fill(stale_nan=False)
    k = b.randn(n, 2, 128) * torch.linspace(0.01, 8, n)[:, None, None]
    v = b.randn(n, 2, 128) * torch.linspace(8, 0.01, n)[:, None, None]
    once, step = to_cache(gdn, b), to_cache(gdn, b)
    table = b.table.cuda()
    gdn.gdn_kv_append(once, k.cuda(), v.cuda(), b.lens.cuda(), table)
    for t in range(n):
        gdn.gdn_kv_append(step, k[t:t + 1].cuda(), v[t:t + 1].cuda(), torch.tensor([t + 1], dtype=torch.int32).cuda(), table)
    assert torch.equal(once.k_scale, step.k_scale) and torch.equal(once.v_scale, step.v_scale)
    # a code can be rounded twice only below the normal range: then by at most one more subnormal step
    pages = b.table[0].long().cuda()
    diff = (once.k.float() - step.k.float()).abs()[pages]
    assert diff.max() <= 2.0 ** -9
    assert torch.equal(once.k.float()[pages][diff == 0], step.k.float()[pages][diff == 0])


def test_append_strided_and_stream(gdn):
    b = U.Batch([5, 130], [69, 130], 2, seed=5)
    b.fill(stale_nan=False)
    wide = b.randn(b.T, 9, 128).to(BF)
    k, v = wide[:, 4:6], wide[:, 7:9]
    cache = to_cache(gdn, b)
    dev, lens, table, cu = wide.cuda(), b.lens.cuda(), b.table.cuda(), b.cu.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gdn.gdn_kv_append(cache, dev[:, 4:6], dev[:, 7:9], lens, table, cu)
    s.synchronize()
    for got, want in zip((cache.k, cache.k_scale, cache.v, cache.v_scale), U.append_ref(b, k, v)):
        assert same(got.float(), want)


# ---------------------------------------------------------------- read
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q,kv,h", [([1], [1], 1), ([64, 65, 200, 0], [64, 65, 333, 7], 3), ([3, 5], [0, 2], 2),
                                    ([40] * 70, [40 + i for i in range(70)], 1)])
def test_read(gdn, q, kv, h, dtype):
    b = U.Batch(q, kv, h, seed=11)
    b.fill()
    cache = to_cache(gdn, b)
    k, v = gdn.gdn_kv_read(cache, b.lens.cuda(), b.table.cuda(), b.cu.cuda(), T=b.T, dtype=dtype)
    for got, which in ((k, "k"), (v, "v")):
        want = torch.zeros(b.T, h, 128, dtype=torch.float64)
        for i, (n, m) in enumerate(zip(q, kv)):
            t = b.tokens(which, i)[max(m - n, 0):]
            e = int(b.cu[i + 1])
            want[e - t.shape[0]:e] = t
        assert same(got, want)  # exact in either type


# ---------------------------------------------------------------- attention
def check_attn(gdn, b, h_q, dtype, causal=True, window=0, scale=0.0, q=None, use_cu=True, **kw):
    q = (b.randn(b.T, h_q, 128) if q is None else q).to(dtype)
    cache = to_cache(gdn, b)
    cu = b.cu.cuda() if use_cu else None
    out, lse = gdn.gdn_kv_attn(q.cuda(), cache, b.lens.cuda(), b.table.cuda(), cu, causal=causal, window=window,
                               scale=scale, **kw)
    assert status(gdn, cache) == (0, 0)
    o, z, mass, reach, top = U.attn_ref(b, q, causal, window, scale)
    bo, bz = U.attn_bounds(o, mass, reach, top, dtype)
    got, got_z = out.double().cpu(), lse.double().cpu()
    empty = z == -math.inf
    assert torch.equal(got_z == -math.inf, empty)
    assert (got[empty] == 0).all()
    nan = o.isnan().any(-1) | z.isnan()
    assert torch.equal(got.isnan().any(-1), nan)
    ok = ~nan
    err = ((got - o).abs() / bo)[ok]
    assert err.numel() == 0 or err.max() <= 1, f"out: {err.max():.3f} of the bound"
    ez = ((got_z - z).abs() / bz)[ok & ~empty]
    assert ez.numel() == 0 or ez.max() <= 1, f"lse: {ez.max():.3f} of the bound"
    return out, lse


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (8, 2), (3, 2), (16, 16), (12, 1), (7, 3)])
@pytest.mark.parametrize("kv", [1, 63, 64, 65, 127, 128, 129, 600, 1290])
def test_attn_one_token(gdn, kv, h_q, h_kv, dtype):
    b = U.Batch([1], [kv], h_kv, seed=kv + h_q)
    b.fill()
    check_attn(gdn, b, h_q, dtype)


BATCHES = {
    "decode_ragged": ([1] * 9, [1, 700, 64, 0, 65, 333, 2000, 128, 5], 8, 2),
    "decode_many": ([1] * 200, [1 + 37 * i % 900 for i in range(200)], 4, 1),
    "decode_long": ([1, 1], [20000, 9000], 8, 2),
    "draft": ([5, 5, 5], [5, 133, 1000], 16, 4),
    "draft_long": ([4], [9001], 8, 1),
    "mixed": ([1, 7, 0, 130, 1], [300, 7, 50, 500, 64], 8, 2),
    "group_40": ([2, 3], [70, 200], 40, 1),
    "prompt": ([200, 333], [200, 333], 8, 2),
    "piece": ([257], [1500], 6, 2),
    "piece_odd_heads": ([129, 64], [129, 1000], 7, 3),
    "rows_one_head": ([300, 1], [300, 700], 2, 2),
    "short_lens": ([6, 3, 2], [3, 0, 2], 4, 2),
    "prompt_long": ([1100], [4200], 4, 1),
}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mask", ["causal", "full", "window", "window_full"])
@pytest.mark.parametrize("name", list(BATCHES))
def test_attn(gdn, name, mask, dtype):
    q, kv, h_q, h_kv = BATCHES[name]
    if name == "prompt_long" and (dtype == F32 or mask == "window_full"):
        pytest.skip("the long prompt runs in bf16 under three masks")
    b = U.Batch(q, kv, h_kv, seed=len(name) + h_q)
    b.fill()
    check_attn(gdn, b, h_q, dtype, causal=mask in ("causal", "window"), window=100 if "window" in mask else 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("n,group", [(2, 4), (3, 3), (1, 16), (17, 1), (5, 4), (6, 4), (5, 5), (31, 1), (8, 4), (11, 3)])
def test_attn_row_counts(gdn, n, group, window, dtype):
    """Rows that share a key, either side of 8, 16, 24 and 32; lengths of one tile, of odd and of even
    numbers of tiles, ending inside, at and just past one; a sequence cut between CTAs."""
    b = U.Batch([n] * 7, [n, 128, 129, 300, 384, 513, 6000], 2, seed=n + group)
    b.fill()
    check_attn(gdn, b, 2 * group, dtype, window=window)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_on_another_stream(gdn, dtype):
    """On a stream of the caller's, with outputs and workspace from the call."""
    b = U.Batch([1, 3, 200], [900, 5000, 2000], 2, seed=4)
    b.fill()
    cache, q = to_cache(gdn, b), b.randn(b.T, 8, 128).to(dtype).cuda()
    lens, table, cu = b.lens.cuda(), b.table.cuda(), b.cu.cuda()
    want = gdn.gdn_kv_attn(q, cache, lens, table, cu)
    kept = gdn.gdn_kv_read(cache, lens, table, cu, T=b.T, dtype=dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = gdn.gdn_kv_attn(q, cache, lens, table, cu, stream=side)
        read = gdn.gdn_kv_read(cache, lens, table, cu, T=b.T, dtype=dtype, stream=side)
        torch.empty(32 << 20, dtype=torch.uint8, device="cuda").fill_(255)  # takes what the current stream has free
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((*got, *read), (*want, *kept)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_sharp_and_flat(gdn, dtype):
    """Scores from far below to far above the others: one key takes all the weight, and none does."""
    b = U.Batch([1, 1, 40], [500, 500, 500], 2, seed=9, spread=0.2)
    b.fill()
    q = b.randn(b.T, 4, 128)
    q[0] *= 200.0
    q[1] = 0.0
    q[2:20] *= 1e-20
    q[30] *= 1e4
    check_attn(gdn, b, 4, dtype, q=q)
    check_attn(gdn, b, 4, dtype, q=b.randn(b.T, 4, 128), scale=0.5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 3, 150])
def test_attn_scales_far_apart(gdn, dtype, n):
    """Pages whose scales differ by many powers of two, pages of zeros among them."""
    b = U.Batch([n], [700], 1, seed=n)
    b.fill()
    e = torch.tensor([0, -40, 12, -9, 3, -20, 20, -3, 0, 1, -1, 5])[: len(b.table[0])].double()
    for slot, x in enumerate(e.tolist()):
        b.vs[b.table[0, slot].long()] *= 2.0 ** max(min(x, 20.0), -20.0)
        b.ks[b.table[0, slot].long()] *= 2.0 ** max(min(x / 8, 2.0), -20.0)
    b.v[b.table[0, 1].long()] = 0.0
    b.vs[b.table[0, 1].long()] = 2.0 ** -40
    b.ks = torch.pow(2.0, torch.round(torch.log2(b.ks)))
    check_attn(gdn, b, 4, dtype)


@pytest.mark.parametrize("n", [1, 3, 9])
def test_attn_one_key_against_many(gdn, n):
    """One key with a weight 2^20 times the others', half a million of which together outweigh it."""
    kv = 500_000
    b = U.Batch([n], [kv], 1, seed=n)
    pages = b.table[0].long()
    b.k, b.ks = torch.zeros(b.n_pages, 1, 64, 128), torch.ones(b.n_pages, 1)
    b.v, b.vs = torch.zeros(b.n_pages, 1, 64, 128), torch.ones(b.n_pages, 1)
    b.v[pages] = 1.0
    b.v[pages[0], 0, 0] = -1.0
    q = torch.zeros(n, 4, 128)
    q[..., 0] = 1.0
    q[..., 1] = 0.5  # not a single e4m3 part of its row
    b.k[pages[0], 0, 0, 0] = 1.0
    scale = 20 * math.log(2.0)
    rest = kv - n + torch.arange(n)  # keys besides the first that row t sees
    w0 = 2.0 ** 20 / (2.0 ** 20 + rest.double())
    cache = to_cache(gdn, b)
    out, lse = gdn.gdn_kv_attn(q.to(BF).cuda(), cache, b.lens.cuda(), b.table.cuda(), scale=scale)
    want = (1 - 2 * w0)[:, None, None]
    # two bf16 roundings of weights and output, relative to the weights' sum of one
    assert (out.double().cpu() - want).abs().max() <= 2.0 ** -7
    assert (lse.double().cpu() - torch.log(2.0 ** 20 + rest.double())[:, None]).abs().max() <= 2.0 ** -14


@pytest.mark.parametrize("n", [1, 3, 9, 100])
def test_attn_weights_far_below_the_largest(gdn, n):
    """The largest weight's value is zero, and the others, 2^-12.3 of it, make the output: each still has
    eight bits, and the output's rounding is one more of nine."""
    kv = 1000
    b = U.Batch([n], [kv], 1, seed=n)
    pages = b.table[0].long()
    b.k, b.ks = torch.zeros(b.n_pages, 1, 64, 128), torch.ones(b.n_pages, 1)
    b.v, b.vs = torch.zeros(b.n_pages, 1, 64, 128), torch.ones(b.n_pages, 1)
    b.v[pages] = 1.0
    b.v[pages[0], 0, 0] = 0.0
    b.k[pages[0], 0, 0, 0] = 1.0
    q = torch.zeros(n, 4, 128)
    q[..., 0] = 1.0
    out, _ = gdn.gdn_kv_attn(q.to(BF).cuda(), to_cache(gdn, b), b.lens.cuda(), b.table.cuda(), scale=12.3 * math.log(2.0))
    w = (kv - n + torch.arange(n)).double() * 2.0 ** -12.3
    want = (w / (1 + w))[:, None, None]
    assert ((out.double().cpu() - want).abs() / want).max() <= 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -12


def test_attn_f32_one_key_against_many(gdn):
    """The same in fp32, to a rounding a tile: 3907 tiles of 2^-24, and 2^-22 of the exponential."""
    kv = 500_000
    b = U.Batch([1], [kv], 1, seed=1)
    pages = b.table[0].long()
    b.k, b.ks = torch.zeros(b.n_pages, 1, 64, 128), torch.ones(b.n_pages, 1)
    b.v, b.vs = torch.zeros(b.n_pages, 1, 64, 128), torch.ones(b.n_pages, 1)
    b.v[pages] = 1.0
    b.v[pages[0], 0, 0] = -1.0
    q = torch.zeros(1, 4, 128)
    q[..., 0] = 1.0
    q[..., 1] = 1 / 3
    b.k[pages[0], 0, 0, 0] = 1.0
    out, lse = gdn.gdn_kv_attn(q.cuda(), to_cache(gdn, b), b.lens.cuda(), b.table.cuda(), scale=20 * math.log(2.0))
    w0 = 2.0 ** 20 / (2.0 ** 20 + kv - 1)
    assert (out.double().cpu() - (1 - 2 * w0)).abs().max() <= 2.0 ** -11
    assert (lse.double().cpu() - math.log(2.0 ** 20 + kv - 1)).abs().max() <= 2.0 ** -11


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,window", [(1, 64), (5, 0), (5, 70), (200, 0), (300, 33)])
def test_attn_nan_outside_masks(gdn, dtype, n, window):
    """Keys and values that no row may use, NaN in both, change nothing; a row that may use one is NaN."""
    b = U.Batch([n], [450], 2, seed=n)
    b.fill()
    def poison(pos):
        page = int(b.table[0, pos // 64])
        b.k[page, :, pos % 64] = math.nan
        b.v[page, :, pos % 64] = math.nan
    if window:
        first = 450 - n - window  # the last position outside every window
        poison(first)
        poison(0)
    else:
        poison(449)  # the last token's own: only the last row sees it
    q = b.randn(b.T, 4, 128).to(dtype)
    cache = to_cache(gdn, b)
    out, lse = gdn.gdn_kv_attn(q.cuda(), cache, b.lens.cuda(), b.table.cuda(), window=window)
    o, z, mass, reach, top = U.attn_ref(b, q, True, window)
    bo, _ = U.attn_bounds(o, mass, reach, top, dtype)
    rows = slice(0, n if window else n - 1)
    assert not out[rows].isnan().any() and not lse[rows].isnan().any()
    assert (((out.double().cpu() - o).abs() / bo)[rows]).nan_to_num(0).max() <= 1 if n > 1 or window else True
    if not window:
        assert out[n - 1].isnan().all() and lse[n - 1].isnan().all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_strided(gdn, dtype):
    b = U.Batch([1, 4, 90], [100, 4, 300], 2, seed=21)
    b.fill()
    cache = to_cache(gdn, b)
    wide = b.randn(b.T, 11, 128).to(dtype)
    dev = wide.cuda()
    into = torch.full((b.T, 9, 128), 7.0, dtype=dtype, device="cuda")
    out, lse = gdn.gdn_kv_attn(dev[:, 2:8], cache, b.lens.cuda(), b.table.cuda(), b.cu.cuda(), out=into[:, 1:7])
    packed, lse2 = gdn.gdn_kv_attn(dev[:, 2:8].contiguous(), cache, b.lens.cuda(), b.table.cuda(), b.cu.cuda())
    assert torch.equal(out, packed) and torch.equal(lse, lse2)
    assert (into[:, 0] == 7).all() and (into[:, 7:] == 7).all()
    no_lse, none = gdn.gdn_kv_attn(dev[:, 2:8], cache, b.lens.cuda(), b.table.cuda(), b.cu.cuda(), return_lse=False)
    assert none is None and torch.equal(no_lse, packed)


@pytest.mark.parametrize("n", [1, 6, 150])
def test_pool_past_32_bits(gdn, n):
    """Pages whose codes lie past 2^31 and 2^32 bytes of the pool."""
    b = U.Batch([n], [400], 2, seed=2)
    b.fill(stale_nan=False)
    pool = 300_000  # 2 heads: 4.9 GB of keys
    cache = gdn.KVCache.empty(pool, 2)
    table = torch.tensor([[pool - 1 - 11 * i for i in range(b.max_pages)]], dtype=torch.int32)
    for i in range(b.max_pages):
        src, dst = int(b.table[0, i]), int(table[0, i])
        cache.k.view(torch.uint8)[dst] = b.k[src].to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        cache.v.view(torch.uint8)[dst] = b.v[src].to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        cache.k_scale[dst], cache.v_scale[dst] = b.ks[src].cuda(), b.vs[src].cuda()
    q = b.randn(n, 4, 128).to(BF)
    small = to_cache(gdn, b)
    a = gdn.gdn_kv_attn(q.cuda(), small, b.lens.cuda(), b.table.cuda())
    c = gdn.gdn_kv_attn(q.cuda(), cache, b.lens.cuda(), table.cuda())
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    x = gdn.gdn_kv_read(small, b.lens.cuda(), b.table.cuda(), T=n)
    y = gdn.gdn_kv_read(cache, b.lens.cuda(), table.cuda(), T=n)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    gdn.gdn_kv_append(small, x[0], x[1], b.lens.cuda(), b.table.cuda())
    gdn.gdn_kv_append(cache, x[0], x[1], b.lens.cuda(), table.cuda())
    for i in range(b.max_pages):
        assert torch.equal(small.k.view(torch.uint8)[int(b.table[0, i])], cache.k.view(torch.uint8)[int(table[0, i])])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 5, 200])
def test_attn_repeats_bitwise(gdn, dtype, n):
    b = U.Batch([n] * 3, [n + 50, n + 3000, n + 700], 2, seed=4)
    b.fill()
    q = b.randn(b.T, 8, 128).to(dtype).cuda()
    cache, lens, table = to_cache(gdn, b), b.lens.cuda(), b.table.cuda()
    first = gdn.gdn_kv_attn(q, cache, lens, table)
    for _ in range(3):
        again = gdn.gdn_kv_attn(q, cache, lens, table)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("n", [1, 4, 140])
def test_attn_graph_replay_with_growing_lengths(gdn, n):
    """A captured append + attention, replayed while the lengths grow on the device, gives what eager calls give."""
    b = U.Batch([n, n], [900, 900], 2, seed=6)
    b.fill(stale_nan=False)
    table = b.table.cuda()
    lens = torch.tensor([n + 60, n], dtype=torch.int32, device="cuda")
    q, k, v = (b.randn(2 * n, h, 128).to(BF).cuda() for h in (8, 2, 2))
    plan = gdn.gdn_kv_attn_plan(T=2 * n, n_seqs=2, h_q=8, h_kv=2, max_q_len=n, max_pages=b.max_pages)
    ws = torch.empty(max(256, plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    cache, eager = to_cache(gdn, b), to_cache(gdn, b)
    out, lse = torch.empty_like(q), torch.empty(2 * n, 8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn.gdn_kv_append(cache, k, v, lens, table)
        gdn.gdn_kv_attn(q, cache, lens, table, plan=plan, out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_kv_append(cache, k, v, lens, table)
        gdn.gdn_kv_attn(q, cache, lens, table, plan=plan, out=out, lse=lse, workspace=ws)
    for step in range(3):
        g.replay()
        gdn.gdn_kv_append(eager, k, v, lens, table)
        o2, z2 = gdn.gdn_kv_attn(q, eager, lens, table, plan=plan)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, z2)
        lens += n
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape).to(x.dtype))
    assert status(gdn, cache) == (0, 0)


# ---------------------------------------------------------------- what the kernels refuse to follow
@pytest.mark.parametrize("n", [1, 5, 200])
@pytest.mark.parametrize("what", ["page_past", "page_negative", "length_past", "length_negative", "offsets_back", "offsets_past"])
def test_device_checks(gdn, what, n):
    """Bad lengths, offsets and pages are recorded, nothing leaves the buffers, and the next call is clean."""
    b = U.Batch([n] * 3, [n + 100] * 3, 2, seed=8)
    b.fill()
    cache = to_cache(gdn, b)
    lens, table, cu = b.lens.clone(), b.table.clone(), b.cu.clone()
    if what == "page_past":
        table[1, 0] = b.n_pages
    elif what == "page_negative":
        table[1, 1] = -1
    elif what == "length_past":
        lens[1] = 64 * b.max_pages + 1
    elif what == "length_negative":
        lens[1] = -1
    elif what == "offsets_back":
        cu[1], cu[2] = cu[2].clone(), cu[1].clone()
    else:
        cu[1] = b.T + 1
    q = b.randn(b.T, 4, 128).to(BF).cuda()
    want = 8 if "page" in what else 7
    good = gdn.gdn_kv_attn(q, cache, b.lens.cuda(), b.table.cuda(), b.cu.cuda())
    out, lse = gdn.gdn_kv_attn(q, cache, lens.cuda(), table.cuda(), cu.cuda())
    assert status(gdn, cache) == (7, want)
    assert "check failed" in gdn.describe_device_status(7, want)
    if "offsets" not in what:  # the other sequences are as they were
        for s in (slice(0, n), slice(2 * n, 3 * n)):
            assert torch.equal(out[s], good[0][s]) and torch.equal(lse[s], good[1][s])
    cache.status.zero_()
    k, v = gdn.gdn_kv_read(cache, lens.cuda(), table.cuda(), cu.cuda(), T=b.T)
    code = status(gdn, cache)
    assert code == (7, 7) if want == 7 else code in ((0, 0), (7, 8))  # the page may not be among those read
    cache.status.zero_()
    before = cache.k.view(torch.uint8).clone()
    gdn.gdn_kv_append(cache, k, v, lens.cuda(), table.cuda(), cu.cuda())
    if what in ("length_past", "length_negative"):
        pages = b.table[1].long().cuda()
        assert torch.equal(before[pages], cache.k.view(torch.uint8)[pages])  # nothing stored for that sequence
    cache = to_cache(gdn, b)
    again = gdn.gdn_kv_attn(q, cache, b.lens.cuda(), b.table.cuda(), b.cu.cuda())
    assert status(gdn, cache) == (0, 0)
    assert torch.equal(again[0], good[0])


def test_more_tokens_than_the_plan(gdn):
    b = U.Batch([1, 300], [50, 300], 2, seed=1)
    b.fill()
    cache = to_cache(gdn, b)
    q = b.randn(b.T, 4, 128).to(BF).cuda()
    plan = gdn.gdn_kv_attn_plan(T=b.T, n_seqs=2, h_q=4, h_kv=2, max_q_len=3, max_kv_len=300)
    gdn.gdn_kv_attn(q, cache, b.lens.cuda(), b.table.cuda(), b.cu.cuda(), plan=plan)
    assert status(gdn, cache) == (7, 7)
