"""The operators between the projections and the mixers, run as they are used:
before the gated delta rule, its decode step and its backward, before the
attention over the cache, captured in CUDA graphs, on other streams."""
from __future__ import annotations

import math

import pytest
import torch

from tests import front_util as F
from tests import kv_check
from tests import kv_util as K

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU, skipped there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import oracle  # noqa: E402
from oracle import backward as OB  # noqa: E402
import gated_deltanet_linear_fwd_gb300 as gdn  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.double().cpu().numpy()


class Layer:
    """A gated-delta-rule layer behind its projections."""

    def __init__(self, lens, h_qk=1, h_v=2, seed=0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.lens, self.h_qk, self.h_v, self.T = lens, h_qk, h_v, sum(lens)
        self.C = (2 * h_qk + h_v) * 128
        self.x = rnd(self.T, self.C).bfloat16()
        self.w = rnd(self.C, 4) / 2
        self.g = torch.nn.functional.logsigmoid(rnd(self.T, h_v) + 3.0)
        self.beta = torch.sigmoid(rnd(self.T, h_v))
        self.d_o = rnd(self.T, h_v, 128).bfloat16()
        self.offsets = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
        self.cu = self.offsets.cuda()


def check_rms(name, got, want, rms=None):
    """The bar of the bf16 paths: 2e-2 of the RMS beyond bf16's own rounding."""
    got, want = got.double().cpu(), torch.as_tensor(want)
    err = ((got - want).abs() - F.half_step(want, BF16)).clamp(min=0).max()
    assert err <= 2e-2 * (rms or want.pow(2).mean().sqrt()), name


def test_training_step_of_a_layer():
    """Convolution, delta rule and both their gradients over packed sequences: each
    against 64 bits, from what the one before gave."""
    s = Layer([70, 1, 130], seed=1)
    ref = F.Conv(s.x, s.w, s.h_qk, lens=s.lens)
    q, k, v, last = gdn.gdn_conv_fwd(s.x.cuda(), s.w.cuda(), s.h_qk, None, None, s.cu)
    for name, got, want, bound in zip("qkv", (q, k, v), ref.out, ref.bounds):
        F.check(name, got, want, bound, BF16)
    g, beta, d_o = s.g.cuda(), s.beta.cuda(), s.d_o.cuda()
    plan = gdn.gdn_cp_plan(T=s.T, h_qk=s.h_qk, h_v=s.h_v, cu_seqlens=s.offsets.tolist(), mode="exact", lambda_=0.5)
    ws = torch.empty(gdn.gdn_bwd_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    o, _ = gdn.gdn_chunk_fwd(q, k, v, g, beta, None, s.cu, plan=plan, workspace=ws, for_backward=True)
    dq, dk, dv, *_ = gdn.gdn_chunk_bwd(q, k, v, g, beta, d_o, None, None, s.cu, plan=plan, workspace=ws, reuse_forward=True)
    zero = torch.zeros(len(s.lens), s.h_v, 128, 128)
    args = (f64(q), f64(k), f64(v), f64(g), f64(beta), f64(zero), s.offsets.tolist())
    want_o, _ = oracle.recurrence(*args)
    check_rms("o", o, want_o)
    grads = OB.grad_chunked(*args, f64(d_o), f64(zero))
    for name, got, want in zip(("dq", "dk", "dv"), (dq, dk, dv), grads):
        check_rms(name, got, want)
    dx, dw, _, _ = gdn.gdn_conv_bwd(s.x.cuda(), s.w.cuda(), s.h_qk, dq, dk, dv, cu_seqlens=s.cu)
    want, bound = ref.backward(dq.cpu(), dk.cpu(), dv.cpu())
    F.check("dx", dx, want[0], bound[0], BF16)
    F.check("dw", dw, want[1], bound[1])


def test_prompt_and_steps_of_a_layer():
    """A prompt, then single tokens through convolution and decode step, against the whole sequence in 64 bits."""
    s = Layer([40], seed=2)
    n, x, w = 33, s.x.cuda(), s.w.cuda()
    q, k, v, conv = gdn.gdn_conv_fwd(x[:n], w, s.h_qk)
    _, state = gdn.gdn_chunk_fwd(q, k, v, s.g[:n].cuda(), s.beta[:n].cuda(), mode="off")
    ref = F.Conv(s.x, s.w, s.h_qk)
    whole = [t.to(BF16).double().numpy() for t in ref.out]
    want, _ = oracle.recurrence(*whole, f64(s.g), f64(s.beta), f64(torch.zeros(1, s.h_v, 128, 128)), [0, s.T])
    for t in range(n, s.T):
        q, k, v = gdn.gdn_conv_step(x[t:t + 1], conv, w, s.h_qk)
        o = gdn.gdn_decode_step(q, k, v, s.g[t:t + 1].cuda(), s.beta[t:t + 1].cuda(), state)
        # o is a bf16: next to 2e-2 of the RMS it is off by its own rounding, half a step, 2^-14 for the
        # values of 2^-6 to 2^-5 here (6.1e-5, a third of 2e-2 x 0.0092)
        check_rms("o", o[0], want[t], rms=float((want ** 2).mean() ** 0.5))
    assert torch.equal(conv[0].cpu(), s.x[-3:])


@pytest.mark.parametrize("dtype,use_cu", [(BF16, False), (BF16, True), (F32, False)])
def test_attention_over_rotated_keys(dtype, use_cu):
    """The rotated append, then attention: as of queries and keys in 64 bits over what the cache holds."""
    b = K.Batch([30, 3, 1], [30, 200, 65], 2, seed=3) if use_cu else K.Batch([2, 2], [130, 64], 2, seed=4)
    b.fill()
    h_q = 4
    q, k, v = (b.randn(b.T, h, 128).to(dtype) for h in (h_q, 2, 2))
    qw, kw = 1 + 0.2 * b.randn(128), 1 + 0.2 * b.randn(128)
    code = lambda c: c.float().to(torch.float8_e4m3fn).cuda()  # noqa: E731
    cache = gdn.KVCache(code(b.k), code(b.v), b.ks.float().cuda(), b.vs.float().cuda())
    lens, table, cu = b.lens.cuda(), b.table.cuda(), b.cu.cuda() if use_cu else None
    turned = gdn.gdn_kv_append_rope(cache, k.cuda(), v.cuda(), lens, table, cu, rope=gdn.gdn_rope_table(64), norm="rms", eps=1e-6,
                                    k_weight=kw.cuda(), q=q.cuda(), q_weight=qw.cuda())
    out, lse = gdn.gdn_kv_attn(turned, cache, lens, table, cu)
    assert gdn.gdn_get_device_status(cache.status) == (0, 0)
    b.k, b.ks, b.v, b.vs = (t.float().cpu() for t in (cache.k, cache.k_scale, cache.v, cache.v_scale))
    plan = gdn.gdn_kv_attn_plan(T=b.T, n_seqs=b.n, h_q=h_q, h_kv=2, max_q_len=0 if use_cu else 2, max_pages=b.max_pages, dtype=dtype)
    again = kv_check.check(gdn, b, h_q, plan, turned.cpu(), use_cu, dtype)   # the attention's own bound, on these queries
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    pos = torch.cat([torch.arange(kv - n, kv) for n, kv in zip(b.q_lens, b.kv_lens)])
    F.check("q", turned, *F.rope_ref(q, pos, F.frequencies(64), norm="rms", weight=qw), dtype)


def capture(run):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    return graph, kept


def test_captured_calls_follow_their_inputs():
    """Each operator captured once and replayed on new inputs, against eager calls bit for bit."""
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    T, cu = 90, torch.tensor([0, 50, 50, 90], dtype=torch.int32, device="cuda")
    qkv, grads = rnd(T, 6, 128).bfloat16(), rnd(T, 6, 128).bfloat16()
    q, k, gq, gk = qkv[:, :4], qkv[:, 4:], grads[:, :4], grads[:, 4:]
    rope, w = gdn.gdn_rope_table(128), rnd(128).abs()
    x, taps, bias, state = rnd(T, 512).bfloat16(), rnd(512, 4), rnd(512), rnd(3, 3, 512).bfloat16()
    d = [rnd(T, 1, 128).bfloat16(), rnd(T, 1, 128).bfloat16(), rnd(T, 2, 128).bfloat16()]
    xs, step_state = rnd(5, 512).bfloat16(), rnd(5, 3, 512).bfloat16()
    keep = step_state.clone()

    def step():
        step_state.copy_(keep)
        return (*gdn.gdn_conv_step(xs, step_state, taps, 1, bias), step_state.clone())

    runs = {
        "rope": lambda: gdn.gdn_qk_rope(q, k, rope, None, cu, norm="rms", q_weight=w, k_weight=w),
        "rope_bwd": lambda: gdn.gdn_qk_rope_bwd(q, k, gq, gk, rope, None, cu, norm="rms", q_weight=w, k_weight=w),
        "conv": lambda: gdn.gdn_conv_fwd(x, taps, 1, bias, state, cu),
        "conv_bwd": lambda: gdn.gdn_conv_bwd(x, taps, 1, *d, bias, state, state, cu),
        "step": step}
    for name, run in runs.items():
        graph, kept = capture(run)
        for _ in range(2):
            for t in (qkv, grads, x, state, *d, xs, keep, taps, w):
                t.copy_(rnd(*t.shape))
            w.abs_()
            if name != "step":
                cu.copy_(torch.tensor([0, int(torch.randint(0, 90, (1,), generator=g)), 90, 90]))
            graph.replay()
            got = [t.clone() for t in kept]
            assert all(torch.equal(a, b) for a, b in zip(got, run())), name


def test_captured_append_follows_the_lengths():
    g = torch.Generator().manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    table = torch.randperm(8, generator=g).to(torch.int32).view(2, 4).cuda()
    lens = torch.tensor([60, 127], dtype=torch.int32, device="cuda")
    q, k, v, w = rnd(2, 4, 128).bfloat16(), rnd(2, 2, 128).bfloat16(), rnd(2, 2, 128).bfloat16(), rnd(128).abs()
    rope = gdn.gdn_rope_table(128, layout="interleaved")
    one, two = gdn.KVCache.empty(8, 2), gdn.KVCache.empty(8, 2)
    call = lambda c: gdn.gdn_kv_append_rope(c, k, v, lens, table, rope=rope, norm="unit", k_weight=w, q=q, q_weight=w)  # noqa: E731
    graph, kept = capture(lambda: call(one))
    call(two)
    for _ in range(8):
        lens += 1
        for t in (q, k, v):
            t.copy_(rnd(*t.shape))
        graph.replay()
        want = call(two)
        assert torch.equal(kept, want)
        for name in ("k", "v"):
            assert torch.equal(getattr(one, name).view(torch.uint8), getattr(two, name).view(torch.uint8))
            assert torch.equal(getattr(one, name + "_scale"), getattr(two, name + "_scale"))


def test_captured_graphs_share_a_workspace():
    """Two captured gradients with one workspace, replayed in turn on a stream: what one left there does not matter to the other."""
    g = torch.Generator().manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, taps, bias = rnd(300, 512), rnd(512, 4), rnd(512)
    d = [rnd(300, h, 128) for h in (1, 1, 2)]
    q, dq, w, rope = rnd(500, 3, 128), rnd(500, 3, 128), rnd(128).abs(), gdn.gdn_rope_table(64)
    n = max(gdn.gdn_conv_bwd_workspace_bytes(300, 1, 2, dtype=F32), gdn.gdn_qk_rope_bwd_workspace_bytes())
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")   # NaN bits
    runs = [lambda: gdn.gdn_conv_bwd(x, taps, 1, *d, bias, workspace=ws)[:3],
            lambda: [t for t in gdn.gdn_qk_rope_bwd(q, None, dq, None, rope, norm="rms", q_weight=w, workspace=ws) if t is not None]]
    graphs = [capture(run) for run in runs]
    want = [[t.clone() for t in run()] for run in runs]
    for graph, kept in graphs * 2:
        for t in kept:
            t.zero_()
        graph.replay()
    for (_, kept), ref in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(kept, ref))


def test_gradients_captured_beside_an_eager_graph():
    """A captured backward while an eager autograd graph over the same leaves is alive."""
    s = Layer([64], seed=7)
    x, w = s.x.float().cuda().requires_grad_(), s.w.cuda().requires_grad_()
    eager = (x * w[:, 0]).sum()   # holds on to both leaves
    d = [torch.ones(64, h, 128, device="cuda") for h in (1, 1, 2)]
    graph, kept = capture(lambda: gdn.gdn_conv_bwd(x, w, 1, *d))
    graph.replay()
    want = gdn.gdn_conv_bwd(x.detach(), w.detach(), 1, *d)
    assert torch.equal(kept[0], want[0]) and torch.equal(kept[1], want[1])
    eager.backward()
    assert torch.equal(x.grad, w.detach()[:, 0].expand_as(x))
    assert kept[0].grad_fn is None and not kept[0].requires_grad


def test_other_streams():
    """On a side stream, by argument and by context, and two at once with their own workspaces."""
    s = Layer([900], seed=8)
    x, w = s.x.cuda(), s.w.cuda()
    d = [torch.randn(900, h, 128, device="cuda").bfloat16() for h in (1, 1, 2)]
    rope, q = gdn.gdn_rope_table(128), torch.randn(900, 8, 128, device="cuda").bfloat16()
    qw = torch.rand(128, device="cuda") + 0.5
    runs = [lambda **kw: gdn.gdn_conv_fwd(x, w, 1, **kw), lambda **kw: gdn.gdn_conv_bwd(x, w, 1, *d, **kw)[:2],
            lambda **kw: gdn.gdn_qk_rope(q, None, rope, norm="rms", q_weight=qw, **kw)[:1],
            lambda **kw: [t for t in gdn.gdn_qk_rope_bwd(q, None, q, None, rope, norm="rms", q_weight=qw, **kw) if t is not None]]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for run, ref in zip(runs, want):
        for st in streams:
            st.wait_stream(torch.cuda.current_stream())
        got = [run(stream=st) for st in streams]
        with torch.cuda.stream(streams[0]):
            got.append(run())
        torch.cuda.synchronize()
        for one in got:
            assert all(torch.equal(a, b) for a, b in zip(one, ref))


def test_kernels_are_named():
    s = Layer([10], seed=9)
    out = gdn.gdn_conv_fwd(s.x.cuda(), s.w.cuda(), 1)
    assert gdn.gdn_trace_last() == ["conv"]
    gdn.gdn_conv_bwd(s.x.cuda(), s.w.cuda(), 1, *out[:3])
    assert gdn.gdn_trace_last() == ["conv_bwd", "conv_bwd_sums"]
    gdn.gdn_qk_rope(out[0], out[1], gdn.gdn_rope_table(128))
    assert gdn.gdn_trace_last() == ["qk_rope"]
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for e in events:
        e.record()
    gdn.gdn_set_trace_events(events)
    gdn.gdn_conv_step(s.x.cuda(), torch.zeros(10, 3, s.C, dtype=BF16, device="cuda"), s.w.cuda(), 1)
    gdn.gdn_set_trace_events([])
    torch.cuda.synchronize()
    assert gdn.gdn_trace_last() == ["conv_step"] and math.isfinite(events[0].elapsed_time(events[1]))
