"""Cases for what stands between a layer's projections and its mixers.

Attention mixers: the queries and keys of each head are normalised and rotated
by their position (rope), with the gradients of that (rope_bwd), and on the way
into the 8-bit paged cache (append): heads of 128 elements, pages of 64 tokens.

Gated-delta-rule mixers: a short causal convolution over the projection's
channels, an activation, and unit length for the heads of q and k (conv), its
gradients (conv_bwd), and its form for one new token a sequence (step).

Tokens of a batch are packed: sequence i has the tokens cu[i] to cu[i + 1].

`own` selects what run() computes: False, the plain forms in elementary torch
operations in fp32 (fp64 for angles, for keys next to a border of their page's
scale, and for sums over all tokens); True, the calls of
gated_deltanet_linear_fwd_gb300.
"""
import math
import random

import torch

own = False

D = 128         # elements of a head
PAGE = 64       # tokens of a cache page, and of a scale
E_MIN, E_MAX = -40, 40     # exponents a scale may have
TOP = 448.0     # largest e4m3 value
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def _rope(name, op, n, len_min, len_max, h_q, h_k, dtype="bf16", layout="half", rot=128, norm="rms", weights=True,
          scaling="none", factor=1.0, start=0, fused=True, mix=0):
    """start: position of each sequence's first token; append: the tokens already there are up to this many."""
    return {"name": name, "op": op, "n": n, "len_min": len_min, "len_max": len_max, "h_q": h_q, "h_k": h_k, "dtype": dtype,
            "layout": layout, "rot": rot, "norm": norm, "weights": weights, "scaling": scaling, "factor": factor,
            "start": start, "fused": fused, "mix": mix}


def _conv(name, op, n, len_min, len_max, h_qk, h_v, dtype="bf16", width=4, bias=False, silu=True, norm=True, state=False,
          fused=True, mix=0, len_list=""):
    return {"name": name, "op": op, "n": n, "len_min": len_min, "len_max": len_max, "h_qk": h_qk, "h_v": h_v, "dtype": dtype,
            "width": width, "bias": bias, "silu": silu, "norm": norm, "state": state, "fused": fused, "mix": mix,
            "len_list": len_list}


def listed():
    return [
        # the queries and keys of one generated token: latency alone
        _rope("rope_one_token", "rope", 1, 1, 1, 8, 2, start=65535, mix=1),
        # those of a whole prompt of 32768 tokens, used in place in the fused projection
        _rope("rope_prompt_32768", "rope", 1, 32768, 32768, 8, 2, mix=2),
        # a training step's gradients over 32768 tokens of ragged packed documents
        _rope("rope_bwd_packed_32768", "rope_bwd", 16, 512, 3000, 8, 2, mix=3),
        # fp32 gradients, neighbouring pairs, half of each head rotated, heads of unit length
        _rope("rope_bwd_ragged_f32", "rope_bwd", 5, 1, 4109, 3, 2, "f32", "interleaved", 64, "unit", False, fused=False, mix=4),
        # one generated token for each of 256 sequences, keys and values into the cache, queries beside them
        _rope("append_decode_256", "append", 256, 1, 1, 8, 2, start=4096, mix=5),
        # a 32768-token piece of a prompt behind 65536 tokens, frequencies scaled for the long context
        _rope("append_piece_32768", "append", 1, 32768, 32768, 8, 2, scaling="parts", factor=8.0, start=65536, mix=6),
        # a whole prompt through the convolution of a layer with 2 + 2 + 8 heads
        _conv("conv_prompt_32768", "conv", 1, 32768, 32768, 2, 8, mix=7),
        # four packed long contexts that go on from kept states
        _conv("conv_varlen_348160", "conv", 4, 0, 0, 2, 8, state=True, mix=8, len_list="262144/65536/16384/4096"),
        # a training step's gradients over 32768 tokens
        _conv("conv_bwd_32768", "conv_bwd", 1, 32768, 32768, 2, 8, mix=9),
        # fp32 gradients over short ragged sequences, three taps and a bias, states on both sides
        _conv("conv_bwd_ragged_f32", "conv_bwd", 7, 1, 2051, 1, 2, "f32", 3, True, state=True, fused=False, mix=10),
        # one generated token for each of 256 sequences
        _conv("step_256", "step", 256, 1, 1, 2, 8, mix=11),
        # one generated token of one sequence of a wider layer, fp32
        _conv("step_one_f32", "step", 1, 1, 1, 16, 16, "f32", mix=12),
    ]


MOST = 348160 * 12 * D * 2      # bytes of one input of the largest listed case


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "rope_bwd", "append", "append", "conv", "conv", "conv_bwd", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    es = 4 if dtype == "f32" else 2
    mix = rng.randrange(1 << 20)
    fused = rng.random() < 0.6
    if op in ("rope", "rope_bwd", "append"):
        h_k = rng.choice([1, 2, 2, 3, 4, 8, 16])
        h_q = h_k * rng.choice([1, 2, 4, 8]) if h_k <= 8 else h_k
        # tokens of all sequences, so that the three tensors of a gradient stay within the largest case
        most = min(131072, MOST // 4 // es // D // (h_q + h_k))
        n = _log(rng, 1, 256)
        length = rng.choice([1, _log(rng, 1, most // n), _log(rng, 1, most // n)])
        if op == "append":
            start = rng.choice([0, _log(rng, 1, 400000 // n // h_k)])
        else:
            start = rng.choice([0, 0, _log(rng, 1, 1 << 20)])
        scaling = rng.choice(["none", "none", "linear", "ntk", "parts"])
        return _rope("", op, n, rng.choice([1, length]), length, h_q, h_k, dtype, rng.choice(["half", "half", "interleaved"]),
                     rng.choice([128, 128, 64, 32, 96, 16, 8]), rng.choice(["rms", "rms", "unit", "none"]), rng.random() < 0.7,
                     scaling, 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]), start, fused, mix)
    h_qk = rng.choice([1, 2, 2, 4, 8, 16])
    h_v = rng.choice([h_qk, 2 * h_qk, 3 * h_qk, 4 * h_qk])
    most = MOST // (4 if op == "conv_bwd" else 2) // es // D // (2 * h_qk + h_v)
    n = _log(rng, 1, 512 if op == "step" else 64)
    length = 1 if op == "step" else rng.choice([_log(rng, 1, 8), _log(rng, 1, most // n), _log(rng, 1, most // n)])
    return _conv("", op, n, rng.choice([0, 1, length]) if op != "step" else 1, length, h_qk, h_v, dtype, rng.choice([4, 4, 4, 3, 2]),
                 rng.random() < 0.3, rng.random() < 0.85, rng.random() < 0.75, rng.random() < 0.5, fused, mix)


def _lens(case):
    """Tokens of each sequence, from the case alone; the first has the most."""
    if case.get("len_list"):
        return [int(x) for x in case["len_list"].split("/")]
    rng = random.Random(case["mix"])
    return [case["len_max"]] + [rng.randint(case["len_min"], case["len_max"]) for _ in range(case["n"] - 1)]


def _past(case):
    """Append: tokens that each sequence has already; the first has the most."""
    rng = random.Random(case["mix"] + 1)
    return [case["start"]] + [_log(rng, 1, case["start"]) if case["start"] else 0 for _ in range(case["n"] - 1)]


def work(case):
    T, es, n = sum(_lens(case)), 4 if case["dtype"] == "f32" else 2, case["n"]
    op = case["op"]
    if op in ("rope", "rope_bwd", "append"):
        h_q, h_k = case["h_q"], case["h_k"]
        heads = T * (h_q + h_k) * D
        if op == "rope":
            return {"bytes": 2 * heads * es + 4 * T * (case["start"] > 0), "flops": 8 * heads}
        if op == "rope_bwd":
            tensors = 2 if case["norm"] == "none" else 3    # without a norm the inputs themselves are not needed
            return {"bytes": tensors * heads * es + 4 * T * (case["start"] > 0), "flops": 16 * heads}
        pages = sum(-(-(a + b) // PAGE) - a // PAGE for a, b in zip(_past(case), _lens(case)) if b)
        return {"bytes": 2 * T * h_q * D * es + 2 * T * h_k * D * (es + 1) + pages * (h_k * 8 + 4) + 4 * n,
                "flops": 8 * heads + 4 * T * h_k * D}
    C, W = (2 * case["h_qk"] + case["h_v"]) * D, case["width"]
    state = n * (W - 1) * C * es
    if op == "conv":
        return {"bytes": 2 * T * C * es + state * (1 + case["state"]) + 4 * C * W, "flops": T * C * (2 * W + 8)}
    if op == "conv_bwd":
        return {"bytes": 3 * T * C * es + 3 * state * case["state"] + 8 * C * W, "flops": T * C * (6 * W + 24)}
    return {"bytes": 2 * T * C * es + 2 * state + 4 * C * W, "flops": T * C * (2 * W + 8)}


# ---------------------------------------------------------------- inputs
def _pow2_scale(a):
    """The smallest power of two s with a / s <= 448, its exponent in [E_MIN, E_MAX]."""
    m, e = torch.frexp(a)                      # a = m 2^e, 0.5 <= m < 1
    e = e - 9 + (m > 0.875).to(e.dtype)
    e = torch.where(a > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x, s):
    """x / s rounded to e4m3; what is not finite becomes NaN."""
    y = (x / s).clamp(-TOP, TOP).float()
    return torch.where(x.isfinite(), y, torch.full_like(y, math.nan)).to(torch.float8_e4m3fn)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    lens, n, dt = _lens(case), case["n"], TYPES[case["dtype"]]
    T = sum(lens)
    cu = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
    st = {"case": case, "T": T, "cu": cu, "cu_arg": None if n == 1 else cu}
    if case["op"] in ("conv", "conv_bwd", "step"):
        return _prepare_conv(case, st, rnd, dt)
    h_q, h_k = case["h_q"], case["h_k"]

    def heads(*sizes):
        """Tensors [T, heads, 128], as parts of one projection's output or alone; channels of different size."""
        if not case["fused"]:
            return [(rnd(T, h, D) * torch.exp(0.4 * rnd(h, D))).to(dt) for h in sizes]
        x = rnd(T, sum(sizes), D).mul_(torch.exp(0.4 * rnd(sum(sizes), D)))
        return list(x.to(dt).split(sizes, dim=1))

    st["q"], st["k"], st["v"] = heads(h_q, h_k, h_k)
    st["q_weight"] = st["k_weight"] = None
    if case["norm"] != "none" and case["weights"]:
        st["q_weight"], st["k_weight"] = 1 + 0.2 * rnd(D), 1 + 0.2 * rnd(D)
    past = _past(case)
    if case["op"] == "append":
        kv = [a + b for a, b in zip(past, lens)]
        pages = [-(-b // PAGE) for b in kv]
        n_pages, max_pages = sum(pages) + 3, max(1, max(pages))
        perm = torch.randperm(n_pages, device=dev, generator=gen).to(torch.int32)
        count = torch.tensor(pages, device=dev)
        slot = torch.arange(max_pages, device=dev)[None, :]
        st["table"] = perm[((count.cumsum(0) - count)[:, None] + slot).clamp(max=n_pages - 1)].contiguous()
        st["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
        st["first"] = torch.tensor(past, device=dev)
        if min(lens) == max(lens):
            st["cu_arg"] = None
        # what earlier tokens left in the pages
        for name in ("k", "v"):
            x = rnd(n_pages, h_k, PAGE, D).mul_(torch.exp(0.3 * rnd(n_pages, 1, PAGE, 1)))
            s = _pow2_scale(x.abs().amax((2, 3)))
            st[name + "_cache"] = _codes(x, s[:, :, None, None])
            st[name + "_scale"] = s
            del x
    else:
        st["first"] = torch.full((n,), case["start"], device=dev)
        st["positions"] = None
        if case["start"]:
            st["positions"], st["cu_arg"] = _positions(st).to(torch.int32), None
    if case["op"] == "rope_bwd":
        st["d_q_out"], st["d_k_out"] = rnd(T, h_q, D).to(dt), rnd(T, h_k, D).to(dt)
    st["q_out"] = torch.empty(T, h_q, D, dtype=dt, device=dev)
    st["k_out"] = torch.empty(T, h_k, D, dtype=dt, device=dev)
    if own:  # the table of frequencies, the cache's handle, the gradients' workspace
        import gated_deltanet_linear_fwd_gb300 as gdn
        st["rope"] = gdn.gdn_rope_table(case["rot"], base=10000.0, layout=case["layout"], scaling=case["scaling"],
                                        factor=case["factor"], original_len=4096, low=1.0, high=32.0, magnitude=_magnitude(case))
        if case["op"] == "append":
            st["cache"] = gdn.KVCache(st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
        if case["op"] == "rope_bwd":
            st["workspace"] = torch.empty(gdn.gdn_qk_rope_bwd_workspace_bytes(), dtype=torch.uint8, device=dev)
    return st


def _prepare_conv(case, st, rnd, dt):
    T, n, W, h_qk, h_v = st["T"], case["n"], case["width"], case["h_qk"], case["h_v"]
    C = (2 * h_qk + h_v) * D
    pad = 2 * h_v if case["fused"] else 0       # a projection that also gives the gates' inputs (padded to 8 columns)
    pad = -(-pad // 8) * 8
    st["x"] = rnd(T, C + pad).to(dt)[:, :C]
    st["weight"] = rnd(C, W) / math.sqrt(W)
    st["bias"] = 0.2 * rnd(C) if case["bias"] else None
    st["state"] = rnd(n, W - 1, C).to(dt) if case["state"] or case["op"] == "step" else None
    shapes = ((T, h_qk, D), (T, h_qk, D), (T, h_v, D))
    if case["op"] == "conv_bwd":
        st["d_out"] = [rnd(*s).to(dt) for s in shapes]
        st["d_final"] = rnd(n, W - 1, C).to(dt) if case["state"] else None
        if own:
            import gated_deltanet_linear_fwd_gb300 as gdn
            size = gdn.gdn_conv_bwd_workspace_bytes(T, h_qk, h_v, n_seqs=n, width=W, dtype=dt)
            st["workspace"] = torch.empty(max(256, size), dtype=torch.uint8, device="cuda")
    else:
        st["out"] = [torch.empty(*s, dtype=dt, device="cuda") for s in shapes]
        if case["op"] == "conv":
            st["final"] = torch.empty(n, W - 1, C, dtype=dt, device="cuda")
    return st


# ---------------------------------------------------------------- the plain forms
def _positions(st):
    t = torch.arange(st["T"], device="cuda")
    seq = torch.searchsorted(st["cu"][1:].long(), t, right=True)
    return st["first"][seq] + t - st["cu"].long()[seq]


def _magnitude(case):
    """What rotated elements are multiplied with: longer contexts flatten the softmax, 0.1 ln(factor) + 1 counters it."""
    return 0.1 * math.log(case["factor"]) + 1 if case["scaling"] == "parts" else 1.0


def _frequencies(case):
    """Radians a token of each pair i < rot / 2, in 64 bits."""
    rot, s = case["rot"], case["factor"]
    base = 10000.0
    if case["scaling"] == "ntk":
        base = base * s ** (rot / (rot - 2))
    f = torch.pow(torch.tensor(base, dtype=torch.float64, device="cuda"), -torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "parts":          # by the turns a pair makes over the original 4096 tokens: up to 1 slowed down, from 32 on kept
        keep = ((4096 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        f = f * keep + f / s * (1 - keep)
    return f


def _turn(case, pos, x, sign=1.0):
    """x [T, heads, 128] rotated at the positions, in x's type; sign -1: the transposed rotation."""
    rot = case["rot"]
    angle = pos.double()[:, None] * _frequencies(case)[None, :]
    c = (torch.cos(angle) * _magnitude(case)).to(x.dtype)[:, None]
    s = (torch.sin(angle) * (sign * _magnitude(case))).to(x.dtype)[:, None]
    y = x.clone()
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def _inverse_norm(kind, x):
    ss = x.square().sum(-1, keepdim=True)
    return torch.rsqrt((ss / D if kind == "rms" else ss) + EPS)


def _norm_turn(case, pos, x, weight):
    if case["norm"] != "none":
        x = x * _inverse_norm(case["norm"], x)
        if weight is not None:
            x = x * weight
    return _turn(case, pos, x)


def _plain_rope(st):
    c, pos = st["case"], _positions(st)
    dt = TYPES[c["dtype"]]
    return tuple(_norm_turn(c, pos, st[x].float(), st[x + "_weight"]).to(dt) for x in "qk")


def _plain_rope_bwd(st):
    c, pos = st["case"], _positions(st)
    dt = TYPES[c["dtype"]]
    grads, weights = [], []
    for name in "qk":
        w = st[name + "_weight"]
        du = _turn(c, pos, st[f"d_{name}_out"].float(), -1.0)
        if c["norm"] != "none":
            x = st[name].float()
            r = _inverse_norm(c["norm"], x)
            n = x * r
            if w is not None:
                weights.append((du * n).sum((0, 1), dtype=torch.float64).float())
                du = du * w
            dot = (du * n).sum(-1, keepdim=True)
            du = r * (du - n * (dot / D if c["norm"] == "rms" else dot))
        grads.append(du.to(dt))
    return (*grads, *weights)


def _plain_append(st):
    """s <- max(s of the tokens already in the page, s of the new ones); the old codes follow a scale that grew."""
    c, pos = st["case"], _positions(st)
    seq = torch.searchsorted(st["cu"][1:].long(), torch.arange(st["T"], device="cuda"), right=True)
    page, slot = st["table"][seq, pos // PAGE].long(), pos % PAGE
    pool = st["k_scale"].shape[0]
    new = torch.zeros(pool, PAGE, dtype=torch.bool, device="cuda")
    new[page, slot] = True
    old_here = torch.zeros(pool, dtype=torch.long, device="cuda")     # rows of the page that hold earlier tokens
    old_here.scatter_reduce_(0, page, torch.where(pos // PAGE == st["first"][seq] // PAGE, st["first"][seq] % PAGE, 0), "amax")
    old = torch.arange(PAGE, device="cuda")[None, :] < old_here[:, None]
    touched = new.any(1)
    w64 = None if st["k_weight"] is None else st["k_weight"].double()
    new_k = _norm_turn(c, pos, st["k"].double(), w64)
    for name, tokens in (("k", new_k), ("v", st["v"].float())):
        codes, scale = st[name + "_cache"], st[name + "_scale"]
        h = scale.shape[1]
        x = torch.zeros(pool, PAGE, h, D, device="cuda", dtype=tokens.dtype)
        x[page, slot] = tokens
        x = x.transpose(1, 2)
        s = _pow2_scale(torch.where(x.isfinite(), x, torch.zeros_like(x)).abs().amax((2, 3)))
        s = torch.where((old_here > 0)[:, None], torch.maximum(s, scale), s)
        again = _codes(codes.float() * scale[:, :, None, None], s[:, :, None, None])
        fresh = _codes(x, s[:, :, None, None])
        sel = lambda m: (m & touched[:, None])[:, None, :, None]  # noqa: E731
        raw = torch.where(sel(new), fresh.view(torch.uint8), torch.where(sel(old), again.view(torch.uint8), codes.view(torch.uint8)))
        codes.view(torch.uint8).copy_(raw)
        scale.copy_(torch.where(touched[:, None], s, scale))
    q = _norm_turn(c, pos, st["q"].float(), st["q_weight"]).to(TYPES[c["dtype"]])
    return st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], q


def _with_states(st):
    """(xp, row): each sequence's state and tokens one after another, fp32, and the row of each token."""
    c, W = st["case"], st["case"]["width"]
    T, n, C = st["T"], c["n"], st["x"].shape[1]
    seq = torch.searchsorted(st["cu"][1:].long(), torch.arange(T, device="cuda"), right=True)
    row = torch.arange(T, device="cuda") + (W - 1) * (seq + 1)
    xp = torch.zeros(T + n * (W - 1), C, device="cuda")
    xp[row] = st["x"].float()
    if st["state"] is not None:
        xp[_edge_rows(st, 0)] = st["state"].float()
    return xp, row


def _edge_rows(st, end):
    """[n, W - 1]: the first (end 0) or last (end 1) W - 1 rows of each sequence and its state."""
    W = st["case"]["width"]
    i = torch.arange(st["case"]["n"], device="cuda")
    begin = st["cu"].long()[end:end + st["case"]["n"]] + i * (W - 1)
    return begin[:, None] + torch.arange(W - 1, device="cuda")[None, :]


def _taps(st, xp, row):
    W, w = st["case"]["width"], st["weight"]
    u = torch.zeros_like(xp[row])
    for j in range(W):
        u = torch.addcmul(u, xp[row - (W - 1) + j], w[:, j])
    return u if st["bias"] is None else u + st["bias"]


def _plain_conv(st):
    c = st["case"]
    xp, row = _with_states(st)
    u = _taps(st, xp, row)
    y = u * torch.sigmoid(u) if c["silu"] else u
    y = y.view(st["T"], -1, D)
    if c["norm"]:
        y[:, :2 * c["h_qk"]] *= _inverse_norm("unit", y[:, :2 * c["h_qk"]])
    dt = TYPES[c["dtype"]]
    q, k, v = (x.to(dt) for x in y.split([c["h_qk"], c["h_qk"], c["h_v"]], dim=1))
    last = xp[_edge_rows(st, 1)].to(dt)
    if c["op"] == "step":
        st["state"].copy_(last)
        last = st["state"]
    return q, k, v, last


def _plain_conv_bwd(st):
    c, W = st["case"], st["case"]["width"]
    xp, row = _with_states(st)
    u = _taps(st, xp, row)
    sig = torch.sigmoid(u)
    y = (u * sig if c["silu"] else u).view(st["T"], -1, D)
    dy = torch.cat(st["d_out"], 1).float()
    if c["norm"]:
        part = y[:, :2 * c["h_qk"]]
        r = _inverse_norm("unit", part)
        unit = part * r
        g = dy[:, :2 * c["h_qk"]]
        dy[:, :2 * c["h_qk"]] = r * (g - unit * (g * unit).sum(-1, keepdim=True))
    du = dy.view(st["T"], -1)
    if c["silu"]:
        du = du * (sig + u * sig * (1 - sig))
    dxp = torch.zeros_like(xp)
    dw = []
    for j in range(W):
        at = row - (W - 1) + j
        dxp[at] += du * st["weight"][:, j]
        dw.append((du * xp[at]).sum(0, dtype=torch.float64).float())
    if st["d_final"] is not None:
        dxp[_edge_rows(st, 1)] += st["d_final"].float()
    dt = TYPES[c["dtype"]]
    outs = [dxp[row].to(dt), torch.stack(dw, 1)]
    if st["bias"] is not None:
        outs.append(du.sum(0, dtype=torch.float64).float())
    if st["state"] is not None:
        outs.append(dxp[_edge_rows(st, 0)].to(dt))
    return tuple(outs)


def run(st):
    c = st["case"]
    if not own:
        return {"rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "append": _plain_append, "conv": _plain_conv, "step": _plain_conv,
                "conv_bwd": _plain_conv_bwd}[c["op"]](st)
    import gated_deltanet_linear_fwd_gb300 as gdn
    if c["op"] == "rope":
        return gdn.gdn_qk_rope(st["q"], st["k"], st["rope"], st["positions"], st["cu_arg"], norm=c["norm"], q_weight=st["q_weight"],
                               k_weight=st["k_weight"], eps=EPS, q_out=st["q_out"], k_out=st["k_out"])
    if c["op"] == "rope_bwd":
        grads = gdn.gdn_qk_rope_bwd(st["q"], st["k"], st["d_q_out"], st["d_k_out"], st["rope"], st["positions"], st["cu_arg"],
                                    norm=c["norm"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS, d_q=st["q_out"],
                                    d_k=st["k_out"], workspace=st["workspace"])
        return tuple(g for g in grads if g is not None)
    if c["op"] == "append":
        q = gdn.gdn_kv_append_rope(st["cache"], st["k"], st["v"], st["kv_lens"], st["table"], st["cu_arg"], rope=st["rope"],
                                   norm=c["norm"], k_weight=st["k_weight"], q=st["q"], q_weight=st["q_weight"], eps=EPS,
                                   q_out=st["q_out"])
        return st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], q
    how = dict(activation="silu" if c["silu"] else "none", norm=c["norm"], eps=EPS)
    if c["op"] == "conv":
        q, k, v = st["out"]
        return gdn.gdn_conv_fwd(st["x"], st["weight"], c["h_qk"], st["bias"], st["state"], st["cu_arg"], q=q, k=k, v=v,
                                final_state=st["final"], **how)
    if c["op"] == "step":
        q, k, v = st["out"]
        return *gdn.gdn_conv_step(st["x"], st["state"], st["weight"], c["h_qk"], st["bias"], q=q, k=k, v=v, **how), st["state"]
    grads = gdn.gdn_conv_bwd(st["x"], st["weight"], c["h_qk"], *st["d_out"], st["bias"], st["state"], st["d_final"], st["cu_arg"],
                             workspace=st["workspace"], **how)
    return tuple(g for g in grads if g is not None)


# ---------------------------------------------------------------- 64 bits
def _rotated64(case, pos, x, weight):
    """The definition with complex numbers: z e^(i p f) for the pairs z of each head."""
    x = x.double()
    if case["norm"] != "none":
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) * (1 if case["norm"] == "rms" else D) + EPS)
    if weight is not None:
        x = x * weight.double()
    half = case["rot"] // 2
    grow = case["factor"]
    freqs = []
    for i in range(half):
        f = (10000.0 * (grow ** (half / (half - 1)) if case["scaling"] == "ntk" else 1.0)) ** (-i / half)
        turns = 4096 * f / (2 * math.pi)
        kept = {"none": 1.0, "ntk": 1.0, "linear": 0.0, "parts": min(1.0, max(0.0, (turns - 1) / 31))}[case["scaling"]]
        freqs.append(f * (kept + (1 - kept) / grow))
    spin = torch.outer(pos.double(), torch.tensor(freqs, dtype=torch.float64, device="cuda"))
    size = 1 + 0.1 * math.log(grow) if case["scaling"] == "parts" else 1.0
    spin = torch.polar(torch.full_like(spin, size), spin)[:, None, :]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if case["layout"] == "half":
        z = torch.complex(turned[..., :half], turned[..., half:]) * spin
        turned = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.complex(turned[..., 0::2], turned[..., 1::2]) * spin
        turned = torch.stack([z.real, z.imag], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _e4m3_64(y):
    """Nearest e4m3 value, ties to even, of finite 64-bit numbers; larger ones become 448."""
    e = (torch.frexp(y)[1] - 1).clamp(min=-6)
    step = _two_to_the(e - 3)
    return (torch.round(y / step) * step).clamp(-TOP, TOP)


def _two_to_the(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_append(st, case):
    lens, past = _lens(case), _past(case)
    pos = torch.cat([torch.arange(a, a + b, device="cuda") for a, b in zip(past, lens)])
    table, cu = st["table"].tolist(), st["cu"].tolist()
    outs = {}
    for name in ("k", "v"):
        codes, scale = st[name + "_cache"].double(), st[name + "_scale"].double()
        x = _rotated64(case, pos, st["k"], st["k_weight"]) if name == "k" else st["v"].double()
        for i, (nq, old) in enumerate(zip(lens, past)):
            kv = old + nq
            for p in range(old // PAGE, -(-kv // PAGE)) if nq else ():
                a, b = max(old, p * PAGE), min(kv, (p + 1) * PAGE)
                page, lo, hi = table[i][p], a - p * PAGE, b - p * PAGE
                rows = x[cu[i] + a - old:cu[i] + b - old].transpose(0, 1)
                top = rows.abs().amax((1, 2))
                e = torch.frexp(top)[1] - 10             # 448 * 2^e < top * 2, so e or e + 1 or e + 2 is the smallest
                e = e + (TOP * _two_to_the(e) < top)
                e = e + (TOP * _two_to_the(e) < top)
                s = _two_to_the(torch.where(top > 0, e, E_MIN).clamp(E_MIN, E_MAX))
                if lo:
                    s = torch.maximum(s, scale[page])
                    codes[page, :, :lo] = _e4m3_64(codes[page, :, :lo] * (scale[page] / s)[:, None, None])
                codes[page, :, lo:hi] = _e4m3_64(rows / s[:, None, None])
                scale[page] = s
        outs[name] = (codes, scale)
    return outs["k"][0], outs["v"][0], outs["k"][1], outs["v"][1], _rotated64(case, pos, st["q"], st["q_weight"])


def _conv64(case, x, weight, bias, state, lens):
    """q, k, v and the last inputs, sequence by sequence."""
    W, outs, last, at = case["width"], [], [], 0
    for i, length in enumerate(lens):
        own_x = torch.cat([state[i], x[at:at + length]])
        at += length
        u = sum(own_x[j:j + length] * weight[:, j] for j in range(W))
        u = u + bias if bias is not None else u
        outs.append(u / (1 + torch.exp(-u)) if case["silu"] else u)
        last.append(own_x[length:])
    y = torch.cat(outs).view(sum(lens), -1, D)
    h = case["h_qk"]
    parts = [y[:, :h], y[:, h:2 * h], y[:, 2 * h:]]
    if case["norm"]:
        parts[:2] = [p / torch.sqrt((p * p).sum(-1, keepdim=True) + EPS) for p in parts[:2]]
    return (*parts, torch.stack(last))


def exact(case, seed):
    st = prepare(case, seed)
    lens = _lens(case)
    if case["op"] == "append":
        if sum(-(-b // PAGE) + 1 for b in lens) > 6000:     # page by page
            return None
        return _exact_append(st, case)
    if case["op"] in ("rope", "rope_bwd"):
        pos = torch.cat([torch.arange(case["start"], case["start"] + b, device="cuda") for b in lens])
        if case["op"] == "rope":
            return tuple(_rotated64(case, pos, st[x], st[x + "_weight"]) for x in "qk")
        grads, weights = [], []
        for name in "qk":
            x = st[name].double().requires_grad_()
            w = None if st[name + "_weight"] is None else st[name + "_weight"].double().requires_grad_()
            y = _rotated64(case, pos, x, w)
            got = torch.autograd.grad((y * st[f"d_{name}_out"].double()).sum(), [x] if w is None else [x, w])
            grads.append(got[0])
            weights += got[1:]
        return (*grads, *weights)
    leaf = lambda t: None if t is None else t.double().requires_grad_(case["op"] == "conv_bwd")  # noqa: E731
    x, weight, bias = leaf(st["x"]), leaf(st["weight"]), leaf(st["bias"])
    state = leaf(st["state"])
    zeros = torch.zeros(case["n"], case["width"] - 1, x.shape[1], dtype=torch.float64, device="cuda")
    outs = _conv64(case, x, weight, bias, zeros if state is None else state, lens)
    if case["op"] != "conv_bwd":
        return outs
    total = sum((y * d.double()).sum() for y, d in zip(outs[:3], st["d_out"]))
    if st["d_final"] is not None:
        total = total + (outs[3] * st["d_final"].double()).sum()
    return torch.autograd.grad(total, [t for t in (x, weight, bias, state) if t is not None])
