"""Python binding of the C ABI (include/gdn.h): argument marshalling only.

Every step of the forward runs in libgdn.so's CUDA kernels; PyTorch only
provides device memory and the stream.  The names mirror the C entry points.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional, Sequence

import torch

from . import _lib as L

_MODES = {"off": L.GDN_CP_OFF, "exact": L.GDN_CP_EXACT, "warmup": L.GDN_CP_WARMUP, "auto": L.GDN_CP_AUTO}
_DT = {torch.bfloat16: L.GDN_BF16, torch.float32: L.GDN_F32}
_TOL_RULES = {"fixed": L.GDN_TOL_FIXED, "noise": L.GDN_TOL_NOISE}


@dataclasses.dataclass
class Plan:
    """A filled gdn_cp_plan_t together with the dims it was made for."""
    raw: L.gdn_cp_plan_t
    dims: L.gdn_dims
    cu_seqlens_host: Optional[list]

    @property
    def mode(self) -> str:
        return {v: k for k, v in _MODES.items()}[self.raw.mode]

    @property
    def workspace_bytes(self) -> int:
        return int(self.raw.workspace_bytes)

    @property
    def n_seg_total(self) -> int:
        return int(self.raw.n_seg_total)


def _cu_list(cu_seqlens) -> Optional[list]:
    if cu_seqlens is None:
        return None
    if isinstance(cu_seqlens, torch.Tensor):
        return [int(x) for x in cu_seqlens.tolist()]
    return [int(x) for x in cu_seqlens]


def gdn_cp_plan(*, T: int, h_qk: int, h_v: int, B: int = 1, cu_seqlens=None,
                dtype: torch.dtype = torch.bfloat16, mode: str = "auto", lambda_: float = 0.0,
                warmup_chunks: int = 8, warmup_tol: float = 1e-4, sm_count: int = 0,
                scale: float = 0.0, d_k: int = 128, d_v: int = 128, tol_rule: str = "noise") -> Plan:
    """Host-only planning (gdn_cp_plan).  T = tokens per row (varlen: total).
    tol_rule: "noise" (a warmup's tolerance is at least the exact path's noise
    floor at the segment start) or "fixed" (warmup_tol alone)."""
    cu = _cu_list(cu_seqlens)
    n_seqs = B if cu is None else len(cu) - 1
    dims = L.gdn_dims(B, T, h_qk, h_v, d_k, d_v, n_seqs, scale, _DT.get(dtype, -1))
    opts = L.gdn_cp_opts(_MODES[mode], lambda_, warmup_chunks, warmup_tol, sm_count, _TOL_RULES[tol_rule])
    raw = L.gdn_cp_plan_t()
    cu_arr = None if cu is None else (ctypes.c_int32 * len(cu))(*cu)
    L.check(L.load().gdn_cp_plan(ctypes.byref(dims), cu_arr, ctypes.byref(opts), ctypes.byref(raw)),
            "gdn_cp_plan")
    return Plan(raw, dims, cu)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def gdn_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                  initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                  *, plan: Optional[Plan] = None, out: Optional[torch.Tensor] = None,
                  final_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
                  workspace: Optional[torch.Tensor] = None, stream=None, scale: float = 0.0,
                  mode: str = "auto", lambda_: float = 0.0, warmup_chunks: int = 8,
                  warmup_tol: float = 1e-4, tol_rule: str = "noise", for_backward: bool = False):
    """The chunked-prefill forward (gdn_chunk_fwd).

    q,k [B,T,h_qk,128] or [T,h_qk,128]; v [.., h_v, 128]; g,beta [.., h_v] fp32;
    initial_state [N,h_v,128,128] fp32 or None; cu_seqlens int32 [N+1] on the
    device (varlen, B = 1) or None.  Returns (o, final_state or None).
    for_backward: gdn_chunk_fwd_train -- the workspace (of gdn_bwd_workspace_bytes)
    keeps what gdn_chunk_bwd(..., reuse_forward=True) needs with the same plan.
    """
    batched = q.dim() == 4
    B = q.shape[0] if batched else 1
    T = q.shape[-3]
    h_qk, h_v = q.shape[-2], v.shape[-2]
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if g.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError("g and beta must be float32")
    if plan is None:
        plan = gdn_cp_plan(T=T, h_qk=h_qk, h_v=h_v, B=B, cu_seqlens=cu_seqlens, dtype=q.dtype, mode=mode,
                           lambda_=lambda_, warmup_chunks=warmup_chunks, warmup_tol=warmup_tol, scale=scale,
                           tol_rule=tol_rule)
    dims = L.gdn_dims(B, T, h_qk, h_v, q.shape[-1], v.shape[-1], plan.raw.n_seqs, scale, _DT.get(q.dtype, -1))
    if out is None:
        out = torch.empty_like(v)
    if final_state is None and output_final_state:
        final_state = torch.empty(plan.raw.n_seqs, h_v, 128, 128, dtype=torch.float32, device=q.device)
    if workspace is None:
        n_ws = gdn_bwd_workspace_bytes(plan) if for_backward else plan.workspace_bytes
        workspace = torch.empty(max(n_ws, 256), dtype=torch.uint8, device=q.device)
    if initial_state is not None and (initial_state.dtype != torch.float32 or not initial_state.is_contiguous()):
        raise ValueError("initial_state must be contiguous float32")
    fn = L.load().gdn_chunk_fwd_train if for_backward else L.load().gdn_chunk_fwd
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens), _ptr(out),
            _ptr(final_state), ctypes.byref(dims), ctypes.byref(plan.raw), _ptr(workspace), workspace.numel(),
            _stream_handle(stream))
    L.check(st, "gdn_chunk_fwd_train" if for_backward else "gdn_chunk_fwd")
    return out, final_state


def gdn_bwd_workspace_bytes(plan: Plan) -> int:
    """Device workspace bytes gdn_chunk_bwd needs for `plan` (gdn_bwd_workspace_bytes)."""
    n = ctypes.c_size_t(0)
    L.check(L.load().gdn_bwd_workspace_bytes(ctypes.byref(plan.raw), ctypes.byref(n)), "gdn_bwd_workspace_bytes")
    return int(n.value)


def gdn_chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                  d_out: torch.Tensor, initial_state: Optional[torch.Tensor] = None,
                  d_final_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                  *, plan: Optional[Plan] = None, grads=None, workspace: Optional[torch.Tensor] = None,
                  stream=None, scale: float = 0.0, mode: str = "auto", lambda_: float = 0.0,
                  want_initial_state_grad: bool = True, reuse_forward: bool = False):
    """Gradients of sum(o * d_out) + sum(final_state * d_final_state) (gdn_chunk_bwd).

    Inputs as gdn_chunk_fwd (bf16 q/k/v); d_out like v (bf16); d_final_state
    [N, h_v, 128, 128] fp32 or None.  grads: optional preallocated
    (dq, dk, dv, dg, dbeta, dh0).  Returns (dq, dk, dv, dg, dbeta, dh0 or None).
    reuse_forward: `workspace` and `plan` are those of a gdn_chunk_fwd(...,
    for_backward=True) on the same inputs; the forward is not recomputed.
    """
    batched = q.dim() == 4
    B = q.shape[0] if batched else 1
    T = q.shape[-3]
    h_qk, h_v = q.shape[-2], v.shape[-2]
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("d_out", d_out)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if q.dtype != torch.bfloat16 or d_out.dtype != torch.bfloat16:
        raise ValueError("the backward takes bf16 q/k/v and d_out")
    if reuse_forward and (workspace is None or plan is None):
        raise ValueError("reuse_forward needs the plan and workspace of the gdn_chunk_fwd(for_backward=True) call")
    if g.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError("g and beta must be float32")
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous float32")
    if plan is None:
        plan = gdn_cp_plan(T=T, h_qk=h_qk, h_v=h_v, B=B, cu_seqlens=cu_seqlens, dtype=q.dtype, mode=mode,
                           lambda_=lambda_, scale=scale)
    dims = L.gdn_dims(B, T, h_qk, h_v, q.shape[-1], v.shape[-1], plan.raw.n_seqs, scale, _DT.get(q.dtype, -1))
    if grads is None:
        dh0 = (torch.empty(plan.raw.n_seqs, h_v, 128, 128, dtype=torch.float32, device=q.device)
               if want_initial_state_grad else None)
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(g),
                 torch.empty_like(beta), dh0)
    dq, dk, dv, dg, dbeta, dh0 = grads
    if workspace is None:
        workspace = torch.empty(max(gdn_bwd_workspace_bytes(plan), 256), dtype=torch.uint8, device=q.device)
    st = L.load().gdn_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                _ptr(cu_seqlens), _ptr(d_out), _ptr(d_final_state), _ptr(dq), _ptr(dk), _ptr(dv),
                                _ptr(dg), _ptr(dbeta), _ptr(dh0), ctypes.byref(dims), ctypes.byref(plan.raw),
                                _ptr(workspace), workspace.numel(), int(bool(reuse_forward)),
                                _stream_handle(stream))
    L.check(st, "gdn_chunk_bwd")
    return dq, dk, dv, dg, dbeta, dh0


def gdn_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                    state: torch.Tensor, *, out: Optional[torch.Tensor] = None, scale: float = 0.0, stream=None):
    """One new token per sequence (gdn_decode_step): q,k [B,h_qk,128], v [B,h_v,128]
    (bf16 or fp32), g,beta [B,h_v] fp32, state [B,h_v,128,128] fp32 (H = S^T,
    updated in place).  Returns o [B,h_v,128]."""
    B, h_qk, h_v = q.shape[0], q.shape[1], v.shape[1]
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("state", state)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if g.dtype != torch.float32 or beta.dtype != torch.float32 or state.dtype != torch.float32:
        raise ValueError("g, beta and state must be float32")
    if out is None:
        out = torch.empty_like(v)
    dims = L.gdn_dims(B, 1, h_qk, h_v, q.shape[-1], v.shape[-1], B, scale, _DT.get(q.dtype, -1))
    st = L.load().gdn_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(out),
                                  ctypes.byref(dims), _stream_handle(stream))
    L.check(st, "gdn_decode_step")
    return out


def gdn_get_device_status(workspace: torch.Tensor, stream=None):
    """(code, detail) of the status word of the last call on this workspace (synchronises)."""
    code, detail = ctypes.c_int(), ctypes.c_int()
    L.check(L.load().gdn_get_device_status(_ptr(workspace), _stream_handle(stream), ctypes.byref(code),
                                           ctypes.byref(detail)), "gdn_get_device_status")
    return code.value, detail.value


_DETAILS = {1: "a bulk copy's wait", 2: "an MMA's wait", 3: "the chunk index or segments disagree with the plan",
            4: "segments combined out of order", 5: "a value outside the fp16 range of the MMA operands",
            6: "the test hook's stall", 7: "key/value offsets or lengths outside their bounds",
            8: "a key/value page outside the pool"}


def describe_device_status(code: int, detail: int) -> str:
    """Text for a (code, detail) pair read from the status word: code is a
    gdn_status (0, 5 timeout or 7 check); detail says which check or wait
    tripped (100 + b: a bounded wait on mbarrier b of the kernel)."""
    if code == L.GDN_OK:
        return "ok"
    what = {L.GDN_ERR_DEVICE_TIMEOUT: "timeout", L.GDN_ERR_DEVICE_CHECK: "check failed"}.get(code, f"code {code}")
    if detail >= 100:
        where = f"the bounded wait on barrier {detail - 100}"
    else:
        where = _DETAILS.get(detail, f"detail {detail}")
    return f"{what}: {where}"


def gdn_debug_stall_ns(ns: int) -> None:
    """Test hook (gdn_debug_stall_ns): while ns > 0 every later forward's
    chunk-local kernel waits ns nanoseconds on a barrier nothing arrives on,
    so the call takes its timeout path; 0 turns it off."""
    L.check(L.load().gdn_debug_stall_ns(int(ns)), "gdn_debug_stall_ns")


def gdn_get_static_device_status(stream=None):
    """(code, detail) of the status word of the last gdn_chunk_fwd_static call
    on the current device (synchronises)."""
    code, detail = ctypes.c_int(), ctypes.c_int()
    L.check(L.load().gdn_get_static_device_status(_stream_handle(stream), ctypes.byref(code), ctypes.byref(detail)),
            "gdn_get_static_device_status")
    return code.value, detail.value


def gdn_cp_head_modes(workspace: torch.Tensor, plan: Plan, stream=None):
    """Per (sequence, head): the mode taken (1 exact, 2 warmup, 0 off) and log warmup bound."""
    n = plan.raw.n_seqs * plan.raw.h_v
    modes = (ctypes.c_int32 * n)()
    bounds = (ctypes.c_float * n)()
    L.check(L.load().gdn_cp_head_modes(_ptr(workspace), ctypes.byref(plan.raw), modes, bounds,
                                       _stream_handle(stream)), "gdn_cp_head_modes")
    shape = (plan.raw.n_seqs, plan.raw.h_v)
    return (torch.tensor(list(modes), dtype=torch.int32).reshape(shape),
            torch.tensor(list(bounds), dtype=torch.float32).reshape(shape))


def gdn_set_trace_events(events) -> None:
    """Register torch.cuda.Event objects (enable_timing=True, recorded once so
    they exist) for per-kernel timing of this thread's next gdn_chunk_fwd
    calls; [] turns it off."""
    n = len(events)
    arr = (ctypes.c_void_p * max(n, 1))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    L.check(L.load().gdn_set_trace_events(arr if n else None, n), "gdn_set_trace_events")


def gdn_trace_last() -> list:
    """Names of the kernels the last gdn_chunk_fwd on this thread launched."""
    names = (ctypes.c_char_p * 16)()
    n = L.load().gdn_trace_last(names, 16)
    return [names[i].decode() for i in range(n)]


def gdn_chunk_fwd_static(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *, plan: Plan, out, final_state=None,
                         stream=None):
    """gdn_chunk_fwd_static: the forward with the library's built-in 8 MiB
    device workspace, for callers that cannot allocate device memory.  The
    caller passes every input and output (nothing is allocated here)."""
    dims = L.gdn_dims(q.shape[0] if q.dim() == 4 else 1, q.shape[-3], q.shape[-2], v.shape[-2], q.shape[-1],
                      v.shape[-1], plan.raw.n_seqs, 0.0, _DT.get(q.dtype, -1))
    st = L.load().gdn_chunk_fwd_static(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                       _ptr(cu_seqlens), _ptr(out), _ptr(final_state), ctypes.byref(dims),
                                       ctypes.byref(plan.raw), _stream_handle(stream))
    L.check(st, "gdn_chunk_fwd_static")
    return out, final_state


class KVCache:
    """The 8-bit key/value cache (gdn_kv_cache): k, v [n_pages, h_kv, 64, 128]
    float8_e4m3fn codes, k_scale, v_scale [n_pages, h_kv] fp32 powers of two,
    all contiguous on one device; status int32 [2], zeroed here.

    KVCache.empty makes a new one; which pages belong to which sequence is the
    caller's (page_table)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if k.dim() != 4 or k.shape[2] != L.GDN_KV_PAGE or k.shape != v.shape:
            raise ValueError(f"k and v must be [n_pages, h_kv, {L.GDN_KV_PAGE}, 128]")
        for name, t, dt in (("k", k, torch.float8_e4m3fn), ("v", v, torch.float8_e4m3fn),
                            ("k_scale", k_scale, torch.float32), ("v_scale", v_scale, torch.float32)):
            if t.dtype != dt or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous {dt}")
        if k_scale.shape != k.shape[:2] or v_scale.shape != k.shape[:2]:
            raise ValueError("k_scale and v_scale must be [n_pages, h_kv]")
        self.device_index = k.get_device()  # negative: not on a GPU, and of no use to the operators
        if not v.get_device() == k_scale.get_device() == v_scale.get_device() == self.device_index:
            raise ValueError("k, v, k_scale and v_scale must be on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.status = torch.zeros(2, dtype=torch.int32, device=k.device)
        self.raw = L.gdn_kv_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                  self.status.data_ptr(), k.shape[0], k.shape[1], k.shape[3])

    @classmethod
    def empty(cls, n_pages: int, h_kv: int, device="cuda") -> "KVCache":
        codes = lambda: torch.zeros(n_pages, h_kv, L.GDN_KV_PAGE, 128, dtype=torch.uint8,  # noqa: E731
                                    device=device).view(torch.float8_e4m3fn)
        scale = lambda: torch.ones(n_pages, h_kv, dtype=torch.float32, device=device)  # noqa: E731
        return cls(codes(), codes(), scale(), scale())


def _kv_rows(name: str, t: torch.Tensor, heads: int, cache: KVCache) -> int:
    """Token stride of a [T, heads, 128] tensor whose tokens are whole; 0 when it is packed."""
    if t.get_device() != cache.device_index or t.dim() != 3 or t.size(1) != heads:
        raise ValueError(f"{name} must be a tensor [T, {heads}, 128] on the cache's device")
    if t.is_contiguous():
        return 0
    s = t.stride()
    if s[2] != 1 or (s[1] != t.size(2) and heads > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if t.size(0) <= 1:
        return 0
    if s[0] < heads * t.size(2):  # an expanded view's 0 would select packed tokens, past the end of what lies behind it
        raise ValueError(f"{name}: tokens must not overlap")
    return s[0]


def _kv_ints(cache: KVCache, kv_lens: torch.Tensor, page_table: torch.Tensor, cu_seqlens: Optional[torch.Tensor]):
    """(sequences, row length of the table, address of the offsets), of tensors the kernels may read."""
    dev = cache.device_index
    if dev < 0:
        raise ValueError("the cache must be on a GPU")
    if kv_lens.dtype != torch.int32 or page_table.dtype != torch.int32 or not kv_lens.get_device() == page_table.get_device() == dev:
        raise ValueError("kv_lens and page_table must be int32 tensors on the cache's device")
    n = kv_lens.shape[0]
    if page_table.dim() != 2 or page_table.shape[0] != n or not page_table.is_contiguous() or not kv_lens.is_contiguous():
        raise ValueError("page_table must be contiguous [n_seqs, max_pages]")
    if cu_seqlens is None:
        return n, page_table.shape[1], None
    if (cu_seqlens.dtype != torch.int32 or cu_seqlens.shape != (n + 1,) or not cu_seqlens.is_contiguous()
            or cu_seqlens.get_device() != dev):
        raise ValueError("cu_seqlens must be contiguous int32 [n_seqs + 1] on the cache's device")
    return n, page_table.shape[1], cu_seqlens.data_ptr()


def _raw_stream(stream, t: torch.Tensor) -> int:
    """The stream's handle; by default the current one of t's device, without a
    Stream object around it (a microsecond of a call that takes eight).  The
    kernels run on the current device, which t has to be on."""
    dev = t.get_device()
    if dev != torch._C._cuda_getDevice():
        raise ValueError("the tensors must be on the current device")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _kv_empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """Memory of the stream the kernels run on, so that its reuse is ordered with them."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def gdn_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, kv_lens: torch.Tensor, page_table: torch.Tensor,
                  cu_seqlens: Optional[torch.Tensor] = None, *, stream=None) -> None:
    """Quantises new tokens into the cache (gdn_kv_append): k, v [T, h_kv, 128]
    bf16 or fp32, packed over the sequences by cu_seqlens (None: T / n_seqs
    each); kv_lens int32 [n_seqs] counts the new tokens too.  k and v may be
    views with a larger token stride (parts of one projection's output)."""
    n, max_pages, cu = _kv_ints(cache, kv_lens, page_table, cu_seqlens)
    h_kv = cache.raw.h_kv
    ks, vs = _kv_rows("k", k, h_kv, cache), _kv_rows("v", v, h_kv, cache)
    if v.dtype != k.dtype or v.shape != k.shape or k.shape[2] != 128:
        raise ValueError("k and v must be alike, with 128 elements a head")
    dims = L.gdn_kv_dims(n, k.shape[0], h_kv, max_pages, 1, 0, 0.0, _DT.get(k.dtype, -1), 0, ks, vs, 0)
    st = L.load().gdn_kv_append(k.data_ptr(), v.data_ptr(), kv_lens.data_ptr(), page_table.data_ptr(), cu, cache.raw,
                                dims, _raw_stream(stream, k))
    L.check(st, "gdn_kv_append")


def gdn_kv_read(cache: KVCache, kv_lens: torch.Tensor, page_table: torch.Tensor,
                cu_seqlens: Optional[torch.Tensor] = None, *, T: Optional[int] = None,
                dtype: torch.dtype = torch.bfloat16, k_out: Optional[torch.Tensor] = None,
                v_out: Optional[torch.Tensor] = None, stream=None):
    """The cache's values of the last n_i tokens of each sequence (gdn_kv_read),
    exact in bf16 or fp32: (k, v), each [T, h_kv, 128].  T: their number over
    all sequences, when no outputs are given."""
    n, max_pages, cu = _kv_ints(cache, kv_lens, page_table, cu_seqlens)
    h_kv = cache.raw.h_kv
    if k_out is None or v_out is None:
        if T is None:
            raise ValueError("gdn_kv_read needs T or both outputs")
        shape = (T, h_kv, 128)
        k_out = _kv_empty(shape, dtype, cache.k.device, stream) if k_out is None else k_out
        v_out = _kv_empty(shape, dtype, cache.k.device, stream) if v_out is None else v_out
    ks, vs = _kv_rows("k_out", k_out, h_kv, cache), _kv_rows("v_out", v_out, h_kv, cache)
    if v_out.dtype != k_out.dtype or v_out.shape != k_out.shape or k_out.shape[2] != 128:
        raise ValueError("k_out and v_out must be alike, with 128 elements a head")
    dims = L.gdn_kv_dims(n, k_out.shape[0], h_kv, max_pages, 1, 0, 0.0, _DT.get(k_out.dtype, -1), 0, ks, vs, 0)
    st = L.load().gdn_kv_read(k_out.data_ptr(), v_out.data_ptr(), kv_lens.data_ptr(), page_table.data_ptr(), cu,
                              cache.raw, dims, _raw_stream(stream, k_out))
    L.check(st, "gdn_kv_read")
    return k_out, v_out


@dataclasses.dataclass
class KVPlan:
    """A filled gdn_kv_plan_t and the masks and scale it was made for."""
    raw: L.gdn_kv_plan_t
    causal: bool
    window: int
    scale: float

    @property
    def workspace_bytes(self) -> int:
        return int(self.raw.workspace_bytes)


def gdn_kv_attn_plan(*, T: int, n_seqs: int, h_q: int, h_kv: int, max_q_len: int = 0, max_kv_len: int = 0,
                     max_pages: int = 0, dtype: torch.dtype = torch.bfloat16, causal: bool = True, window: int = 0,
                     scale: float = 0.0, sm_count: int = 0) -> KVPlan:
    """Host-only planning of gdn_kv_attn.  max_q_len: the most tokens a sequence
    brings (0: any number, planned as T / n_seqs); max_kv_len: the longest
    sequence expected (0: 64 max_pages)."""
    if not max_pages:
        max_pages = max(1, -(-max_kv_len // L.GDN_KV_PAGE))
    dims = L.gdn_kv_dims(n_seqs, T, h_q, max_pages, int(causal), window, scale, _DT.get(dtype, -1), 0, 0, 0, 0)
    raw = L.gdn_kv_plan_t()
    L.check(L.load().gdn_kv_attn_plan(dims, h_kv, max_q_len, max_kv_len, sm_count, raw), "gdn_kv_attn_plan")
    return KVPlan(raw, causal, window, scale)


def gdn_kv_attn(q: torch.Tensor, cache: KVCache, kv_lens: torch.Tensor, page_table: torch.Tensor,
                cu_seqlens: Optional[torch.Tensor] = None, *, plan: Optional[KVPlan] = None,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                workspace: Optional[torch.Tensor] = None, causal: bool = True, window: int = 0, scale: float = 0.0,
                max_q_len: int = 0, max_kv_len: int = 0, stream=None):
    """Attention of each new token over its sequence's cached keys and values
    (gdn_kv_attn): q [T, h_q, 128] bf16 or fp32, packed like gdn_kv_append's k
    and v, which go into the cache first.  Returns (out [T, h_q, 128],
    lse [T, h_q] fp32 or None); neither has a history, there is no backward.
    causal, window, scale and the bounds are the plan's when one is given; a plan
    holds for calls of the same sizes.  max_q_len, the most tokens a sequence
    brings, may be left out: offsets alone then plan for T / n_seqs."""
    n, max_pages, cu = _kv_ints(cache, kv_lens, page_table, cu_seqlens)
    T, h_q, d = q.shape
    qs = _kv_rows("q", q, h_q, cache)
    if d != 128:
        raise ValueError("q must have 128 elements a head")
    if plan is None:
        plan = gdn_kv_attn_plan(T=T, n_seqs=n, h_q=h_q, h_kv=cache.raw.h_kv,
                                max_q_len=max_q_len or (0 if cu is not None else T // max(n, 1)), max_kv_len=max_kv_len,
                                max_pages=max_pages, dtype=q.dtype, causal=causal, window=window, scale=scale)
    if out is None:
        out = _kv_empty(q.shape, q.dtype, q.device, stream)
    elif out.dtype != q.dtype or out.shape != q.shape:
        raise ValueError("out must be like q")
    if lse is None:
        if return_lse:
            lse = _kv_empty((T, h_q), torch.float32, q.device, stream)
    elif (lse.dtype != torch.float32 or lse.shape != (T, h_q) or not lse.is_contiguous()
          or lse.get_device() != cache.device_index):
        raise ValueError("lse must be contiguous float32 [T, h_q] on the cache's device")
    if workspace is None:
        workspace = _kv_empty(max(plan.workspace_bytes, 256), torch.uint8, q.device, stream)
    elif workspace.get_device() != cache.device_index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous, on the cache's device")
    dims = L.gdn_kv_dims(n, T, h_q, max_pages, int(plan.causal), plan.window, plan.scale, _DT.get(q.dtype, -1), qs, 0, 0,
                         _kv_rows("out", out, h_q, cache))
    st = L.load().gdn_kv_attn(q.data_ptr(), kv_lens.data_ptr(), page_table.data_ptr(), cu, cache.raw, out.data_ptr(),
                              None if lse is None else lse.data_ptr(), dims, plan.raw, workspace.data_ptr(),
                              workspace.numel(), _raw_stream(stream, q))
    L.check(st, "gdn_kv_attn")
    return out, lse


_SCALINGS = {"none": L.GDN_ROPE_PLAIN, "linear": L.GDN_ROPE_LINEAR, "ntk": L.GDN_ROPE_NTK, "parts": L.GDN_ROPE_PARTS}
_LAYOUTS = {"half": L.GDN_ROPE_HALF, "interleaved": L.GDN_ROPE_INTERLEAVED}
_NORMS = {"none": L.GDN_NORM_NONE, "rms": L.GDN_NORM_RMS, "unit": L.GDN_NORM_UNIT}
_ACTIVATIONS = {"none": L.GDN_ACT_NONE, "silu": L.GDN_ACT_SILU}


def _choice(what: str, table: dict, name: str) -> int:
    if name not in table:
        raise ValueError(f"{what} must be one of {', '.join(table)}")
    return table[name]


class Rope:
    """Rotary positions (gdn_rope): turns int64 [rot / 2] on the device, the bits
    of gdn_rope_table's uint64; layout "half" or "interleaved"; magnitude of the
    turned elements (0: 1).  gdn_rope_table makes one."""

    def __init__(self, turns: torch.Tensor, layout: str = "half", magnitude: float = 0.0):
        if turns.dtype != torch.int64 or turns.dim() != 1 or not turns.is_contiguous():
            raise ValueError("turns must be contiguous int64 [rot / 2]")
        self.turns, self.rot, self.device_index = turns, 2 * turns.shape[0], turns.get_device()
        self.raw = L.gdn_rope(turns.data_ptr(), self.rot, _choice("layout", _LAYOUTS, layout), magnitude)


def gdn_rope_table(rot: int = 128, *, base: float = 10000.0, layout: str = "half", scaling: str = "none", factor: float = 1.0,
                   original_len: float = 0.0, low: float = 1.0, high: float = 32.0, magnitude: float = 0.0,
                   device="cuda") -> Rope:
    """The frequencies of rotary positions (gdn_rope_table), for the first `rot`
    elements of a head.  scaling, for contexts `factor` times longer: "none",
    "linear", "ntk" or "parts" (by the turns a pair makes over original_len
    tokens: up to `low` slowed down, from `high` on kept)."""
    opts = L.gdn_rope_opts(rot, _choice("scaling", _SCALINGS, scaling), base, factor, original_len, low, high)
    turns = (ctypes.c_uint64 * max(1, rot // 2))()
    L.check(L.load().gdn_rope_table(opts, turns), "gdn_rope_table")
    signed = [x - (1 << 64) if x >> 63 else x for x in turns]
    return Rope(torch.tensor(signed, dtype=torch.int64, device=device), layout, magnitude)


def _spacing(name: str, t: torch.Tensor, inner: int) -> int:
    """Token stride of [T, ..] or [B, T, ..], not packed, whose last `inner` dimensions
    are a token, whole, the tokens evenly spaced; 0 for one token."""
    shape, strides = t.shape, t.stride()
    lead = len(shape) - inner
    if strides[-1] != 1 or (inner == 2 and shape[-2] > 1 and strides[-2] != shape[-1]):
        raise ValueError(f"{name}: a token's elements must be contiguous")
    n, step = shape[lead - 1], strides[lead - 1]
    if lead == 2 and shape[0] > 1:
        if n > 1 and strides[0] != n * step:
            raise ValueError(f"{name}: tokens must be evenly spaced")
        n, step = shape[0] * n, step if n > 1 else strides[0]
    if n <= 1:
        return 0
    if step < (shape[-1] if inner == 1 else shape[-2] * shape[-1]):
        # an expanded view's 0 would select packed tokens, past the end of what lies behind it
        raise ValueError(f"{name}: tokens must not overlap")
    return step


def _empty_like(t: torch.Tensor, stream) -> torch.Tensor:
    """As _kv_empty, packed, of t's shape, type and device."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)
    return _kv_empty(t.shape, t.dtype, t.device, stream)


def _place(name: str, t: torch.Tensor, shape, inner: int, dtype: torch.dtype, device: int):
    """(address, token stride) of t, checked to be of that shape, type and device."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, of the call's type and on its device")
    return t.data_ptr(), 0 if t.is_contiguous() else _spacing(name, t, inner)


def _f32(name: str, t: Optional[torch.Tensor], shape, device: int):
    """Address of a float32 tensor, or None."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be contiguous float32 {list(shape)} on the call's device")
    return t.data_ptr()


def _i32(name: str, t: Optional[torch.Tensor], numel: int, device: int):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.numel() != numel or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be contiguous int32 with {numel} elements on the call's device")
    return t.data_ptr()


def _rope_raw(rope: Optional[Rope], device: int):
    if rope is None:
        return None
    if rope.device_index != device:
        raise ValueError("rope must be on the call's device")
    return rope.raw


def _call(x: torch.Tensor, stream):
    """(type, device, stream handle) of a call on x."""
    device = x.get_device()
    if device < 0:
        raise ValueError("the tensors must be on a GPU")
    return x.dtype, device, _raw_stream(stream, x)


def _sequences(lead, cu_seqlens: Optional[torch.Tensor], device: int):
    """(sequences, tokens, address of the offsets) of a call whose tensors begin with the dimensions [T] or [B, T]."""
    if len(lead) == 1:
        n, T = 1, lead[0]
    else:
        n, T = lead[0], lead[0] * lead[1]
    if cu_seqlens is None:
        return n, T, None
    if len(lead) == 2 and n != 1:
        raise ValueError("cu_seqlens is for packed tokens, not for a batch of rows")
    n = cu_seqlens.numel() - 1
    return n, T, _i32("cu_seqlens", cu_seqlens, n + 1, device)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _heads(name: str, t: torch.Tensor, like: torch.Tensor, dtype: torch.dtype, device: int):
    """(address, token stride, heads, shape) of queries or keys that go with `like`."""
    shape = t.shape
    n = len(shape)
    if (n != 3 and n != 4) or shape[-1] != 128 or (t is not like and shape[:-2] != like.shape[:-2]):
        raise ValueError(f"{name} must be [T, heads, 128] or [B, T, heads, 128], alike in q and k")
    if t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must be of the call's type and on its device")
    return t.data_ptr(), 0 if t.is_contiguous() else _spacing(name, t, 2), shape[-2], shape


_NO_HEADS = (None, 0, 0, None)


def gdn_qk_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], rope: Optional[Rope] = None,
                positions: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *, norm: str = "none",
                q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 0.0,
                q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Queries and keys, each head normalised ("none", "rms" or "unit"), then
    rotated by its token's position (gdn_qk_rope): q [T, h_q, 128], k [T, h_k, 128]
    or with a batch in front, bf16 or fp32; either may be None.  Positions: int32,
    one a token; else counted within each sequence of cu_seqlens, or each row.
    The tensors may be parts of one projection; an output may be its input.
    Returns (q_out, k_out), without a history (gdn_qk_rope_bwd)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k is needed")
    if (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError("q_out and k_out go with q and k")
    dtype, dev, handle = _call(x, stream)
    qp, qs, h_q, q_shape = _NO_HEADS if q is None else _heads("q", q, x, dtype, dev)
    kp, ks, h_k, k_shape = _NO_HEADS if k is None else _heads("k", k, x, dtype, dev)
    n, T, cu = _sequences((q_shape or k_shape)[:-2], cu_seqlens, dev)
    qo = ko = None
    qos = kos = 0
    if q is not None:
        if q_out is None:
            q_out = _empty_like(q, stream)
        qo, qos = _place("q_out", q_out, q_shape, 2, dtype, dev)
    if k is not None:
        if k_out is None:
            k_out = _empty_like(k, stream)
        ko, kos = _place("k_out", k_out, k_shape, 2, dtype, dev)
    st = L.load().gdn_qk_rope(qp, kp, _f32("q_weight", q_weight, (128,), dev), _f32("k_weight", k_weight, (128,), dev),
                              _i32("positions", positions, T, dev), cu, _rope_raw(rope, dev), qo, ko,
                              L.rope_dims(n, T, h_q, h_k, _choice("norm", _NORMS, norm), eps, _DT.get(dtype, -1), qs, ks, qos, kos,
                                          0, 0), handle)
    L.check(st, "gdn_qk_rope")
    return q_out, k_out


def gdn_qk_rope_bwd_workspace_bytes() -> int:
    """Device workspace of gdn_qk_rope_bwd, whatever its sizes."""
    n = ctypes.c_size_t(0)
    L.check(L.load().gdn_qk_rope_bwd_workspace_bytes(n), "gdn_qk_rope_bwd_workspace_bytes")
    return int(n.value)


def gdn_qk_rope_bwd(q: Optional[torch.Tensor], k: Optional[torch.Tensor], d_q_out: Optional[torch.Tensor],
                    d_k_out: Optional[torch.Tensor], rope: Optional[Rope] = None, positions: Optional[torch.Tensor] = None,
                    cu_seqlens: Optional[torch.Tensor] = None, *, norm: str = "none", q_weight: Optional[torch.Tensor] = None,
                    k_weight: Optional[torch.Tensor] = None, eps: float = 0.0, d_q: Optional[torch.Tensor] = None,
                    d_k: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of gdn_qk_rope (gdn_qk_rope_bwd), whose inputs come again.
    Returns (d_q, d_k, d_q_weight, d_k_weight), the latter fp32 [128] and None
    without the weight.  d_q may be d_q_out, d_k may be d_k_out."""
    if (q is None) != (d_q_out is None) or (k is None) != (d_k_out is None):
        raise ValueError("d_q_out and d_k_out go with q and k")
    if (q is None and d_q is not None) or (k is None and d_k is not None):
        raise ValueError("d_q and d_k go with q and k")
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k is needed")
    dtype, dev, handle = _call(x, stream)
    qp, qs, h_q, q_shape = _NO_HEADS if q is None else _heads("q", q, x, dtype, dev)
    kp, ks, h_k, k_shape = _NO_HEADS if k is None else _heads("k", k, x, dtype, dev)
    n, T, cu = _sequences((q_shape or k_shape)[:-2], cu_seqlens, dev)
    gq = gk = dqp = dkp = None
    gqs = gks = dqs = dks = 0
    if q is not None:
        gq, gqs = _place("d_q_out", d_q_out, q_shape, 2, dtype, dev)
        if d_q is None:
            d_q = _empty_like(q, stream)
        dqp, dqs = _place("d_q", d_q, q_shape, 2, dtype, dev)
    if k is not None:
        gk, gks = _place("d_k_out", d_k_out, k_shape, 2, dtype, dev)
        if d_k is None:
            d_k = _empty_like(k, stream)
        dkp, dks = _place("d_k", d_k, k_shape, 2, dtype, dev)
    qw, kw = _f32("q_weight", q_weight, (128,), dev), _f32("k_weight", k_weight, (128,), dev)
    dqw = None if qw is None else _empty_like(q_weight, stream)
    dkw = None if kw is None else _empty_like(k_weight, stream)
    if workspace is None and (dqw is not None or dkw is not None):
        workspace = _kv_empty(gdn_qk_rope_bwd_workspace_bytes(), torch.uint8, x.device, stream)
    st = L.load().gdn_qk_rope_bwd(qp, kp, qw, kw, _i32("positions", positions, T, dev), cu, _rope_raw(rope, dev), gq, gk, dqp, dkp,
                                  _at(dqw), _at(dkw),
                                  L.rope_dims(n, T, h_q, h_k, _choice("norm", _NORMS, norm), eps, _DT.get(dtype, -1), qs, ks, gqs,
                                              gks, dqs, dks), *_workspace(workspace, dev), handle)
    L.check(st, "gdn_qk_rope_bwd")
    return d_q, d_k, dqw, dkw


def _workspace(t: Optional[torch.Tensor], device: int):
    """(address, bytes) of a call's workspace."""
    if t is None:
        return None, 0
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError("workspace must be contiguous, on the call's device")
    return t.data_ptr(), t.numel() * t.element_size()


def gdn_kv_append_rope(cache: KVCache, k: torch.Tensor, v: torch.Tensor, kv_lens: torch.Tensor, page_table: torch.Tensor,
                       cu_seqlens: Optional[torch.Tensor] = None, *, rope: Optional[Rope] = None, norm: str = "none",
                       k_weight: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                       q_weight: Optional[torch.Tensor] = None, eps: float = 0.0, q_out: Optional[torch.Tensor] = None,
                       stream=None) -> Optional[torch.Tensor]:
    """gdn_kv_append of keys that are normalised and rotated on the way, and the
    queries of the same tokens beside them, in one launch (gdn_kv_append_rope).
    Positions are those of the cache.  Returns q_out [T, h_q, 128], or None
    without q; q_out may be q itself."""
    n, max_pages, cu = _kv_ints(cache, kv_lens, page_table, cu_seqlens)
    h_kv = cache.raw.h_kv
    shape = k.shape
    if len(shape) != 3 or shape[1] != h_kv or shape[2] != 128:
        raise ValueError(f"k must be [T, {h_kv}, 128]")
    dtype, dev, handle = _call(k, stream)
    if dev != cache.device_index:
        raise ValueError("k must be on the cache's device")
    kp, ks = k.data_ptr(), 0 if k.is_contiguous() else _spacing("k", k, 2)
    vp, vs = _place("v", v, shape, 2, dtype, dev)
    h_q, qp, qo, qs, qos = h_kv, None, None, 0, 0
    if q is not None:
        qp, qs, h_q, q_shape = _heads("q", q, k, dtype, dev)
        if q_out is None:
            q_out = _empty_like(q, stream)
        qo, qos = _place("q_out", q_out, q_shape, 2, dtype, dev)
    elif q_out is not None:
        raise ValueError("q_out goes with q")
    st = L.load().gdn_kv_append_rope(kp, vp, _f32("k_weight", k_weight, (128,), dev), qp, _f32("q_weight", q_weight, (128,), dev), qo,
                                     kv_lens.data_ptr(), page_table.data_ptr(), cu, cache.raw,
                                     L.kv_dims(n, shape[0], h_q, max_pages, 1, 0, 0.0, _DT.get(dtype, -1), qs, ks, vs, qos),
                                     _rope_raw(rope, dev), _choice("norm", _NORMS, norm), eps, handle)
    L.check(st, "gdn_kv_append_rope")
    return q_out


def _conv(x, weight, h_qk, bias, cu_seqlens, activation, norm, eps, stream):
    """What the calls of a convolution share: (dimensions before the channels,
    channels, value heads, sequences, tokens, taps, type, device, stream handle,
    addresses of weight, bias and offsets, the dims' values after the first two)."""
    shape = x.shape
    if len(shape) not in (2, 3):
        raise ValueError("x must be [T, C] or [B, T, C]")
    lead, C = shape[:-1], shape[-1]
    h_v = C // 128 - 2 * h_qk
    if C % 128 or h_qk < 1 or h_v < 1:
        raise ValueError("x must have (2 h_qk + h_v) * 128 channels")
    if weight.dim() != 2:
        raise ValueError("weight must be [C, W]")
    W = weight.shape[1]
    dtype, device, handle = _call(x, stream)
    n, T, cu = _sequences(lead, cu_seqlens, device)
    how = (h_qk, h_v, W, _choice("activation", _ACTIVATIONS, activation), 1 if norm else 0, eps, _DT.get(dtype, -1),
           0 if x.is_contiguous() else _spacing("x", x, 1))
    return (lead, C, h_v, n, T, W, dtype, device, handle, _f32("weight", weight, (C, W), device), _f32("bias", bias, (C,), device), cu,
            how)


def _packed(name: str, t: Optional[torch.Tensor], shape, dtype: torch.dtype, device: int):
    """Address of t, checked to be contiguous, of that shape, type and device; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}, of x's type, on its device")
    return t.data_ptr()


def gdn_conv_fwd(x: torch.Tensor, weight: torch.Tensor, h_qk: int, bias: Optional[torch.Tensor] = None,
                 initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
                 activation: str = "silu", norm: bool = True, eps: float = 0.0, q: Optional[torch.Tensor] = None,
                 k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                 output_final_state: bool = True, stream=None):
    """The short causal convolution before the gated delta rule (gdn_conv_fwd):
    x [T, C] packed by cu_seqlens, or [B, T, C], bf16 or fp32, C = (2 h_qk + h_v) *
    128 channels of q, k and v; weight [C, W] fp32, bias [C] fp32 or None;
    initial_state [N, W - 1, C] like x, or None.  norm: q's and k's heads to unit
    length.  Returns (q, k, v, final_state or None), q, k, v as gdn_chunk_fwd
    takes them, without a history (gdn_conv_bwd)."""
    lead, C, h_v, n, T, W, dtype, dev, handle, w, b, cu, how = _conv(x, weight, h_qk, bias, cu_seqlens, activation, norm, eps, stream)
    states, heads, v_heads = (n, W - 1, C), (*lead, h_qk, 128), (*lead, h_v, 128)
    if q is None:
        q = _kv_empty(heads, dtype, x.device, stream)
    if k is None:
        k = _kv_empty(heads, dtype, x.device, stream)
    if v is None:
        v = _kv_empty(v_heads, dtype, x.device, stream)
    if final_state is None and output_final_state:
        final_state = _kv_empty(states, dtype, x.device, stream)
    st = L.load().gdn_conv_fwd(x.data_ptr(), w, b, _packed("initial_state", initial_state, states, dtype, dev), cu,
                               _packed("q", q, heads, dtype, dev), _packed("k", k, heads, dtype, dev),
                               _packed("v", v, v_heads, dtype, dev), _packed("final_state", final_state, states, dtype, dev),
                               L.conv_dims(n, T, *how, 0), handle)
    L.check(st, "gdn_conv_fwd")
    return q, k, v, final_state


def gdn_conv_bwd_workspace_bytes(T: int, h_qk: int, h_v: int, *, n_seqs: int = 1, width: int = 4,
                                 dtype: torch.dtype = torch.bfloat16) -> int:
    """Device workspace of gdn_conv_bwd for calls of T tokens in all (gdn_conv_bwd_workspace_bytes)."""
    n = ctypes.c_size_t(0)
    dims = L.gdn_conv_dims(n_seqs, T, h_qk, h_v, width, L.GDN_ACT_SILU, 1, 0.0, _DT.get(dtype, -1), 0, 0)
    L.check(L.load().gdn_conv_bwd_workspace_bytes(dims, n), "gdn_conv_bwd_workspace_bytes")
    return int(n.value)


def gdn_conv_bwd(x: torch.Tensor, weight: torch.Tensor, h_qk: int, d_q: torch.Tensor, d_k: torch.Tensor, d_v: torch.Tensor,
                 bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                 d_final_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
                 activation: str = "silu", norm: bool = True, eps: float = 0.0, dx: Optional[torch.Tensor] = None,
                 want_initial_state_grad: Optional[bool] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of gdn_conv_fwd (gdn_conv_bwd), whose inputs come again; d_q, d_k,
    d_v and d_final_state (None: zero) like its outputs.  Returns (dx, d_weight,
    d_bias or None, d_initial_state or None): the bias's without a bias and, unless
    want_initial_state_grad says so, the state's without a state are None."""
    lead, C, h_v, n, T, W, dtype, dev, handle, w, b, cu, how = _conv(x, weight, h_qk, bias, cu_seqlens, activation, norm, eps, stream)
    states, heads = (n, W - 1, C), (*lead, h_qk, 128)
    gq, gk = _packed("d_q", d_q, heads, dtype, dev), _packed("d_k", d_k, heads, dtype, dev)
    gv = _packed("d_v", d_v, (*lead, h_v, 128), dtype, dev)
    before, after = _packed("initial_state", initial_state, states, dtype, dev), _packed("d_final_state", d_final_state, states, dtype, dev)
    if dx is None:
        dx = _empty_like(x, stream)
    dxp, dx_stride = _place("dx", dx, x.shape, 1, dtype, dev)
    d_state = None
    if initial_state is not None if want_initial_state_grad is None else want_initial_state_grad:
        d_state = _kv_empty(states, dtype, x.device, stream) if initial_state is None else _empty_like(initial_state, stream)
    d_weight = _empty_like(weight, stream)
    d_bias = None if bias is None else _empty_like(bias, stream)
    lib, dims = L.load(), L.conv_dims(n, T, *how, dx_stride)
    if workspace is None:
        size = ctypes.c_size_t(0)
        L.check(lib.gdn_conv_bwd_workspace_bytes(dims, size), "gdn_conv_bwd_workspace_bytes")
        workspace = _kv_empty(max(256, int(size.value)), torch.uint8, x.device, stream)
    st = lib.gdn_conv_bwd(x.data_ptr(), w, b, before, cu, gq, gk, gv, after, dxp, d_weight.data_ptr(), _at(d_bias), _at(d_state), dims,
                          *_workspace(workspace, dev), handle)
    L.check(st, "gdn_conv_bwd")
    return dx, d_weight, d_bias, d_state


def gdn_conv_step(x: torch.Tensor, state: torch.Tensor, weight: torch.Tensor, h_qk: int, bias: Optional[torch.Tensor] = None, *,
                  activation: str = "silu", norm: bool = True, eps: float = 0.0, q: Optional[torch.Tensor] = None,
                  k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None, stream=None):
    """One new token a sequence (gdn_conv_step): x [N, C], state [N, W - 1, C] like x,
    gdn_conv_fwd's final_state, updated in place.  Returns (q, k, v), [N, heads,
    128], as gdn_decode_step takes them."""
    if x.dim() != 2:
        raise ValueError("x must be [N, C]")
    _, C, h_v, _, n, W, dtype, dev, handle, w, b, _, how = _conv(x, weight, h_qk, bias, None, activation, norm, eps, stream)
    if state is None:
        raise ValueError("state is needed")
    heads, v_heads = (n, h_qk, 128), (n, h_v, 128)
    if q is None:
        q = _kv_empty(heads, dtype, x.device, stream)
    if k is None:
        k = _kv_empty(heads, dtype, x.device, stream)
    if v is None:
        v = _kv_empty(v_heads, dtype, x.device, stream)
    st = L.load().gdn_conv_step(x.data_ptr(), w, b, _packed("state", state, (n, W - 1, C), dtype, dev),
                                _packed("q", q, heads, dtype, dev), _packed("k", k, heads, dtype, dev),
                                _packed("v", v, v_heads, dtype, dev), L.conv_dims(n, n, *how, 0), handle)
    L.check(st, "gdn_conv_step")
    return q, k, v
