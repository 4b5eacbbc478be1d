"""ctypes view of libgdn.so, the C ABI declared in include/gdn.h.

Loading fails loudly when the library has not been built: there is no other
implementation behind these names.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_OK = 0
GDN_ERR_INVALID_ARG = 1
GDN_ERR_UNSUPPORTED = 2
GDN_ERR_MISALIGNED = 3
GDN_ERR_CUDA = 4
GDN_ERR_DEVICE_TIMEOUT = 5
GDN_ERR_WORKSPACE = 6
GDN_ERR_DEVICE_CHECK = 7

GDN_BF16 = 0
GDN_F32 = 1
GDN_TOL_FIXED = 0
GDN_TOL_NOISE = 1

GDN_CP_OFF = 0
GDN_CP_EXACT = 1
GDN_CP_WARMUP = 2
GDN_CP_AUTO = 3

EXPORTED = ["gdn_cp_plan", "gdn_chunk_fwd", "gdn_status_string", "gdn_last_cuda_error",
            "gdn_get_device_status", "gdn_cp_head_modes", "gdn_set_trace_events", "gdn_trace_last", "gdn_chunk_fwd_static",
            "gdn_get_static_device_status", "gdn_decode_step", "gdn_debug_stall_ns", "gdn_bwd_workspace_bytes",
            "gdn_chunk_bwd", "gdn_chunk_fwd_train", "gdn_kv_append", "gdn_kv_read", "gdn_kv_attn_plan", "gdn_kv_attn",
            "gdn_rope_table", "gdn_qk_rope", "gdn_qk_rope_bwd_workspace_bytes", "gdn_qk_rope_bwd", "gdn_kv_append_rope",
            "gdn_conv_fwd", "gdn_conv_bwd_workspace_bytes", "gdn_conv_bwd", "gdn_conv_step"]

GDN_KV_PAGE = 64

GDN_ROPE_HALF, GDN_ROPE_INTERLEAVED = 0, 1
GDN_ROPE_PLAIN, GDN_ROPE_LINEAR, GDN_ROPE_NTK, GDN_ROPE_PARTS = 0, 1, 2, 3
GDN_NORM_NONE, GDN_NORM_RMS, GDN_NORM_UNIT = 0, 1, 2
GDN_ACT_NONE, GDN_ACT_SILU = 0, 1


class gdn_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("h_qk", ctypes.c_int), ("h_v", ctypes.c_int),
                ("d_k", ctypes.c_int), ("d_v", ctypes.c_int), ("n_seqs", ctypes.c_int),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int)]


class gdn_cp_opts(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("lambda_", ctypes.c_float), ("warmup_chunks", ctypes.c_int),
                ("warmup_tol", ctypes.c_float), ("sm_count", ctypes.c_int), ("tol_rule", ctypes.c_int)]


class gdn_cp_plan_t(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("n_seqs", ctypes.c_int), ("T_total", ctypes.c_int),
                ("h_v", ctypes.c_int), ("h_qk", ctypes.c_int), ("dtype", ctypes.c_int),
                ("lambda_q8", ctypes.c_int), ("warmup_chunks", ctypes.c_int),
                ("warmup_tol", ctypes.c_float), ("sm_count", ctypes.c_int), ("tol_rule", ctypes.c_int),
                ("n_seg_total", ctypes.c_int), ("max_seg_chunks", ctypes.c_int),
                ("max_chunks", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t),
                ("off_head", ctypes.c_size_t), ("off_seg_bound", ctypes.c_size_t),
                ("off_R", ctypes.c_size_t), ("off_Sloc", ctypes.c_size_t), ("off_Sstart", ctypes.c_size_t),
                ("n_chunks_total", ctypes.c_int), ("off_chunk_map", ctypes.c_size_t),
                ("off_wy", ctypes.c_size_t)]


class gdn_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("status", ctypes.c_void_p), ("n_pages", ctypes.c_int),
                ("h_kv", ctypes.c_int), ("d", ctypes.c_int)]


class gdn_kv_dims(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("T", ctypes.c_int), ("h_q", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("causal", ctypes.c_int), ("window", ctypes.c_int), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]


class gdn_kv_plan_t(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("rows", ctypes.c_int), ("max_row_tiles", ctypes.c_int),
                ("n_ctas", ctypes.c_int), ("item_cost", ctypes.c_int), ("n_seqs", ctypes.c_int), ("T", ctypes.c_int),
                ("h_q", ctypes.c_int), ("h_kv", ctypes.c_int), ("dtype", ctypes.c_int), ("max_q_len", ctypes.c_int),
                ("off_desc", ctypes.c_size_t), ("off_ml", ctypes.c_size_t), ("off_o", ctypes.c_size_t),
                ("workspace_bytes", ctypes.c_size_t)]


class gdn_rope_opts(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int), ("scaling", ctypes.c_int), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double)]


class gdn_rope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot", ctypes.c_int), ("layout", ctypes.c_int), ("magnitude", ctypes.c_float)]


class gdn_rope_dims(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("T", ctypes.c_int), ("h_q", ctypes.c_int), ("h_k", ctypes.c_int),
                ("norm", ctypes.c_int), ("eps", ctypes.c_float), ("dtype", ctypes.c_int), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64),
                ("dq_stride", ctypes.c_int64), ("dk_stride", ctypes.c_int64)]


class gdn_conv_dims(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("T", ctypes.c_int), ("h_qk", ctypes.c_int), ("h_v", ctypes.c_int),
                ("width", ctypes.c_int), ("activation", ctypes.c_int), ("norm", ctypes.c_int), ("eps", ctypes.c_float),
                ("dtype", ctypes.c_int), ("x_stride", ctypes.c_int64), ("dx_stride", ctypes.c_int64)]


# The dims of the calls that a decode step makes, from their fields' values: a
# third of the time that filling a Structure field by field takes.
_pack_rope_dims = struct.Struct("@iiiiifi4x6q").pack
_pack_conv_dims = struct.Struct("@iiiiiiifi4x2q").pack
_pack_kv_dims = struct.Struct("@iiiiiifi4q").pack
assert struct.calcsize("@iiiiifi4x6q") == ctypes.sizeof(gdn_rope_dims)
assert struct.calcsize("@iiiiiiifi4x2q") == ctypes.sizeof(gdn_conv_dims)
assert struct.calcsize("@iiiiiifi4q") == ctypes.sizeof(gdn_kv_dims)


def rope_dims(*fields) -> gdn_rope_dims:
    return gdn_rope_dims.from_buffer_copy(_pack_rope_dims(*fields))


def conv_dims(*fields) -> gdn_conv_dims:
    return gdn_conv_dims.from_buffer_copy(_pack_conv_dims(*fields))


def kv_dims(*fields) -> gdn_kv_dims:
    return gdn_kv_dims.from_buffer_copy(_pack_kv_dims(*fields))


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load libgdn.so (built in-tree by gated_deltanet_linear_fwd_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"libgdn.so not found at {path}: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` (nvcc, sm_103a)")
        lib = ctypes.CDLL(path)
        vp, i32p, fp = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_float)
        lib.gdn_cp_plan.argtypes = [ctypes.POINTER(gdn_dims), i32p, ctypes.POINTER(gdn_cp_opts),
                                    ctypes.POINTER(gdn_cp_plan_t)]
        lib.gdn_cp_plan.restype = ctypes.c_int
        lib.gdn_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(gdn_dims),
                                      ctypes.POINTER(gdn_cp_plan_t), vp, ctypes.c_size_t, vp]
        lib.gdn_chunk_fwd.restype = ctypes.c_int
        lib.gdn_status_string.argtypes = [ctypes.c_int]
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_last_cuda_error.argtypes = []
        lib.gdn_last_cuda_error.restype = ctypes.c_int
        lib.gdn_get_device_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
        lib.gdn_get_device_status.restype = ctypes.c_int
        lib.gdn_cp_head_modes.argtypes = [vp, ctypes.POINTER(gdn_cp_plan_t), i32p, fp, vp]
        lib.gdn_cp_head_modes.restype = ctypes.c_int
        lib.gdn_chunk_fwd_static.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(gdn_dims),
                                             ctypes.POINTER(gdn_cp_plan_t), vp]
        lib.gdn_chunk_fwd_static.restype = ctypes.c_int
        lib.gdn_get_static_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
        lib.gdn_get_static_device_status.restype = ctypes.c_int
        lib.gdn_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(gdn_dims), vp]
        lib.gdn_decode_step.restype = ctypes.c_int
        lib.gdn_set_trace_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]
        lib.gdn_set_trace_events.restype = ctypes.c_int
        lib.gdn_trace_last.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.c_int]
        lib.gdn_trace_last.restype = ctypes.c_int
        lib.gdn_bwd_workspace_bytes.argtypes = [ctypes.POINTER(gdn_cp_plan_t), ctypes.POINTER(ctypes.c_size_t)]
        lib.gdn_bwd_workspace_bytes.restype = ctypes.c_int
        lib.gdn_chunk_bwd.argtypes = [vp] * 15 + [ctypes.POINTER(gdn_dims), ctypes.POINTER(gdn_cp_plan_t), vp,
                                                  ctypes.c_size_t, ctypes.c_int, vp]
        lib.gdn_chunk_fwd_train.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(gdn_dims),
                                            ctypes.POINTER(gdn_cp_plan_t), vp, ctypes.c_size_t, vp]
        lib.gdn_chunk_fwd_train.restype = ctypes.c_int
        lib.gdn_chunk_bwd.restype = ctypes.c_int
        lib.gdn_debug_stall_ns.argtypes = [ctypes.c_uint32]
        lib.gdn_debug_stall_ns.restype = ctypes.c_int
        kc, kd, kp = ctypes.POINTER(gdn_kv_cache), ctypes.POINTER(gdn_kv_dims), ctypes.POINTER(gdn_kv_plan_t)
        for fn in (lib.gdn_kv_append, lib.gdn_kv_read):
            fn.argtypes = [vp, vp, vp, vp, vp, kc, kd, vp]
            fn.restype = ctypes.c_int
        lib.gdn_kv_attn_plan.argtypes = [kd, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, kp]
        lib.gdn_kv_attn_plan.restype = ctypes.c_int
        lib.gdn_kv_attn.argtypes = [vp, vp, vp, vp, kc, vp, vp, kd, kp, vp, ctypes.c_size_t, vp]
        lib.gdn_kv_attn.restype = ctypes.c_int
        rp, rd, cd, sp = (ctypes.POINTER(x) for x in (gdn_rope, gdn_rope_dims, gdn_conv_dims, ctypes.c_size_t))
        for name, args in (("gdn_rope_table", [ctypes.POINTER(gdn_rope_opts), ctypes.POINTER(ctypes.c_uint64)]),
                           ("gdn_qk_rope", [vp] * 6 + [rp, vp, vp, rd, vp]),
                           ("gdn_qk_rope_bwd_workspace_bytes", [sp]),
                           ("gdn_qk_rope_bwd", [vp] * 6 + [rp] + [vp] * 6 + [rd, vp, ctypes.c_size_t, vp]),
                           ("gdn_kv_append_rope", [vp] * 9 + [kc, kd, rp, ctypes.c_int, ctypes.c_float, vp]),
                           ("gdn_conv_fwd", [vp] * 9 + [cd, vp]),
                           ("gdn_conv_bwd_workspace_bytes", [cd, sp]),
                           ("gdn_conv_bwd", [vp] * 13 + [cd, vp, ctypes.c_size_t, vp]),
                           ("gdn_conv_step", [vp] * 7 + [cd, vp])):
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        _lib = lib
        return lib


class GDNError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load()
        msg = lib.gdn_status_string(status).decode()
        if status == GDN_ERR_CUDA:
            msg += f" (cuda error {lib.gdn_last_cuda_error()})"
        super().__init__(f"{where}: {msg}")
        self.status = status


def check(status: int, where: str):
    if status != GDN_OK:
        raise GDNError(status, where)
