"""Thin Python binding of libgdn.so (the C ABI declared in include/gdn.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of the library. Functions named gdn_* mirror the C entry points one
for one and take torch tensors (or None for a NULL pointer), which the caller
keeps until the stream has done with them; the lower-case helpers at the end
allocate outputs and workspaces with torch, on the stream that they run on, and
call them.

The library is loaded from this package directory. If it is missing, importing
this module raises ImportError: there is no fallback of any kind.
"""
import ctypes
import functools
import inspect
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgdn.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is not built; run `python -m chunked_gated_delta_04_amd.build` "
        "(hipcc, gfx950) first")
_lib = ctypes.CDLL(_LIB_PATH)

GDN_OK = 0
STATUS_NAMES = {
    0: "GDN_OK", 1: "GDN_ERR_NULL", 2: "GDN_ERR_SHAPE", 3: "GDN_ERR_UNSUPPORTED",
    4: "GDN_ERR_SEQLENS", 5: "GDN_ERR_INDEX", 6: "GDN_ERR_WORKSPACE", 7: "GDN_ERR_HIP",
    8: "GDN_ERR_ALIGN", 9: "GDN_ERR_SCRATCH",
}
EXPORTED = (
    "gdn_status_string", "gdn_num_chunks", "gdn_chunk_saved_size",
    "gdn_chunk_fwd_workspace_size", "gdn_chunk_bwd_workspace_size",
    "gdn_chunk_bwd_recompute_workspace_size",
    "gdn_chunk_fwd", "gdn_chunk_fwd_paged", "gdn_chunk_bwd", "gdn_chunk_bwd_recompute",
    "gdn_chunk_transition", "gdn_recurrent_step",
    "gdn_conv_fwd", "gdn_conv_fwd_paged", "gdn_conv_bwd", "gdn_conv_bwd_workspace_size",
    "gdn_conv_update",
    "gdn_chunk_fwd_timed", "gdn_chunk_bwd_timed", "gdn_stage_name",
    "gdn_chunk_fwd_paged_noalloc", "gdn_chunk_fwd_paged_noalloc_max_bytes",
    "gdn_linear_saved_size", "gdn_linear_fwd_workspace_size", "gdn_linear_bwd_workspace_size",
    "gdn_linear_fwd", "gdn_linear_fwd_paged", "gdn_linear_bwd", "gdn_linear_step",
    "gdn_rotary", "gdn_rotary_bwd", "gdn_rotary_inv_freq",
    "gdn_rmsnorm_fwd", "gdn_rmsnorm_bwd", "gdn_rmsnorm_bwd_workspace_size",
    "gdn_kv_append", "gdn_attn_fwd", "gdn_attn_fwd_paged", "gdn_attn_step", "gdn_attn_bwd",
    "gdn_attn_fwd_workspace_size", "gdn_attn_fwd_paged_workspace_size",
    "gdn_attn_step_workspace_size", "gdn_attn_bwd_workspace_size",
)
GDN_MAX_STAGES = 8


class GdnProblem(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
        ("HV", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32),
        ("chunk", ctypes.c_int32), ("scale", ctypes.c_float),
        ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_host", ctypes.c_void_p),
    ]


class GdnConvProblem(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int32), ("T", ctypes.c_int32), ("C", ctypes.c_int32),
        ("W", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_host", ctypes.c_void_p),
    ]


class GdnLinearProblem(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
        ("HV", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_host", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
    ]


class GdnRotaryProblem(ctypes.Structure):
    _fields_ = [(_n, ctypes.c_int32) for _n in ("T", "HQ", "HK", "D", "R", "interleaved", "dtype")] + [
        ("mscale", ctypes.c_float), ("positions", ctypes.c_void_p), ("N", ctypes.c_int32),
        ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_host", ctypes.c_void_p),
        ("offsets", ctypes.c_void_p),
    ] + [(_n, ctypes.c_int64) for _n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")]


class GdnRmsnormProblem(ctypes.Structure):
    _fields_ = [(_n, ctypes.c_int32) for _n in ("rows", "D", "dtype", "unit_offset", "group")] + [
        ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64),
    ]


class GdnAttnProblem(ctypes.Structure):
    _fields_ = [(_n, ctypes.c_int32) for _n in ("N", "T", "HQ", "HK", "D", "dtype", "window", "sinks")] + [
        ("scale", ctypes.c_float), ("cu_seqlens", ctypes.c_void_p),
        ("cu_seqlens_host", ctypes.c_void_p),
    ] + [(_n, ctypes.c_int64) for _n in ("q_stride", "k_stride", "v_stride")]


class GdnKvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (_n, ctypes.c_int32) for _n in ("pages", "page_size", "columns")] + [
        (_n, ctypes.c_int64) for _n in ("table_stride", "page_stride", "token_stride", "head_stride")
    ] + [("page_table", ctypes.c_void_p), ("offsets", ctypes.c_void_p)]


class GdnKvAppendProblem(ctypes.Structure):
    _fields_ = [(_n, ctypes.c_int32) for _n in ("N", "T", "HQ", "HK", "D", "R", "interleaved", "dtype")] + [
        ("mscale", ctypes.c_float), ("cu_seqlens", ctypes.c_void_p),
        ("cu_seqlens_host", ctypes.c_void_p),
    ] + [(_n, ctypes.c_int64) for _n in ("q_stride", "k_stride", "v_stride", "q_out_stride")]


class GdnError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} "
                         f"({gdn_status_string(status)})")


_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_i32 = ctypes.c_int32
_P = ctypes.POINTER(GdnProblem)

_lib.gdn_status_string.restype = ctypes.c_char_p
_lib.gdn_status_string.argtypes = [ctypes.c_int]
_lib.gdn_num_chunks.restype = ctypes.c_int64
_lib.gdn_num_chunks.argtypes = [_P]
for _n in ("gdn_chunk_saved_size", "gdn_chunk_fwd_workspace_size", "gdn_chunk_bwd_workspace_size",
           "gdn_chunk_bwd_recompute_workspace_size"):
    getattr(_lib, _n).restype = _sz
    getattr(_lib, _n).argtypes = [_P]
_lib.gdn_chunk_fwd.restype = ctypes.c_int
_lib.gdn_chunk_fwd.argtypes = [_P] + [_vp] * 10 + [_sz, _vp]
_lib.gdn_chunk_fwd_paged.restype = ctypes.c_int
_lib.gdn_chunk_fwd_paged.argtypes = [_P] + [_vp] * 6 + [_i32] + [_vp] * 6 + [_sz, _vp]
_lib.gdn_chunk_fwd_paged_noalloc.restype = ctypes.c_int
_lib.gdn_chunk_fwd_paged_noalloc.argtypes = [_P] + [_vp] * 6 + [_i32] + [_vp] * 6
_lib.gdn_chunk_fwd_paged_noalloc_max_bytes.restype = _sz
_lib.gdn_chunk_fwd_paged_noalloc_max_bytes.argtypes = []
_lib.gdn_chunk_bwd.restype = ctypes.c_int
_lib.gdn_chunk_bwd.argtypes = [_P] + [_vp] * 15 + [_sz, _vp]
_lib.gdn_chunk_bwd_recompute.restype = ctypes.c_int
_lib.gdn_chunk_bwd_recompute.argtypes = [_P] + [_vp] * 15 + [_sz, _vp]
_lib.gdn_chunk_transition.restype = ctypes.c_int
_lib.gdn_chunk_transition.argtypes = [_P] + [_vp] * 8 + [_sz, _vp]
_lib.gdn_chunk_fwd_timed.restype = ctypes.c_int
_lib.gdn_chunk_fwd_timed.argtypes = ([_P] + [_vp] * 10 + [_sz, _vp] +
                                     [ctypes.POINTER(_vp), ctypes.POINTER(ctypes.c_int)])
_lib.gdn_chunk_bwd_timed.restype = ctypes.c_int
_lib.gdn_chunk_bwd_timed.argtypes = ([_P] + [_vp] * 15 + [_sz, _vp] +
                                     [ctypes.POINTER(_vp), ctypes.POINTER(ctypes.c_int)])
_CP = ctypes.POINTER(GdnConvProblem)
_lib.gdn_conv_fwd.restype = ctypes.c_int
_lib.gdn_conv_fwd.argtypes = [_CP] + [_vp] * 7
_lib.gdn_conv_fwd_paged.restype = ctypes.c_int
_lib.gdn_conv_fwd_paged.argtypes = [_CP] + [_vp] * 4 + [_i32] + [_vp] * 5
_lib.gdn_conv_bwd_workspace_size.restype = _sz
_lib.gdn_conv_bwd_workspace_size.argtypes = [_CP]
_lib.gdn_conv_bwd.restype = ctypes.c_int
_lib.gdn_conv_bwd.argtypes = [_CP] + [_vp] * 10 + [_sz, _vp]
_lib.gdn_conv_update.restype = ctypes.c_int
_lib.gdn_conv_update.argtypes = [_i32] * 4 + [_vp] * 4 + [_i32] + [_vp] * 4
_lib.gdn_stage_name.restype = ctypes.c_char_p
_lib.gdn_stage_name.argtypes = [ctypes.c_int, ctypes.c_int]
_lib.gdn_recurrent_step.restype = ctypes.c_int
_lib.gdn_recurrent_step.argtypes = ([_i32] * 5 + [ctypes.c_float] + [_vp] * 8 + [_i32] +
                                    [_vp] * 4)

_LP = ctypes.POINTER(GdnLinearProblem)
for _n in ("gdn_linear_saved_size", "gdn_linear_fwd_workspace_size",
           "gdn_linear_bwd_workspace_size"):
    getattr(_lib, _n).restype = _sz
    getattr(_lib, _n).argtypes = [_LP]
_lib.gdn_linear_fwd.restype = ctypes.c_int
_lib.gdn_linear_fwd.argtypes = [_LP] + [_vp] * 9 + [_sz, _vp]
_lib.gdn_linear_fwd_paged.restype = ctypes.c_int
_lib.gdn_linear_fwd_paged.argtypes = [_LP] + [_vp] * 5 + [_i32] + [_vp] * 6 + [_sz, _vp]
_lib.gdn_linear_bwd.restype = ctypes.c_int
_lib.gdn_linear_bwd.argtypes = [_LP] + [_vp] * 12 + [_sz, _vp]
_lib.gdn_linear_step.restype = ctypes.c_int
_lib.gdn_linear_step.argtypes = [_LP] + [_vp] * 5 + [_i32] + [_vp] * 4

_RP = ctypes.POINTER(GdnRotaryProblem)
for _n in ("gdn_rotary", "gdn_rotary_bwd"):
    getattr(_lib, _n).restype = ctypes.c_int
    getattr(_lib, _n).argtypes = [_RP] + [_vp] * 6
_lib.gdn_rotary_inv_freq.restype = ctypes.c_int
_lib.gdn_rotary_inv_freq.argtypes = [_i32, ctypes.c_double, _i32, ctypes.c_double, ctypes.c_double,
                                     _vp, ctypes.POINTER(ctypes.c_float)]
_NP = ctypes.POINTER(GdnRmsnormProblem)
_lib.gdn_rmsnorm_fwd.restype = ctypes.c_int
_lib.gdn_rmsnorm_fwd.argtypes = [_NP] + [_vp] * 9
_lib.gdn_rmsnorm_bwd.restype = ctypes.c_int
_lib.gdn_rmsnorm_bwd.argtypes = [_NP] + [_vp] * 8 + [_sz, _vp]
_lib.gdn_rmsnorm_bwd_workspace_size.restype = _sz
_lib.gdn_rmsnorm_bwd_workspace_size.argtypes = [_NP]

_AP, _KP = ctypes.POINTER(GdnAttnProblem), ctypes.POINTER(GdnKvCache)
for _n, _args in (("gdn_attn_fwd", [_AP]), ("gdn_attn_fwd_paged", [_AP, _KP]),
                  ("gdn_attn_step", [_AP, _KP]), ("gdn_attn_bwd", [_AP])):
    getattr(_lib, _n + "_workspace_size").restype = _sz
    getattr(_lib, _n + "_workspace_size").argtypes = _args
    getattr(_lib, _n).restype = ctypes.c_int
_lib.gdn_attn_fwd.argtypes = [_AP] + [_vp] * 6 + [_sz, _vp]
_lib.gdn_attn_fwd_paged.argtypes = [_AP, _KP] + [_vp] * 4 + [_sz, _vp]
_lib.gdn_attn_step.argtypes = [_AP, _KP] + [_vp] * 4 + [_sz, _vp]
_lib.gdn_attn_bwd.argtypes = [_AP] + [_vp] * 10 + [_sz, _vp]
_lib.gdn_kv_append.restype = ctypes.c_int
_lib.gdn_kv_append.argtypes = [ctypes.POINTER(GdnKvAppendProblem), _KP] + [_vp] * 6


def _ptr(t, dtype=None, name="tensor"):
    """Device pointer of a contiguous tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor or None")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() if t.numel() > 0 else None


def _host_ptr(t, name):
    """Pointer of a host-side int32 tensor (None -> NULL)."""
    if t is not None and isinstance(t, torch.Tensor) and t.device.type != "cpu":
        raise ValueError(f"{name} must be a CPU tensor")
    return _ptr(t, torch.int32, name)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return stream


def make_problem(N, T, H, HV, cu_seqlens, cu_seqlens_host=None, scale=0.0, K=128, V=128,
                 chunk=64):
    """Build the gdn_problem descriptor. cu_seqlens: int32 device tensor [N+1];
    cu_seqlens_host: optional int32 CPU tensor [N+1] (kept alive by the caller)."""
    p = GdnProblem()
    p.N, p.T, p.H, p.HV, p.K, p.V, p.chunk = N, T, H, HV, K, V, chunk
    p.scale = float(scale)
    p.cu_seqlens = _ptr(cu_seqlens, torch.int32, "cu_seqlens")
    if cu_seqlens_host is not None:
        if cu_seqlens_host.device.type != "cpu":
            raise ValueError("cu_seqlens_host must be a CPU tensor")
        p.cu_seqlens_host = _host_ptr(cu_seqlens_host, "cu_seqlens_host")
    return p


def gdn_status_string(status):
    return _lib.gdn_status_string(int(status)).decode()


def gdn_num_chunks(problem):
    return int(_lib.gdn_num_chunks(ctypes.byref(problem)))


def gdn_chunk_saved_size(problem):
    return int(_lib.gdn_chunk_saved_size(ctypes.byref(problem)))


def gdn_chunk_fwd_workspace_size(problem):
    return int(_lib.gdn_chunk_fwd_workspace_size(ctypes.byref(problem)))


def gdn_chunk_bwd_workspace_size(problem):
    return int(_lib.gdn_chunk_bwd_workspace_size(ctypes.byref(problem)))


def gdn_chunk_bwd_recompute_workspace_size(problem):
    return int(_lib.gdn_chunk_bwd_recompute_workspace_size(ctypes.byref(problem)))


def _check(status, where):
    if status != GDN_OK:
        raise GdnError(status, where)


def _check_saved(problem, saved, where):
    """The C calls take `saved` as a bare pointer; refuse a buffer smaller than
    the layout the library reads and writes for this problem."""
    if saved is None:
        return
    have = saved.numel() * saved.element_size()
    need = gdn_chunk_saved_size(problem)
    if have < need:
        raise ValueError(f"{where}: saved holds {have} bytes, the problem needs {need} "
                         "(gdn_chunk_saved_size)")


def gdn_chunk_fwd(problem, q, k, v, g, beta, h0, o, hT, saved, workspace, stream=None):
    bf, f32 = torch.bfloat16, torch.float32
    _check_saved(problem, saved, "gdn_chunk_fwd")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _lib.gdn_chunk_fwd(
        ctypes.byref(problem), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
        _ptr(g, f32, "g"), _ptr(beta, f32, "beta"), _ptr(h0, f32, "h0"), _ptr(o, bf, "o"),
        _ptr(hT, f32, "hT"), _ptr(saved, None, "saved"), _ptr(workspace, None, "workspace"),
        ws_bytes, _stream(stream))
    _check(st, "gdn_chunk_fwd")


def gdn_chunk_fwd_paged(problem, q, k, v, g, beta, state_pool, slots, ssm_state_indices,
                        has_initial_state, indices_host, o, saved, workspace, stream=None):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    _check_saved(problem, saved, "gdn_chunk_fwd_paged")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _lib.gdn_chunk_fwd_paged(
        ctypes.byref(problem), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
        _ptr(g, f32, "g"), _ptr(beta, f32, "beta"), _ptr(state_pool, f32, "state_pool"),
        int(slots), _ptr(ssm_state_indices, i32, "ssm_state_indices"),
        _ptr(has_initial_state, i32, "has_initial_state"),
        _host_ptr(indices_host, "indices_host"), _ptr(o, bf, "o"), _ptr(saved, None, "saved"),
        _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream))
    _check(st, "gdn_chunk_fwd_paged")


def gdn_chunk_fwd_paged_noalloc_max_bytes():
    return int(_lib.gdn_chunk_fwd_paged_noalloc_max_bytes())


def gdn_chunk_fwd_paged_noalloc(problem, q, k, v, g, beta, state_pool, slots, ssm_state_indices,
                                has_initial_state, indices_host, o, saved, stream=None):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    _check_saved(problem, saved, "gdn_chunk_fwd_paged_noalloc")
    st = _lib.gdn_chunk_fwd_paged_noalloc(
        ctypes.byref(problem), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
        _ptr(g, f32, "g"), _ptr(beta, f32, "beta"), _ptr(state_pool, f32, "state_pool"),
        int(slots), _ptr(ssm_state_indices, i32, "ssm_state_indices"),
        _ptr(has_initial_state, i32, "has_initial_state"),
        _host_ptr(indices_host, "indices_host"), _ptr(o, bf, "o"), _ptr(saved, None, "saved"),
        _stream(stream))
    _check(st, "gdn_chunk_fwd_paged_noalloc")


def gdn_stage_name(op, stage):
    return _lib.gdn_stage_name(int(op), int(stage)).decode()


def gdn_chunk_fwd_timed(problem, q, k, v, g, beta, h0, o, hT, saved, workspace, events,
                        stream=None):
    """gdn_chunk_fwd recording events (a ctypes array of 2*GDN_MAX_STAGES hipEvent_t;
    NULL entries are skipped) around each stage. Returns the number of stages launched."""
    bf, f32 = torch.bfloat16, torch.float32
    _check_saved(problem, saved, "gdn_chunk_fwd_timed")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    n = ctypes.c_int(0)
    st = _lib.gdn_chunk_fwd_timed(
        ctypes.byref(problem), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
        _ptr(g, f32, "g"), _ptr(beta, f32, "beta"), _ptr(h0, f32, "h0"), _ptr(o, bf, "o"),
        _ptr(hT, f32, "hT"), _ptr(saved, None, "saved"), _ptr(workspace, None, "workspace"),
        ws_bytes, _stream(stream), events, ctypes.byref(n))
    _check(st, "gdn_chunk_fwd_timed")
    return n.value


def gdn_chunk_bwd_timed(problem, q, k, v, g, beta, saved, dO, dhT, dq, dk, dv, dg, dbeta, dh0,
                        workspace, events, stream=None):
    bf, f32 = torch.bfloat16, torch.float32
    _check_saved(problem, saved, "gdn_chunk_bwd_timed")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    n = ctypes.c_int(0)
    st = _lib.gdn_chunk_bwd_timed(
        ctypes.byref(problem), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
        _ptr(g, f32, "g"), _ptr(beta, f32, "beta"), _ptr(saved, None, "saved"),
        _ptr(dO, bf, "dO"), _ptr(dhT, f32, "dhT"), _ptr(dq, bf, "dq"), _ptr(dk, bf, "dk"),
        _ptr(dv, bf, "dv"), _ptr(dg, f32, "dg"), _ptr(dbeta, f32, "dbeta"),
        _ptr(dh0, f32, "dh0"), _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream),
        events, ctypes.byref(n))
    _check(st, "gdn_chunk_bwd_timed")
    return n.value


def gdn_chunk_bwd(problem, q, k, v, g, beta, saved, dO, dhT, dq, dk, dv, dg, dbeta, dh0,
                  workspace, stream=None):
    bf, f32 = torch.bfloat16, torch.float32
    _check_saved(problem, saved, "gdn_chunk_bwd")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _lib.gdn_chunk_bwd(
        ctypes.byref(problem), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
        _ptr(g, f32, "g"), _ptr(beta, f32, "beta"), _ptr(saved, None, "saved"),
        _ptr(dO, bf, "dO"), _ptr(dhT, f32, "dhT"), _ptr(dq, bf, "dq"), _ptr(dk, bf, "dk"),
        _ptr(dv, bf, "dv"), _ptr(dg, f32, "dg"), _ptr(dbeta, f32, "dbeta"),
        _ptr(dh0, f32, "dh0"), _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream))
    _check(st, "gdn_chunk_bwd")


def gdn_chunk_bwd_recompute(problem, q, k, v, g, beta, h0, dO, dhT, dq, dk, dv, dg, dbeta, dh0,
                            workspace, stream=None):
    bf, f32 = torch.bfloat16, torch.float32
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _lib.gdn_chunk_bwd_recompute(
        ctypes.byref(problem), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
        _ptr(g, f32, "g"), _ptr(beta, f32, "beta"), _ptr(h0, f32, "h0"),
        _ptr(dO, bf, "dO"), _ptr(dhT, f32, "dhT"), _ptr(dq, bf, "dq"), _ptr(dk, bf, "dk"),
        _ptr(dv, bf, "dv"), _ptr(dg, f32, "dg"), _ptr(dbeta, f32, "dbeta"),
        _ptr(dh0, f32, "dh0"), _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream))
    _check(st, "gdn_chunk_bwd_recompute")


def gdn_chunk_transition(problem, q, k, v, g, beta, M, s, workspace, stream=None):
    bf, f32 = torch.bfloat16, torch.float32
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _lib.gdn_chunk_transition(
        ctypes.byref(problem), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
        _ptr(g, f32, "g"), _ptr(beta, f32, "beta"), _ptr(M, f32, "M"), _ptr(s, f32, "s"),
        _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream))
    _check(st, "gdn_chunk_transition")


def gdn_recurrent_step(N, H, HV, K, V, scale, q, k, v, a, b, A_log, dt_bias, state_pool, slots,
                       ssm_state_indices, indices_host, o, stream=None):
    bf, f32 = torch.bfloat16, torch.float32
    st = _lib.gdn_recurrent_step(
        N, H, HV, K, V, float(scale), _ptr(q, bf, "q"), _ptr(k, bf, "k"), _ptr(v, bf, "v"),
        _ptr(a, bf, "a"), _ptr(b, bf, "b"), _ptr(A_log, f32, "A_log"),
        _ptr(dt_bias, f32, "dt_bias"), _ptr(state_pool, f32, "state_pool"), slots,
        _ptr(ssm_state_indices, torch.int32, "ssm_state_indices"),
        _host_ptr(indices_host, "indices_host"), _ptr(o, bf, "o"), _stream(stream))
    _check(st, "gdn_recurrent_step")


# ---------------------------------------------------------------- allocating helpers
def _for_stream(f):
    """f(..., stream=None) run with a given stream current, so that its outputs and workspace are that
    stream's memory, and its tensors recorded on it (see _on_stream)."""
    place = list(inspect.signature(f).parameters).index("stream")

    @functools.wraps(f)
    def on_given(*args, **kw):
        stream = args[place] if len(args) > place else kw.get("stream")
        if stream is None:
            return f(*args, **kw)
        tensors = [t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor) and t.is_cuda]
        if not tensors:
            return f(*args, **kw)
        return _on_stream(tensors[0].device, stream, lambda _: f(*args, **kw), *tensors)

    return on_given


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


@_for_stream
def chunk_fwd(q, k, v, g, beta, cu_seqlens, h0=None, scale=0.0, cu_seqlens_host=None,
              save_for_backward=False, output_final_state=True, stream=None):
    """Allocate outputs and workspace and run gdn_chunk_fwd.

    q, k [T, H, 128] bf16; v [T, HV, 128] bf16; g, beta [T, HV] fp32 (device);
    cu_seqlens [N+1] int32 (device). Returns (o, hT or None, saved or None).
    """
    T, H, _ = q.shape
    HV = v.shape[1]
    N = cu_seqlens.numel() - 1
    p = make_problem(N, T, H, HV, cu_seqlens, cu_seqlens_host, scale)
    dev = q.device
    o = torch.empty(T, HV, 128, dtype=torch.bfloat16, device=dev)
    hT = torch.empty(N, HV, 128, 128, dtype=torch.float32, device=dev) if output_final_state else None
    saved = _ws(gdn_chunk_saved_size(p), dev) if save_for_backward else None
    ws = _ws(gdn_chunk_fwd_workspace_size(p), dev)
    gdn_chunk_fwd(p, q, k, v, g, beta, h0, o, hT, saved, ws, stream)
    return o, hT, saved


@_for_stream
def chunk_fwd_paged(q, k, v, g, beta, cu_seqlens, state_pool, ssm_state_indices,
                    has_initial_state=None, indices_host=None, scale=0.0, cu_seqlens_host=None,
                    save_for_backward=False, stream=None):
    """Allocate o (and saved, workspace) and run gdn_chunk_fwd_paged; the pool
    [slots, HV, 128, 128] fp32 is updated in place. Returns (o, saved or None)."""
    T, H, _ = q.shape
    HV = v.shape[1]
    N = cu_seqlens.numel() - 1
    p = make_problem(N, T, H, HV, cu_seqlens, cu_seqlens_host, scale)
    dev = q.device
    o = torch.empty(T, HV, 128, dtype=torch.bfloat16, device=dev)
    saved = _ws(gdn_chunk_saved_size(p), dev) if save_for_backward else None
    ws = _ws(gdn_chunk_fwd_workspace_size(p), dev)
    gdn_chunk_fwd_paged(p, q, k, v, g, beta, state_pool, state_pool.shape[0], ssm_state_indices,
                        has_initial_state, indices_host, o, saved, ws, stream)
    return o, saved


@_for_stream
def chunk_bwd(q, k, v, g, beta, cu_seqlens, saved, dO, dhT=None, scale=0.0,
              cu_seqlens_host=None, want_dh0=True, stream=None):
    """Allocate gradients and workspace and run gdn_chunk_bwd.

    Returns dict dq, dk, dv, dg, dbeta, dh0 (dh0 None unless want_dh0).
    """
    T, H, _ = q.shape
    HV = v.shape[1]
    N = cu_seqlens.numel() - 1
    p = make_problem(N, T, H, HV, cu_seqlens, cu_seqlens_host, scale)
    dev = q.device
    out = dict(
        dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
        dg=torch.empty(T, HV, dtype=torch.float32, device=dev),
        dbeta=torch.empty(T, HV, dtype=torch.float32, device=dev),
        dh0=torch.empty(N, HV, 128, 128, dtype=torch.float32, device=dev) if want_dh0 else None,
    )
    ws = _ws(gdn_chunk_bwd_workspace_size(p), dev)
    gdn_chunk_bwd(p, q, k, v, g, beta, saved, dO, dhT, out["dq"], out["dk"], out["dv"],
                  out["dg"], out["dbeta"], out["dh0"], ws, stream)
    return out


@_for_stream
def chunk_bwd_recompute(q, k, v, g, beta, cu_seqlens, dO, h0=None, dhT=None, scale=0.0,
                        cu_seqlens_host=None, want_dh0=True, stream=None):
    """Allocate gradients and workspace and run gdn_chunk_bwd_recompute (no saved
    buffer: the per-chunk states are rebuilt from h0). Returns the dict of chunk_bwd."""
    T, H, _ = q.shape
    HV = v.shape[1]
    N = cu_seqlens.numel() - 1
    p = make_problem(N, T, H, HV, cu_seqlens, cu_seqlens_host, scale)
    dev = q.device
    out = dict(
        dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
        dg=torch.empty(T, HV, dtype=torch.float32, device=dev),
        dbeta=torch.empty(T, HV, dtype=torch.float32, device=dev),
        dh0=torch.empty(N, HV, 128, 128, dtype=torch.float32, device=dev) if want_dh0 else None,
    )
    ws = _ws(gdn_chunk_bwd_recompute_workspace_size(p), dev)
    gdn_chunk_bwd_recompute(p, q, k, v, g, beta, h0, dO, dhT, out["dq"], out["dk"], out["dv"],
                            out["dg"], out["dbeta"], out["dh0"], ws, stream)
    return out


@_for_stream
def chunk_transition(q, k, v, g, beta, cu_seqlens, scale=0.0, cu_seqlens_host=None,
                     stream=None):
    """Allocate M [N, HV, 128, 128] and s [N, HV, 128, 128] (fp32) and run
    gdn_chunk_transition: each sequence's end state is S_0 @ M + s."""
    T, H, _ = q.shape
    HV = v.shape[1]
    N = cu_seqlens.numel() - 1
    p = make_problem(N, T, H, HV, cu_seqlens, cu_seqlens_host, scale)
    dev = q.device
    M = torch.empty(N, HV, 128, 128, dtype=torch.float32, device=dev)
    s = torch.empty(N, HV, 128, 128, dtype=torch.float32, device=dev)
    ws = _ws(gdn_chunk_fwd_workspace_size(p), dev)
    gdn_chunk_transition(p, q, k, v, g, beta, M, s, ws, stream)
    return M, s


@_for_stream
def recurrent_step(q, k, v, a, b, A_log, dt_bias, state_pool, ssm_state_indices,
                   indices_host=None, scale=0.0, stream=None):
    """Allocate o and run gdn_recurrent_step (the pool is updated in place)."""
    N, H, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    o = torch.empty(N, HV, V, dtype=torch.bfloat16, device=q.device)
    gdn_recurrent_step(N, H, HV, K, V, scale, q, k, v, a, b, A_log, dt_bias, state_pool,
                       state_pool.shape[0], ssm_state_indices, indices_host, o, stream)
    return o


# ---------------------------------------------------------------- short convolution
_ACT = {None: 0, "none": 0, "silu": 1}


def make_conv_problem(N, T, C, W, cu_seqlens, cu_seqlens_host=None, activation="silu"):
    """Descriptor of one short-convolution call (cu_seqlens: int32 device [N+1];
    cu_seqlens_host: optional int32 CPU copy, kept alive by the caller)."""
    p = GdnConvProblem()
    p.N, p.T, p.C, p.W = N, T, C, W
    p.activation = _ACT[activation]
    p.cu_seqlens = _ptr(cu_seqlens, torch.int32, "cu_seqlens")
    if cu_seqlens_host is not None:
        p.cu_seqlens_host = _host_ptr(cu_seqlens_host, "cu_seqlens_host")
    return p


def gdn_conv_fwd(problem, x, weight, bias, state_in, y, state_out, stream=None):
    bf = torch.bfloat16
    st = _lib.gdn_conv_fwd(ctypes.byref(problem), _ptr(x, bf, "x"), _ptr(weight, bf, "weight"),
                           _ptr(bias, bf, "bias"), _ptr(state_in, bf, "state_in"),
                           _ptr(y, bf, "y"), _ptr(state_out, bf, "state_out"), _stream(stream))
    _check(st, "gdn_conv_fwd")


def gdn_conv_fwd_paged(problem, x, weight, bias, state_pool, slots, indices, has_initial_state,
                       indices_host, y, stream=None):
    bf, i32 = torch.bfloat16, torch.int32
    st = _lib.gdn_conv_fwd_paged(
        ctypes.byref(problem), _ptr(x, bf, "x"), _ptr(weight, bf, "weight"),
        _ptr(bias, bf, "bias"), _ptr(state_pool, bf, "state_pool"), int(slots),
        _ptr(indices, i32, "indices"), _ptr(has_initial_state, i32, "has_initial_state"),
        _host_ptr(indices_host, "indices_host"), _ptr(y, bf, "y"), _stream(stream))
    _check(st, "gdn_conv_fwd_paged")


def gdn_conv_bwd_workspace_size(problem):
    return int(_lib.gdn_conv_bwd_workspace_size(ctypes.byref(problem)))


def gdn_conv_bwd(problem, x, weight, bias, state_in, dy, dx, dweight, dbias, dstate_in,
                 workspace, stream=None):
    bf, f32 = torch.bfloat16, torch.float32
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _lib.gdn_conv_bwd(
        ctypes.byref(problem), _ptr(x, bf, "x"), _ptr(weight, bf, "weight"),
        _ptr(bias, bf, "bias"), _ptr(state_in, bf, "state_in"), _ptr(dy, bf, "dy"),
        _ptr(dx, bf, "dx"), _ptr(dweight, f32, "dweight"), _ptr(dbias, f32, "dbias"),
        _ptr(dstate_in, f32, "dstate_in"), _ptr(workspace, None, "workspace"), ws_bytes,
        _stream(stream))
    _check(st, "gdn_conv_bwd")


def gdn_conv_update(N, C, W, activation, x, weight, bias, state_pool, slots, indices,
                    indices_host, y, stream=None):
    bf, i32 = torch.bfloat16, torch.int32
    st = _lib.gdn_conv_update(
        int(N), int(C), int(W), _ACT[activation], _ptr(x, bf, "x"), _ptr(weight, bf, "weight"),
        _ptr(bias, bf, "bias"), _ptr(state_pool, bf, "state_pool"), int(slots),
        _ptr(indices, i32, "indices"), _host_ptr(indices_host, "indices_host"), _ptr(y, bf, "y"),
        _stream(stream))
    _check(st, "gdn_conv_update")


@_for_stream
def conv_fwd(x, weight, bias, cu_seqlens, state_in=None, activation="silu",
             cu_seqlens_host=None, want_state=True, stream=None):
    """x [T, C] bf16, weight [C, W] bf16, bias [C] bf16 or None (device).
    Returns (y [T, C] bf16, end states [N, C, W-1] bf16 or None)."""
    T, C = x.shape
    W = weight.shape[1]
    N = cu_seqlens.numel() - 1
    p = make_conv_problem(N, T, C, W, cu_seqlens, cu_seqlens_host, activation)
    y = torch.empty_like(x)
    so = torch.empty(N, C, W - 1, dtype=torch.bfloat16, device=x.device) if want_state else None
    gdn_conv_fwd(p, x, weight, bias, state_in, y, so, stream)
    return y, so


@_for_stream
def conv_fwd_paged(x, weight, bias, cu_seqlens, state_pool, indices, has_initial_state=None,
                   indices_host=None, activation="silu", cu_seqlens_host=None, stream=None):
    """Paged forward: state_pool [slots, C, W-1] bf16 is read and updated in place."""
    T, C = x.shape
    W = weight.shape[1]
    N = cu_seqlens.numel() - 1
    p = make_conv_problem(N, T, C, W, cu_seqlens, cu_seqlens_host, activation)
    y = torch.empty_like(x)
    gdn_conv_fwd_paged(p, x, weight, bias, state_pool, state_pool.shape[0], indices,
                       has_initial_state, indices_host, y, stream)
    return y


@_for_stream
def conv_bwd(x, weight, bias, cu_seqlens, dy, state_in=None, activation="silu",
             cu_seqlens_host=None, want_dstate=True, stream=None):
    """Returns dict dx [T, C] bf16, dweight [C, W] fp32, dbias [C] fp32 (None
    without a bias), dstate [N, C, W-1] fp32 (None unless want_dstate)."""
    T, C = x.shape
    W = weight.shape[1]
    N = cu_seqlens.numel() - 1
    dev = x.device
    p = make_conv_problem(N, T, C, W, cu_seqlens, cu_seqlens_host, activation)
    out = dict(dx=torch.empty_like(x),
               dweight=torch.empty(C, W, dtype=torch.float32, device=dev),
               dbias=torch.empty(C, dtype=torch.float32, device=dev) if bias is not None else None,
               dstate=torch.empty(N, C, W - 1, dtype=torch.float32, device=dev)
               if want_dstate else None)
    ws = _ws(gdn_conv_bwd_workspace_size(p), dev)
    gdn_conv_bwd(p, x, weight, bias, state_in, dy, out["dx"], out["dweight"], out["dbias"],
                 out["dstate"], ws, stream)
    return out


@_for_stream
def conv_update(x, weight, bias, state_pool, indices, indices_host=None, activation="silu",
                stream=None):
    """One decode token per row; state_pool [slots, C, W-1] bf16 updated in place."""
    N, C = x.shape
    W = weight.shape[1]
    y = torch.empty_like(x)
    gdn_conv_update(N, C, W, activation, x, weight, bias, state_pool, state_pool.shape[0],
                    indices, indices_host, y, stream)
    return y


# ---------------------------------------------------------------- device tensors of a call
# The operators below check every tensor's device, type and shape before its
# pointer is handed on, run on the tensors' device whichever is current, and
# allocate on the stream that they run on.
def _dev(t, shape, dtype, name, dev):
    """Device pointer of a contiguous tensor of this shape on this device (None -> NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, dtype, name, dev):
    """Device pointer and token stride (0: dense) of a [tokens, heads, columns] tensor whose heads
    are dense rows: a tensor of its own or a slice of a wider buffer's rows."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), 0
    n, h, d = t.shape
    sn, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1) or (sn < h * d and n > 1):
        raise ValueError(f"{name} must have dense heads and tokens apart, got strides {t.stride()}")
    return t.data_ptr(), sn if n > 1 and sn != h * d else 0


def _on_device(t, name):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a tensor on the GPU")
    return t.device


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on_stream(dev, stream, call, *tensors):
    """call(stream handle) with the tensors' device current, on `stream` (a torch stream or a raw
    handle, of a stream that outlives the tensors), which is then current too, or by default on the
    device's current stream. The call's tensors are recorded on a given stream: the memory of one
    that is freed before the stream is through is not handed out until then. Waiting for what
    other streams write into them is the caller's."""
    if stream is None:
        if dev.index == torch.cuda.current_device():
            return call(_raw_stream(dev.index))
        with torch.cuda.device(dev):
            return call(_raw_stream(dev.index))
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.stream(stream):
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(stream)
        return call(stream.cuda_stream)


# ---------------------------------------------------------------- linear attention
_bf16, _f32 = torch.bfloat16, torch.float32


def make_linear_problem(N, T, H, HV, D, cu_seqlens=None, cu_seqlens_host=None, scale=0.0,
                        q_stride=0, k_stride=0, v_stride=0):
    """Build the gdn_linear_problem descriptor (K = V = D). cu_seqlens: int32 device tensor [N+1];
    cu_seqlens_host: optional int32 CPU tensor [N+1] (both kept alive by the caller)."""
    cu = host = None
    if cu_seqlens is not None:
        cu = _dev(cu_seqlens, (N + 1,), torch.int32, "cu_seqlens",
                  _on_device(cu_seqlens, "cu_seqlens"))
    if cu_seqlens_host is not None:
        if cu_seqlens_host.numel() != N + 1:
            raise ValueError(f"cu_seqlens_host must hold {N + 1} boundaries")
        host = _host_ptr(cu_seqlens_host, "cu_seqlens_host")
    return GdnLinearProblem(N, T, H, HV, D, D, scale, cu, host, q_stride, k_stride, v_stride)


def gdn_linear_saved_size(problem):
    return int(_lib.gdn_linear_saved_size(ctypes.byref(problem)))


def gdn_linear_fwd_workspace_size(problem):
    return int(_lib.gdn_linear_fwd_workspace_size(ctypes.byref(problem)))


def gdn_linear_bwd_workspace_size(problem):
    return int(_lib.gdn_linear_bwd_workspace_size(ctypes.byref(problem)))


def _linear_shapes(q, k, v):
    T, H, D = q.shape
    if k.shape != q.shape or v.dim() != 3 or v.shape[0] != T or v.shape[2] != D:
        raise ValueError(f"q, k, v must be [T, H, D], [T, H, D], [T, HV, D], got {tuple(q.shape)}, "
                         f"{tuple(k.shape)}, {tuple(v.shape)}")
    return T, H, v.shape[1], D


def _linear_call(q, k, v, log_decay, cu_seqlens, cu_seqlens_host, scale):
    """(device, problem, pointers of q, k, v, log_decay) of one call."""
    dev = _on_device(q, "q")
    T, H, HV, D = _linear_shapes(q, k, v)
    (qp, qs), (kp, ks), (vp, vs) = (_rows(q, _bf16, "q", dev), _rows(k, _bf16, "k", dev),
                                    _rows(v, _bf16, "v", dev))
    N = cu_seqlens.numel() - 1 if cu_seqlens is not None else T
    if cu_seqlens is not None and cu_seqlens.device != dev:
        raise ValueError(f"cu_seqlens must be on {dev}, got {cu_seqlens.device}")
    p = make_linear_problem(N, T, H, HV, D, cu_seqlens, cu_seqlens_host, scale, qs, ks, vs)
    return dev, p, (qp, kp, vp, _dev(log_decay, (HV,), _f32, "log_decay", dev))


def _bytes(t):
    return t.numel() * t.element_size() if t is not None else 0


def _buffer(t, name, dev):
    if t is None:
        return None
    if t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {dev}")
    return t.data_ptr()


def _at(t):
    return t.data_ptr() if t is not None else None


def _alloc_bytes(n, dev):
    return torch.empty(n, dtype=torch.uint8, device=dev) if n else None


def linear_fwd(q, k, v, log_decay, cu_seqlens, h0=None, scale=0.0, cu_seqlens_host=None,
               save_for_backward=False, output_final_state=True, stream=None):
    """Linear attention with a decay for each head over a pack (gdn_linear_fwd).

    q, k [T, H, D], v [T, HV, D] bf16, D = 64 or 128, dense or slices of a wider buffer's rows;
    log_decay [HV] fp32; cu_seqlens [N+1] int32; h0 [N, HV, D, D] fp32 or None.
    Returns (o [T, HV, D] bf16, hT [N, HV, D, D] fp32 or None, saved or None)."""
    dev, p, ptrs = _linear_call(q, k, v, log_decay, cu_seqlens, cu_seqlens_host, scale)
    N, T, HV, D = p.N, p.T, p.HV, p.K
    h0p = _dev(h0, (N, HV, D, D), _f32, "h0", dev)

    def call(s):
        o = torch.empty(T, HV, D, dtype=_bf16, device=dev)
        hT = torch.empty(N, HV, D, D, dtype=_f32, device=dev) if output_final_state else None
        saved = _alloc_bytes(gdn_linear_saved_size(p), dev) if save_for_backward else None
        ws = None if save_for_backward else _alloc_bytes(gdn_linear_fwd_workspace_size(p), dev)
        _check(_lib.gdn_linear_fwd(ctypes.byref(p), *ptrs, h0p, o.data_ptr(), _at(hT), _at(saved),
                                   _at(ws), _bytes(ws), s), "gdn_linear_fwd")
        return o, hT, saved

    return _on_stream(dev, stream, call, q, k, v, log_decay, cu_seqlens, h0)


def linear_fwd_paged(q, k, v, log_decay, cu_seqlens, state_pool, ssm_state_indices,
                     has_initial_state=None, indices_host=None, scale=0.0, cu_seqlens_host=None,
                     save_for_backward=False, stream=None):
    """linear_fwd whose sequences' states are blocks of state_pool [slots, HV, D, D] fp32, updated
    in place (gdn_linear_fwd_paged). Returns (o, saved or None)."""
    dev, p, ptrs = _linear_call(q, k, v, log_decay, cu_seqlens, cu_seqlens_host, scale)
    N, T, HV, D = p.N, p.T, p.HV, p.K
    slots = state_pool.shape[0]
    if indices_host is not None and indices_host.numel() != N:
        raise ValueError(f"indices_host must hold {N} indices")
    more = (_dev(state_pool, (slots, HV, D, D), _f32, "state_pool", dev), slots,
            _dev(ssm_state_indices, (N,), torch.int32, "ssm_state_indices", dev),
            _dev(has_initial_state, (N,), torch.int32, "has_initial_state", dev),
            _host_ptr(indices_host, "indices_host"))

    def call(s):
        o = torch.empty(T, HV, D, dtype=_bf16, device=dev)
        saved = _alloc_bytes(gdn_linear_saved_size(p), dev) if save_for_backward else None
        ws = None if save_for_backward else _alloc_bytes(gdn_linear_fwd_workspace_size(p), dev)
        _check(_lib.gdn_linear_fwd_paged(ctypes.byref(p), *ptrs, *more, o.data_ptr(), _at(saved),
                                         _at(ws), _bytes(ws), s), "gdn_linear_fwd_paged")
        return o, saved

    return _on_stream(dev, stream, call, q, k, v, log_decay, cu_seqlens, state_pool, ssm_state_indices,
                      has_initial_state)


def linear_bwd(q, k, v, log_decay, cu_seqlens, saved, dO, dhT=None, scale=0.0,
               cu_seqlens_host=None, want_dh0=True, stream=None):
    """Gradients of linear_fwd (gdn_linear_bwd): dict dq, dk [T, H, D], dv [T, HV, D] bf16 and
    dh0 [N, HV, D, D] fp32 (None unless want_dh0)."""
    dev, p, ptrs = _linear_call(q, k, v, log_decay, cu_seqlens, cu_seqlens_host, scale)
    N, T, H, HV, D = p.N, p.T, p.H, p.HV, p.K
    if _bytes(saved) < gdn_linear_saved_size(p):
        raise ValueError(f"saved holds {_bytes(saved)} bytes, the problem needs "
                         f"{gdn_linear_saved_size(p)} (gdn_linear_saved_size)")
    more = (_buffer(saved, "saved", dev), _dev(dO, (T, HV, D), _bf16, "dO", dev),
            _dev(dhT, (N, HV, D, D), _f32, "dhT", dev))

    def call(s):
        dq, dk = (torch.empty(T, H, D, dtype=_bf16, device=dev) for _ in range(2))
        dv = torch.empty(T, HV, D, dtype=_bf16, device=dev)
        dh0 = torch.empty(N, HV, D, D, dtype=_f32, device=dev) if want_dh0 else None
        ws = _alloc_bytes(gdn_linear_bwd_workspace_size(p), dev)
        _check(_lib.gdn_linear_bwd(ctypes.byref(p), *ptrs, *more, dq.data_ptr(), dk.data_ptr(),
                                   dv.data_ptr(), _at(dh0), _at(ws), _bytes(ws), s),
               "gdn_linear_bwd")
        return dict(dq=dq, dk=dk, dv=dv, dh0=dh0)

    return _on_stream(dev, stream, call, q, k, v, log_decay, cu_seqlens, saved, dO, dhT)


def linear_step(q, k, v, log_decay, state_pool, ssm_state_indices, indices_host=None, scale=0.0,
                stream=None):
    """One token per row (gdn_linear_step): q, k [N, H, D], v [N, HV, D]; state_pool
    [slots, HV, D, D] fp32 is updated in place. Returns o [N, HV, D] bf16."""
    dev, p, ptrs = _linear_call(q, k, v, log_decay, None, None, scale)
    N, HV, D = p.N, p.HV, p.K
    slots = state_pool.shape[0]
    if indices_host is not None and indices_host.numel() != N:
        raise ValueError(f"indices_host must hold {N} indices")
    more = (_dev(state_pool, (slots, HV, D, D), _f32, "state_pool", dev), slots,
            _dev(ssm_state_indices, (N,), torch.int32, "ssm_state_indices", dev),
            _host_ptr(indices_host, "indices_host"))

    def call(s):
        o = torch.empty(N, HV, D, dtype=_bf16, device=dev)
        _check(_lib.gdn_linear_step(ctypes.byref(p), *ptrs, *more, o.data_ptr(), s),
               "gdn_linear_step")
        return o

    return _on_stream(dev, stream, call, q, k, v, log_decay, state_pool, ssm_state_indices)


# ---------------------------------------------------------------- rotary positions and the norm
_ELEM = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ROPE = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}


def _elem(t, name):
    if t.dtype not in _ELEM:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return _ELEM[t.dtype]


def rotary_inv_freq(R, base=10000.0, scaling=None, factor=1.0, original=4096, device=None):
    """(inv_freq [R / 2] fp32, attention factor) of R turning columns (gdn_rotary_inv_freq).
    scaling: None, "linear", "ntk" or "yarn", for contexts `factor` times as long as `original`."""
    f, m = torch.empty(max(R // 2, 1), dtype=torch.float32), ctypes.c_float(1.0)
    _check(_lib.gdn_rotary_inv_freq(R, base, _ROPE[scaling], factor, original, f.data_ptr(),
                                    ctypes.byref(m)), "gdn_rotary_inv_freq")
    return f.to(device) if device is not None else f, m.value


def _rotary(call, q, k, inv_freq, positions, cu_seqlens, offsets, cu_seqlens_host, interleaved,
            mscale, q_out, k_out, stream, back):
    dev = _on_device(q, "q")
    T, HQ, D = q.shape
    HK = 0
    if k is not None:
        if k.shape[0] != T or k.shape[2] != D:
            raise ValueError(f"k must be [{T}, HK, {D}], got {tuple(k.shape)}")
        HK = k.shape[1]
    pos = cu = host = off = None
    N = 0
    if positions is not None:
        pos = _dev(positions, (T,), torch.int32, "positions", dev)
    elif cu_seqlens is None:
        raise ValueError("positions or cu_seqlens are needed")
    else:
        N = cu_seqlens.numel() - 1
        cu = _dev(cu_seqlens, (N + 1,), torch.int32, "cu_seqlens", dev)
        off = _dev(offsets, (N,), torch.int32, "offsets", dev)
        if cu_seqlens_host is not None:
            if cu_seqlens_host.numel() != N + 1:
                raise ValueError(f"cu_seqlens_host must hold {N + 1} boundaries")
            host = _host_ptr(cu_seqlens_host, "cu_seqlens_host")
    p = GdnRotaryProblem(T, HQ, HK, D, 2 * inv_freq.numel(), bool(interleaved), _elem(q, "q"),
                         mscale, pos, N, cu, host, off)
    freq = _dev(inv_freq, (inv_freq.numel(),), _f32, "inv_freq", dev)
    qp, qs = _rows(q, q.dtype, "q", dev)
    kp, ks = _rows(k, q.dtype, "k", dev) if k is not None else (None, 0)

    def result(t, heads, name):
        """(tensor, pointer, token stride) of one output: t, or a new one without it."""
        if t is None:
            t = torch.empty(T, heads, D, dtype=q.dtype, device=dev)
            return t, t.data_ptr(), 0
        if t.shape != (T, heads, D):
            raise ValueError(f"{name} must have the shape {(T, heads, D)}, got {tuple(t.shape)}")
        return (t, *_rows(t, q.dtype, name, dev))

    def launch(s):
        qr, qo, qos = result(q_out, HQ, "dq" if back else "q_out")
        kr, ko, kos = result(k_out, HK, "dk" if back else "k_out") if k is not None else (None, None, 0)
        if back:
            p.q_out_stride, p.k_out_stride, p.q_stride, p.k_stride = qs, ks, qos, kos
        else:
            p.q_stride, p.k_stride, p.q_out_stride, p.k_out_stride = qs, ks, qos, kos
        _check(call(ctypes.byref(p), freq, qp, kp, qo, ko, s), "gdn_rotary_bwd" if back else "gdn_rotary")
        return qr, kr

    return _on_stream(dev, stream, launch, q, k, inv_freq, positions, cu_seqlens, offsets, q_out, k_out)


def rotary(q, k, inv_freq, positions=None, cu_seqlens=None, offsets=None, cu_seqlens_host=None,
           interleaved=False, mscale=1.0, q_out=None, k_out=None, stream=None):
    """Rotary positions (gdn_rotary) of q [T, HQ, D] and k [T, HK, D] (or None), bf16, fp16 or fp32,
    dense or slices of a wider buffer's rows; inv_freq [R / 2] fp32. Positions [T] int32, or each
    token's place in its sequence by cu_seqlens [N+1] plus offsets [N]. q_out, k_out: where the
    results go (q and k themselves: in place), by default new tensors. Returns (q_out, k_out)."""
    return _rotary(_lib.gdn_rotary, q, k, inv_freq, positions, cu_seqlens, offsets,
                   cu_seqlens_host, interleaved, mscale, q_out, k_out, stream, False)


def rotary_bwd(dq_out, dk_out, inv_freq, positions=None, cu_seqlens=None, offsets=None,
               cu_seqlens_host=None, interleaved=False, mscale=1.0, dq=None, dk=None, stream=None):
    """Gradients of rotary (gdn_rotary_bwd): (dq, dk) from those of its outputs."""
    return _rotary(_lib.gdn_rotary_bwd, dq_out, dk_out, inv_freq, positions, cu_seqlens,
                   offsets, cu_seqlens_host, interleaved, mscale, dq, dk, stream, True)


def _norm_rows(t, dtype, shape, name, dev):
    """Pointer and row stride (0: dense) of a [rows, D] tensor whose rows are dense."""
    if t is None:
        return None, 0
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), 0
    rows, D = shape
    sr, sd = t.stride()
    if (sd != 1 and D > 1) or (sr < D and rows > 1):
        raise ValueError(f"{name} must have dense rows apart, got strides {t.stride()}")
    return t.data_ptr(), sr if rows > 1 and sr != D else 0


def _norm_problem(x, weight, unit_offset, eps, group, dev):
    rows, D = x.shape
    p = GdnRmsnormProblem(rows, D, _elem(x, "x"), bool(unit_offset), group, eps, 0, 0)
    return p, _dev(weight, (D,), x.dtype, "weight", dev)


def rmsnorm_fwd(x, weight=None, residual=None, eps=1e-6, unit_offset=False, quant=None,
                want_y=None, want_rstd=False, residual_out=None, stream=None):
    """Root-mean-square norm (gdn_rmsnorm_fwd) of x [rows, D] (+ residual), bf16, fp16 or fp32, rows
    dense or slices of wider ones. quant: None, "row" or 128 for an e4m3 output with a scale for each
    row or each 128 columns. want_y: the output in x's type (by default where there is no e4m3 one).
    Returns a dict of residual_out (with a residual), y, y8, scales, rstd (those asked for)."""
    dev = _on_device(x, "x")
    if quant not in (None, "row", 128):
        raise ValueError(f'quant must be None, "row" or 128, got {quant!r}')
    rows, D = x.shape
    p, wp = _norm_problem(x, weight, unit_offset, eps, 128 if quant == 128 else 0, dev)
    xp, p.x_stride = _norm_rows(x, x.dtype, (rows, D), "x", dev)
    rp, p.residual_stride = _norm_rows(residual, x.dtype, (rows, D), "residual", dev)
    if want_y is False and quant is None:
        raise ValueError("nothing to compute: want_y is False and quant is None")

    def call(s):
        out = {}
        so = y = y8 = scales = r = None
        if residual is not None:
            t = torch.empty(rows, D, dtype=x.dtype, device=dev) if residual_out is None else residual_out
            out["residual_out"], so = t, _dev(t, (rows, D), x.dtype, "residual_out", dev)
        if want_y or quant is None:
            t = out["y"] = torch.empty(rows, D, dtype=x.dtype, device=dev)
            y = t.data_ptr()
        if quant is not None:
            t = out["y8"] = torch.empty(rows, D, dtype=torch.float8_e4m3fn, device=dev)
            y8 = t.data_ptr()
            shape = (rows,) if quant == "row" else (rows, (D + 127) // 128)
            t = out["scales"] = torch.empty(*shape, dtype=_f32, device=dev)
            scales = t.data_ptr()
        if want_rstd:
            t = out["rstd"] = torch.empty(rows, dtype=_f32, device=dev)
            r = t.data_ptr()
        _check(_lib.gdn_rmsnorm_fwd(ctypes.byref(p), xp, rp, wp, so, y, y8, scales, r, s),
               "gdn_rmsnorm_fwd")
        return out

    return _on_stream(dev, stream, call, x, weight, residual, residual_out)


def gdn_rmsnorm_bwd_workspace_size(problem):
    return int(_lib.gdn_rmsnorm_bwd_workspace_size(ctypes.byref(problem)))


def rmsnorm_bwd(dy, s, weight, rstd, dresidual_out=None, unit_offset=False, want_dweight=None,
                stream=None):
    """Gradients of rmsnorm_fwd (gdn_rmsnorm_bwd): s is its residual_out (x without a residual).
    Returns dict dx [rows, D] (of x and of residual) and dweight [D] fp32 (None without a weight)."""
    dev = _on_device(dy, "dy")
    rows, D = dy.shape
    p, wp = _norm_problem(dy, weight, unit_offset, 0.0, 0, dev)
    sp, p.x_stride = _norm_rows(s, dy.dtype, (rows, D), "s", dev)
    dyp = _dev(dy, (rows, D), dy.dtype, "dy", dev)
    dsp = _dev(dresidual_out, (rows, D), dy.dtype, "dresidual_out", dev)
    rp = _dev(rstd, (rows,), _f32, "rstd", dev)
    want_dweight = weight is not None if want_dweight is None else want_dweight

    def call(stream_):
        dx = torch.empty(rows, D, dtype=dy.dtype, device=dev)
        dw = torch.empty(D, dtype=_f32, device=dev) if want_dweight else None
        ws = _alloc_bytes(gdn_rmsnorm_bwd_workspace_size(p), dev) if want_dweight else None
        _check(_lib.gdn_rmsnorm_bwd(ctypes.byref(p), sp, wp, rp, dyp, dsp, dx.data_ptr(), _at(dw),
                                    _at(ws), _bytes(ws), stream_), "gdn_rmsnorm_bwd")
        return dict(dx=dx, dweight=dw)

    return _on_stream(dev, stream, call, dy, s, weight, rstd, dresidual_out)


# ---------------------------------------------------------------- softmax attention and its cache
_HALF = {torch.bfloat16: 0, torch.float16: 1}


def _half(t, name):
    if t.dtype not in _HALF:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return _HALF[t.dtype]


def _bad_cache(k_cache, v_cache, page_table, N, HK, D, dtype, dev):
    """Why these are no cache and table of a call, as an exception."""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dtype is not dtype:
            return TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.device != dev:
            return ValueError(f"{name} must be on {dev}, got {t.device}")
        if t.dim() != 4 or t.shape[2] != HK or t.shape[3] != D or t.shape != k_cache.shape:
            return ValueError(f"{name} must be [pages, page_size, {HK}, {D}], got {tuple(t.shape)}")
    if page_table.dtype is not torch.int32 or page_table.device != dev:
        return ValueError(f"page_table must be int32 on {dev}")
    if page_table.dim() != 2 or page_table.shape[0] != N:
        return ValueError(f"page_table must be [{N}, columns], got {tuple(page_table.shape)}")
    if page_table.stride(1) != 1 or page_table.stride(0) < page_table.shape[1]:
        return ValueError(f"page_table must have dense rows apart, got strides {page_table.stride()}")
    return ValueError(f"k_cache and v_cache must have the same strides and dense columns, got "
                      f"{k_cache.stride()} and {v_cache.stride()}")


def _cache_heads(k_cache):
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache must be [pages, page_size, HK, D], got {tuple(k_cache.shape)}")
    return k_cache.shape[2]


def _unlike(a, b, shape):
    """Whether strides differ where there is more than one element."""
    return a != b and any(x != y for x, y, n in zip(a, b, shape) if n > 1)


def _cache(k_cache, v_cache, page_table, offsets, N, HK, D, dtype, dev):
    """The gdn_kv_cache of tensors [pages, page_size, HK, D] in any order of memory."""
    shape, strides, table = k_cache.shape, k_cache.stride(), page_table.stride()
    if (k_cache.dtype is not dtype or v_cache.dtype is not dtype or k_cache.device != dev
            or v_cache.device != dev or v_cache.shape != shape or len(shape) != 4 or shape[2] != HK
            or shape[3] != D or _unlike(v_cache.stride(), strides, shape) or (strides[3] != 1 and D > 1)
            or page_table.dtype is not torch.int32 or page_table.device != dev or len(table) != 2):
        raise _bad_cache(k_cache, v_cache, page_table, N, HK, D, dtype, dev)
    rows, columns = page_table.shape
    if rows != N or (table[1] != 1 and columns > 1) or (table[0] < columns and N > 1):
        raise _bad_cache(k_cache, v_cache, page_table, N, HK, D, dtype, dev)
    pages, size = shape[0], shape[1]
    page, token, head = strides[:3]
    # an extent of 1 has no stride of its own
    return GdnKvCache(k_cache.data_ptr(), v_cache.data_ptr(), pages, size, columns,
                      table[0] if N > 1 else 0, page if pages > 1 else D, token if size > 1 else D,
                      head if HK > 1 else D,
                      page_table.data_ptr(), _dev(offsets, (N,), torch.int32, "offsets", dev))


def _bounds(cu_seqlens, cu_seqlens_host, dev):
    """(N, device pointer, host pointer) of a pack's boundaries."""
    N = cu_seqlens.numel() - 1
    if cu_seqlens_host is not None and cu_seqlens_host.numel() != N + 1:
        raise ValueError(f"cu_seqlens_host must hold {N + 1} boundaries")
    return (N, _dev(cu_seqlens, (N + 1,), torch.int32, "cu_seqlens", dev),
            _host_ptr(cu_seqlens_host, "cu_seqlens_host"))


def _attn_rows(q, k, v, dev):
    """(HK, pointers, strides) of q [T, HQ, D] and k, v [T, HK, D]."""
    T, _, D = q.shape
    for t, name in ((k, "k"), (v, "v")):
        if t.dim() != 3 or t.shape[0] != T or t.shape[2] != D or t.shape != k.shape:
            raise ValueError(f"{name} must be [{T}, HK, {D}], got {tuple(t.shape)}")
    rows = [_rows(t, q.dtype, n, dev) for t, n in ((q, "q"), (k, "k"), (v, "v"))]
    return k.shape[1], [r[0] for r in rows], [r[1] for r in rows]


def kv_append(k, v, k_cache, v_cache, page_table, offsets, cu_seqlens=None, q=None, inv_freq=None,
              interleaved=False, mscale=1.0, cu_seqlens_host=None, q_out=None, stream=None):
    """New tokens' k, v [T, HK, D] into a paged cache (gdn_kv_append), k turned by rotary positions on
    the way and q [T, HQ, D] beside it; bf16 or fp16, dense or slices of a wider buffer's rows.

    k_cache, v_cache [pages, page_size, HK, D], in any order of memory, are updated in place; page_table
    [N, columns] and offsets [N] (tokens that each sequence had before) int32. cu_seqlens [N+1] int32, or
    None for one token of each sequence. inv_freq [R / 2] fp32, or None: nothing turns. q_out: where q's
    result goes (q itself: in place), by default a new tensor. Returns q_out, or None without q."""
    dev, kind = _on_device(k, "k"), _half(k, "k")
    dtype, shape = k.dtype, k.shape
    T, HK, D = shape
    if v.shape != shape:
        raise ValueError(f"v must be {tuple(shape)}, got {tuple(v.shape)}")
    HQ = 0
    if q is not None:
        wide = q.shape
        if len(wide) != 3 or wide[0] != T or wide[2] != D:
            raise ValueError(f"q must be [{T}, HQ, {D}], got {tuple(wide)}")
        HQ = wide[1]
    N, cu, host = T, None, None
    if cu_seqlens is not None:
        N, cu, host = _bounds(cu_seqlens, cu_seqlens_host, dev)
    kp, ks = _rows(k, dtype, "k", dev)
    vp, vs = _rows(v, dtype, "v", dev)
    qp, qs = _rows(q, dtype, "q", dev) if HQ else (None, 0)
    R = 2 * inv_freq.numel() if inv_freq is not None else 0
    p = GdnKvAppendProblem(N, T, HQ, HK, D, R, bool(interleaved), kind, mscale, cu, host, qs, ks, vs, 0)
    freq = _dev(inv_freq, (R // 2,), _f32, "inv_freq", dev)
    cache = _cache(k_cache, v_cache, page_table, offsets, N, HK, D, dtype, dev)

    def call(s):
        out, op = q_out, None
        if HQ and out is None:
            out = torch.empty(wide, dtype=dtype, device=dev)
            op = out.data_ptr()
        elif HQ:
            if out.shape != wide:
                raise ValueError(f"q_out must have the shape {tuple(wide)}, got {tuple(out.shape)}")
            op, p.q_out_stride = _rows(out, dtype, "q_out", dev)
        _check(_lib.gdn_kv_append(ctypes.byref(p), ctypes.byref(cache), freq, qp, kp, vp, op, s),
               "gdn_kv_append")
        return out if HQ else None

    return _on_stream(dev, stream, call, q, k, v, inv_freq, cu_seqlens, k_cache, v_cache, page_table,
                      offsets, q_out)


def _attn_call(name, p, cache, q, want_lse, ptrs):
    """call(stream) of one forward: allocates o, lse and the workspace."""
    size, run, dev = getattr(_lib, name + "_workspace_size"), getattr(_lib, name), q.device
    args = [ctypes.byref(p)] + ([ctypes.byref(cache)] if cache is not None else [])

    def call(s):
        o = torch.empty(q.shape, dtype=q.dtype, device=dev)
        lse = torch.empty(q.shape[:2], dtype=_f32, device=dev) if want_lse else None
        n = size(*args)
        ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        _check(run(*args, *ptrs, o.data_ptr(), _at(lse), _at(ws), n, s), name)
        return o, lse

    return call


def attn_fwd(q, k, v, cu_seqlens, window=0, sinks=0, scale=0.0, cu_seqlens_host=None, want_lse=False,
             stream=None):
    """Causal softmax attention over a pack (gdn_attn_fwd).

    q [T, HQ, D], k, v [T, HK, D], bf16 or fp16, D = 64, 128 or 256, dense or slices of a wider buffer's
    rows; cu_seqlens [N+1] int32. window: the last positions that a token sees (0: all), sinks: the
    first positions that it sees besides. Returns (o [T, HQ, D], lse [T, HQ] fp32 or None)."""
    dev = _on_device(q, "q")
    T, HQ, D = q.shape
    HK, ptrs, strides = _attn_rows(q, k, v, dev)
    N, cu, host = _bounds(cu_seqlens, cu_seqlens_host, dev)
    p = GdnAttnProblem(N, T, HQ, HK, D, _half(q, "q"), window, sinks, scale, cu, host, *strides)
    return _on_stream(dev, stream, _attn_call("gdn_attn_fwd", p, None, q, want_lse, ptrs), q, k, v,
                      cu_seqlens)


def attn_bwd(q, k, v, cu_seqlens, o, lse, dO, window=0, sinks=0, scale=0.0, cu_seqlens_host=None,
             stream=None):
    """Gradients of attn_fwd (gdn_attn_bwd), o and lse as it gave them: dict dq [T, HQ, D] and
    dk, dv [T, HK, D]."""
    dev = _on_device(q, "q")
    T, HQ, D = q.shape
    HK, ptrs, strides = _attn_rows(q, k, v, dev)
    N, cu, host = _bounds(cu_seqlens, cu_seqlens_host, dev)
    p = GdnAttnProblem(N, T, HQ, HK, D, _half(q, "q"), window, sinks, scale, cu, host, *strides)
    more = (_dev(o, (T, HQ, D), q.dtype, "o", dev), _dev(lse, (T, HQ), _f32, "lse", dev),
            _dev(dO, (T, HQ, D), q.dtype, "dO", dev))

    def call(s):
        dq = torch.empty(T, HQ, D, dtype=q.dtype, device=dev)
        dk, dv = (torch.empty(T, HK, D, dtype=q.dtype, device=dev) for _ in range(2))
        ws = _alloc_bytes(_lib.gdn_attn_bwd_workspace_size(ctypes.byref(p)), dev)
        _check(_lib.gdn_attn_bwd(ctypes.byref(p), *ptrs, *more, dq.data_ptr(), dk.data_ptr(),
                                 dv.data_ptr(), _at(ws), _bytes(ws), s), "gdn_attn_bwd")
        return dict(dq=dq, dk=dk, dv=dv)

    return _on_stream(dev, stream, call, q, k, v, cu_seqlens, o, lse, dO)


def attn_fwd_paged(q, k_cache, v_cache, page_table, cu_seqlens, offsets, window=0, sinks=0, scale=0.0,
                   cu_seqlens_host=None, want_lse=False, stream=None):
    """attn_fwd over a paged cache that holds the tokens' keys and values already (gdn_attn_fwd_paged):
    token i of sequence n is at position offsets[n] + i. The cache as in kv_append."""
    dev = _on_device(q, "q")
    T, HQ, D = q.shape
    qp, qs = _rows(q, q.dtype, "q", dev)
    N, cu, host = _bounds(cu_seqlens, cu_seqlens_host, dev)
    HK = _cache_heads(k_cache)
    p = GdnAttnProblem(N, T, HQ, HK, D, _half(q, "q"), window, sinks, scale, cu, host, qs, 0, 0)
    cache = _cache(k_cache, v_cache, page_table, offsets, N, HK, D, q.dtype, dev)
    return _on_stream(dev, stream, _attn_call("gdn_attn_fwd_paged", p, cache, q, want_lse, (qp,)), q,
                      k_cache, v_cache, page_table, cu_seqlens, offsets)


def attn_step(q, k_cache, v_cache, page_table, offsets, window=0, sinks=0, scale=0.0, want_lse=False,
              stream=None):
    """Attention of one new token a row over a paged cache that holds it already (gdn_attn_step): q
    [N, HQ, D], the token of row n at position offsets[n] (negative: an idle row, o = 0). The cache as
    in kv_append. Returns (o [N, HQ, D], lse [N, HQ] fp32 or None)."""
    dev = _on_device(q, "q")
    N, HQ, D = q.shape
    qp, qs = _rows(q, q.dtype, "q", dev)
    HK = _cache_heads(k_cache)
    p = GdnAttnProblem(N, N, HQ, HK, D, _half(q, "q"), window, sinks, scale, None, None, qs, 0, 0)
    cache = _cache(k_cache, v_cache, page_table, offsets, N, HK, D, q.dtype, dev)
    return _on_stream(dev, stream, _attn_call("gdn_attn_step", p, cache, q, want_lse, (qp,)), q, k_cache,
                      v_cache, page_table, offsets)
