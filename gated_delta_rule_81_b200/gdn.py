"""Thin ctypes binding of libgdn.so (the C ABI in include/gdn.h).

Argument marshalling only: every step of the mixer runs in the library's CUDA
kernels.  torch supplies device memory and the current stream.  There is no
fallback: if the library is missing or a call is rejected, an exception is
raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

HEAD_DIM = 128
CHUNK = 64

_STATUS = {
    0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED", 3: "GDN_ERR_MISALIGNED",
    4: "GDN_ERR_ALIAS", 5: "GDN_ERR_CUDA", 6: "GDN_ERR_DEVICE_TIMEOUT", 7: "GDN_ERR_WORKSPACE",
}


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)}")


class GdnInputs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("z", ctypes.c_void_p),
        ("stride_q", ctypes.c_longlong), ("stride_k", ctypes.c_longlong), ("stride_v", ctypes.c_longlong),
        ("stride_z", ctypes.c_longlong), ("stride_a", ctypes.c_longlong), ("stride_b", ctypes.c_longlong),
        ("conv_w", ctypes.c_void_p), ("A_log", ctypes.c_void_p), ("norm_w", ctypes.c_void_p),
        ("H_k", ctypes.c_int), ("H_v", ctypes.c_int), ("scale", ctypes.c_float),
        ("events", ctypes.c_void_p),
        ("schedule", ctypes.c_int),
    ]
    tokens = devices = None  # of the tensors, where make_inputs has filled it


class GdnLayer(ctypes.Structure):
    """gdn_layer: the weights of one delta-rule layer (device pointers)."""
    _fields_ = [
        ("w_in", ctypes.c_void_p), ("ld_w_in", ctypes.c_longlong),
        ("w_out", ctypes.c_void_p), ("ld_w_out", ctypes.c_longlong),
        ("conv_w", ctypes.c_void_p), ("A_log", ctypes.c_void_p), ("norm_w", ctypes.c_void_p),
        ("H_k", ctypes.c_int), ("H_v", ctypes.c_int), ("hidden", ctypes.c_int),
        ("scale", ctypes.c_float), ("schedule", ctypes.c_int),
        ("events", ctypes.c_void_p),
    ]
    devices = None  # of the tensors, where make_layer has filled it


class GdnAttnLayer(ctypes.Structure):
    """gdn_attn_layer: the weights of one global-attention layer (device pointers)."""
    _fields_ = [
        ("w_in", ctypes.c_void_p), ("ld_w_in", ctypes.c_longlong),
        ("w_out", ctypes.c_void_p), ("ld_w_out", ctypes.c_longlong),
        ("q_norm_w", ctypes.c_void_p), ("k_norm_w", ctypes.c_void_p),
        ("hidden", ctypes.c_int),
        ("events", ctypes.c_void_p),
    ]
    devices = None  # of the tensors, where make_attn_layer has filled it


ROPE_MAX_HEAD_DIM = 256
MAX_TREE_NODES = 64
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class GdnRope(ctypes.Structure):
    """gdn_rope: the table of one rotary embedding (filled by gdn_rope_init, then only read)."""
    _fields_ = [
        ("head_dim", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int),
        ("eps", ctypes.c_float), ("amplitude", ctypes.c_float),
        ("turns", ctypes.c_ulonglong * (ROPE_MAX_HEAD_DIM // 2)),
    ]


ATTN_Q_HEADS, ATTN_KV_HEADS, ATTN_HEAD_DIM = 24, 4, 256
ATTN_N_IN = 2 * 24 * 256 + 2 * 4 * 256


SCHEDULE_AUTO = 0          # one overlapped launch when it pays (few scan units, many prep items)
SCHEDULE_TWO_LAUNCHES = 1  # prep kernel, then scan kernel
SCHEDULE_FUSED = 2         # one overlapped launch whenever the scan units fit in half the SMs


_lib = None
_vp, _sz, _i, _ll = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_longlong
_f, _d = ctypes.c_float, ctypes.c_double

EXPORTS = ("gdn_prefill_workspace_size", "gdn_prefill", "gdn_prefill_varlen", "gdn_prefill_host_workspace_size",
           "gdn_prefill_host", "gdn_decode_step",
           "gdn_decode_multi", "gdn_gemm_bf16", "gdn_layer_n_in", "gdn_layer_workspace_size", "gdn_layer_prefill",
           "gdn_layer_decode_workspace_size", "gdn_layer_decode",
           "gdn_attn_layer_workspace_size", "gdn_attn_layer_prefill", "gdn_attention_prefill",
           "gdn_attn_decode_workspace_size", "gdn_attn_layer_decode_step", "gdn_status_string",
           "gdn_err_status", "gdn_prefill_fused_plan",
           "gdn_decode_tree", "gdn_decode_tree_commit", "gdn_layer_tree_workspace_size", "gdn_layer_decode_tree",
           "gdn_layer_tree_commit", "gdn_rope_init", "gdn_qk_norm_rope", "gdn_attention_tree_workspace_size",
           "gdn_attention_tree", "gdn_attn_tree_commit", "gdn_attn_layer_tree_workspace_size",
           "gdn_attn_layer_decode_tree", "gdn_attn_layer_tree_commit")
MAX_DECODE_TOKENS = 8


def load(path: str | None = None, fresh: bool = False):
    """Load libgdn.so from the package directory (it must have been built).  The first library
    loaded is kept for every later call; `fresh` loads `path` (e.g. libgdn_debug.so) and
    returns it without making it that library."""
    global _lib
    if _lib is not None and not fresh:
        return _lib
    path = path or _build.lib_path("libgdn.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: run gated_delta_rule_81_b200.build.build() first")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(GdnInputs)
    lib.gdn_prefill_workspace_size.argtypes = [_i, _i, _i, _ll]
    lib.gdn_prefill_workspace_size.restype = _sz
    lib.gdn_prefill.argtypes = [P, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]
    lib.gdn_prefill.restype = _i
    lib.gdn_prefill_host_workspace_size.argtypes = [_i, _i, _i, _i]
    lib.gdn_prefill_host_workspace_size.restype = _sz
    lib.gdn_prefill_host.argtypes = [P, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]
    lib.gdn_prefill_host.restype = _i
    lib.gdn_prefill_varlen.argtypes = [P, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]
    lib.gdn_prefill_varlen.restype = _i
    lib.gdn_decode_step.argtypes = [P, _i, _vp, _vp, _vp, _vp, _vp]
    lib.gdn_decode_step.restype = _i
    lib.gdn_decode_multi.argtypes = [P, _i, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp]
    lib.gdn_decode_multi.restype = _i
    lib.gdn_gemm_bf16.argtypes = [_vp, _ll, _vp, _ll, _vp, _ll, _i, _i, _i, _vp, _vp]
    lib.gdn_gemm_bf16.restype = _i
    lib.gdn_layer_n_in.argtypes = [_i, _i]
    lib.gdn_layer_n_in.restype = _ll
    lib.gdn_layer_workspace_size.argtypes = [_i, _i, _i, _i]
    lib.gdn_layer_workspace_size.restype = _sz
    lib.gdn_layer_prefill.argtypes = [ctypes.POINTER(GdnLayer), _i, _i, _vp, _ll, _vp, _vp, _vp, _vp, _vp, _ll, _vp,
                                      _sz, _vp, _vp]
    lib.gdn_layer_prefill.restype = _i
    lib.gdn_layer_decode_workspace_size.argtypes = [_i, _i, _i, _i]
    lib.gdn_layer_decode_workspace_size.restype = _sz
    lib.gdn_layer_decode.argtypes = [ctypes.POINTER(GdnLayer), _i, _i, _vp, _ll, _vp, _vp, _vp, _i, _vp, _ll, _vp, _sz,
                                     _vp, _vp]
    lib.gdn_layer_decode.restype = _i
    lib.gdn_attn_layer_workspace_size.argtypes = [_i, _i]
    lib.gdn_attn_layer_workspace_size.restype = _sz
    lib.gdn_attn_layer_prefill.argtypes = [ctypes.POINTER(GdnAttnLayer), _i, _i, _vp, _ll, _vp, _vp, _i, _vp, _ll,
                                           _vp, _sz, _vp, _vp]
    lib.gdn_attn_decode_workspace_size.argtypes = [_i, _i]
    lib.gdn_attn_decode_workspace_size.restype = _sz
    lib.gdn_attn_layer_decode_step.argtypes = [ctypes.POINTER(GdnAttnLayer), _i, _vp, _ll, _vp, _vp, _i, _vp, _vp,
                                               _ll, _vp, _sz, _vp, _vp]
    lib.gdn_attn_layer_decode_step.restype = _i
    lib.gdn_attn_layer_prefill.restype = _i
    lib.gdn_attention_prefill.argtypes = [_vp, _vp, _vp, _vp, _ll, _i, _i, _vp, _vp, _vp]
    lib.gdn_attention_prefill.restype = _i
    lib.gdn_status_string.argtypes = [_i]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_err_status.argtypes = [_i]
    lib.gdn_err_status.restype = _i
    lib.gdn_prefill_fused_plan.argtypes = [_i, _i, _i, _ll, _i, _i]
    lib.gdn_prefill_fused_plan.restype = _i
    lib.gdn_decode_tree.argtypes = [P, _i, _i, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp]
    lib.gdn_decode_tree_commit.argtypes = [P, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp]
    lib.gdn_layer_tree_workspace_size.argtypes = [_i, _i, _i, _i]
    lib.gdn_layer_decode_tree.argtypes = [ctypes.POINTER(GdnLayer), _i, _i, _vp, _vp, _ll, _vp, _vp, _vp, _i, _vp, _ll,
                                          _vp, _sz, _vp, _vp]
    lib.gdn_layer_tree_commit.argtypes = [ctypes.POINTER(GdnLayer), _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp,
                                          _vp]
    lib.gdn_rope_init.argtypes = [ctypes.POINTER(GdnRope), _i, _i, _i, _i, _d, _d, _i, _d, _d, _f]
    lib.gdn_qk_norm_rope.argtypes = [ctypes.POINTER(GdnRope), _ll, _i, _i, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _vp,
                                     _vp, _ll, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp]
    lib.gdn_attention_tree_workspace_size.argtypes = [_i, _i, _i, _i, _i]
    lib.gdn_attention_tree.argtypes = [_vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _i, _vp, _vp, _vp, _ll, _i, _i, _i, _f, _i,
                                       _i, _vp, _vp, _sz, _vp, _vp]
    lib.gdn_attn_tree_commit.argtypes = [_vp, _ll, _vp, _ll, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp]
    lib.gdn_attn_layer_tree_workspace_size.argtypes = [_i, _i]
    lib.gdn_attn_layer_decode_tree.argtypes = [ctypes.POINTER(GdnAttnLayer), _i, _i, _vp, _vp, _ll, _vp, _vp, _i, _vp,
                                               _vp, _ll, _vp, _sz, _vp, _vp]
    lib.gdn_attn_layer_tree_commit.argtypes = [_i, _i, _vp, _vp, _vp, _vp, _i, _vp, _vp, _sz, _vp, _vp]
    for name in ("gdn_decode_tree", "gdn_decode_tree_commit", "gdn_layer_decode_tree", "gdn_layer_tree_commit",
                 "gdn_rope_init", "gdn_qk_norm_rope", "gdn_attention_tree", "gdn_attn_tree_commit",
                 "gdn_attn_layer_decode_tree", "gdn_attn_layer_tree_commit"):
        getattr(lib, name).restype = _i
    for name in ("gdn_layer_tree_workspace_size", "gdn_attention_tree_workspace_size",
                 "gdn_attn_layer_tree_workspace_size"):
        getattr(lib, name).restype = _sz
    if not fresh:
        _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _tok_stride(t, T_tot):
    """Token stride (elements) of a [T_tot, ...] tensor whose per-token channels are contiguous."""
    if t.dim() == 1:
        return t.numel() // max(T_tot, 1)
    inner = t[0] if t.shape[0] > 0 else t
    if t.shape[0] > 0 and not inner.is_contiguous():
        raise ValueError("per-token channels must be contiguous")
    return t.stride(0)


def make_inputs(q, k, v, a, b, z, conv_w, A_log, norm_w, scale=1.0, schedule=SCHEDULE_AUTO) -> GdnInputs:
    T_tot = q.shape[0]
    H_k = q.shape[1] if q.dim() == 3 else q.shape[-1] // HEAD_DIM
    H_v = v.shape[1] if v.dim() == 3 else v.shape[-1] // HEAD_DIM
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b), ("z", z), ("conv_w", conv_w),
                    ("norm_w", norm_w)):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bf16")
    if A_log.dtype != torch.float32:
        raise TypeError("A_log must be fp32")
    s = GdnInputs()
    s.q, s.k, s.v, s.a, s.b, s.z = (t.data_ptr() for t in (q, k, v, a, b, z))
    s.stride_q, s.stride_k, s.stride_v = (_tok_stride(t, T_tot) for t in (q, k, v))
    s.stride_z, s.stride_a, s.stride_b = (_tok_stride(t, T_tot) for t in (z, a, b))
    s.conv_w, s.A_log, s.norm_w = conv_w.data_ptr(), A_log.data_ptr(), norm_w.data_ptr()
    s.H_k, s.H_v, s.scale = int(H_k), int(H_v), float(scale)
    s.schedule = int(schedule)
    s.tokens = min(t.shape[0] for t in (q, k, v, a, b, z))
    s.devices = {t.device for t in (q, k, v, a, b, z, conv_w, A_log, norm_w)}
    return s


def set_timing_events(inp: GdnInputs, events):
    """Attach torch.cuda.Event objects (enable_timing=True) that the library records
    around its kernels (3 for prefill, 2 for decode); None detaches.  Returns the
    ctypes array, which must stay alive while the call is in use."""
    if events is None:
        inp.events = None
        return None
    for ev in events:
        if not ev.cuda_event:
            ev.record()  # materialise the handle
    arr = (ctypes.c_void_p * len(events))(*[ev.cuda_event for ev in events])
    inp.events = ctypes.cast(arr, ctypes.c_void_p)
    return arr


def _check(status, where):
    if status != 0:
        raise GdnError(status, where)


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def workspace_size(H_k: int, H_v: int, N: int, n_chunks: int) -> int:
    return int(load().gdn_prefill_workspace_size(H_k, H_v, N, n_chunks))


def chunk_count(lengths) -> int:
    return sum((int(L) + CHUNK - 1) // CHUNK for L in lengths)


def _outputs(dev, T_tot, H_k, H_v, N, want_state, want_conv, out, state_out, conv_out):
    C_conv = (2 * H_k + H_v) * HEAD_DIM
    if out is None:
        out = torch.empty(T_tot, H_v, HEAD_DIM, dtype=torch.bfloat16, device=dev)
    if state_out is None and want_state:
        state_out = torch.empty(N, H_v, HEAD_DIM, HEAD_DIM, dtype=torch.float32, device=dev)
    if conv_out is None and want_conv:
        conv_out = torch.empty(N, 3, C_conv, dtype=torch.bfloat16, device=dev)
    return out, state_out, conv_out


def prefill(inp: GdnInputs, B: int, T: int, state_in=None, conv_in=None, *, want_state=True, want_conv=True,
            out=None, state_out=None, conv_out=None, workspace=None, err=None, device=None):
    """gdn_prefill: B sequences of T tokens, packed [B*T].  Returns (out, state_out, conv_out)."""
    lib = load()
    dev = device or torch.device("cuda", torch.cuda.current_device())
    out, state_out, conv_out = _outputs(dev, B * T, inp.H_k, inp.H_v, B, want_state, want_conv, out, state_out,
                                        conv_out)
    n_chunks = B * ((T + CHUNK - 1) // CHUNK)
    need = lib.gdn_prefill_workspace_size(inp.H_k, inp.H_v, B, n_chunks)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(lib.gdn_prefill(ctypes.byref(inp), B, T, _ptr(state_in), _ptr(state_out), _ptr(conv_in),
                           _ptr(conv_out), _ptr(out), _ptr(workspace), workspace.numel(), _ptr(err), _stream()),
           "gdn_prefill")
    return out, state_out, conv_out


def prefill_host_workspace_size(H_k: int, H_v: int, B: int, T: int) -> int:
    return int(load().gdn_prefill_host_workspace_size(H_k, H_v, B, T))


def prefill_host(inp: GdnInputs, B: int, T: int, out, state_in=None, state_out=None, conv_in=None, conv_out=None, *,
                 workspace=None, err=None, stream=None):
    """gdn_prefill_host: `inp` built from pinned host tensors (q, k, v, a, b, z) and device
    weights; out, state_in / state_out, conv_in / conv_out are pinned host tensors (or None).
    Asynchronous on `stream` (a torch.cuda.Stream, default the current one); returns out."""
    lib = load()
    if workspace is None:
        workspace = torch.empty(prefill_host_workspace_size(inp.H_k, inp.H_v, B, T), dtype=torch.uint8,
                                device=torch.device("cuda", torch.cuda.current_device()))
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream()
    _check(lib.gdn_prefill_host(ctypes.byref(inp), B, T, _ptr(state_in), _ptr(state_out), _ptr(conv_in),
                                _ptr(conv_out), _ptr(out), _ptr(workspace), workspace.numel(), _ptr(err), st),
           "gdn_prefill_host")
    return out


def prefill_varlen(inp: GdnInputs, cu_seqlens, cu_seqlens_host, state_in=None, conv_in=None, *, want_state=True,
                   want_conv=True, out=None, state_out=None, conv_out=None, workspace=None, err=None):
    """gdn_prefill_varlen.  cu_seqlens: device int32 [N+1]; cu_seqlens_host: CPU int32 [N+1]."""
    lib = load()
    dev = cu_seqlens.device
    host = cu_seqlens_host.to(torch.int32).contiguous()
    N = host.numel() - 1
    T_tot = int(host[-1])
    out, state_out, conv_out = _outputs(dev, T_tot, inp.H_k, inp.H_v, N, want_state, want_conv, out, state_out,
                                        conv_out)
    n_chunks = chunk_count((host[1:] - host[:-1]).tolist())
    need = lib.gdn_prefill_workspace_size(inp.H_k, inp.H_v, N, n_chunks)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    host_ptr = ctypes.cast(host.data_ptr(), ctypes.c_void_p)
    _check(lib.gdn_prefill_varlen(ctypes.byref(inp), N, _ptr(cu_seqlens), host_ptr, _ptr(state_in),
                                  _ptr(state_out), _ptr(conv_in), _ptr(conv_out), _ptr(out), _ptr(workspace),
                                  workspace.numel(), _ptr(err), _stream()),
           "gdn_prefill_varlen")
    return out, state_out, conv_out


def decode_step(inp: GdnInputs, N: int, state, conv_state, out=None, err=None):
    """gdn_decode_step: one token per sequence; state and conv_state updated in place.  Returns out."""
    lib = load()
    if out is None:
        out = torch.empty(N, inp.H_v, HEAD_DIM, dtype=torch.bfloat16, device=state.device)
    _check(lib.gdn_decode_step(ctypes.byref(inp), N, _ptr(state), _ptr(conv_state), _ptr(out), _ptr(err),
                               _stream()),
           "gdn_decode_step")
    return out


def decode_multi(inp: GdnInputs, N: int, T: int, state, conv_state, state_slot=None, out=None, err=None):
    """gdn_decode_multi: T new tokens per sequence (token n*T + t), states in pool slots.

    state [n_slots][H_v][128][128] fp32 and conv_state [n_slots][3][C_conv] bf16 are
    updated in place; state_slot is a device int32 [N] (None: sequence n uses slot n).
    Returns out [N*T][H_v][128] bf16."""
    lib = load()
    if out is None:
        out = torch.empty(N * T, inp.H_v, HEAD_DIM, dtype=torch.bfloat16, device=state.device)
    n_slots = state.shape[0]
    _check(lib.gdn_decode_multi(ctypes.byref(inp), N, T, _ptr(state), _ptr(conv_state), _ptr(state_slot), n_slots,
                                _ptr(out), _ptr(err), _stream()),
           "gdn_decode_multi")
    return out


def gemm_bf16(a, b, out=None, err=None):
    """gdn_gemm_bf16: out[M][N] = a[M][K] @ b[N][K]^T (bf16, fp32 accumulation).  a and b may be
    row-strided views (last dimension contiguous)."""
    lib = load()
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("a and b disagree on K")
    for name, t in (("a", a), ("b", b)):
        if t.dtype != torch.bfloat16 or t.stride(1) != 1:
            raise TypeError(f"{name} must be bf16 with a contiguous last dimension")
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=a.device)
    _check(lib.gdn_gemm_bf16(_ptr(a), a.stride(0), _ptr(b), b.stride(0), _ptr(out), out.stride(0), M, N, K,
                             _ptr(err), _stream()), "gdn_gemm_bf16")
    return out


def make_layer(w_in, w_out, conv_w, A_log, norm_w, H_k, H_v, scale=1.0, schedule=SCHEDULE_AUTO) -> GdnLayer:
    """gdn_layer from device tensors: w_in bf16 [n_in][hidden], w_out bf16 [hidden][H_v*128]."""
    for name, t in (("w_in", w_in), ("w_out", w_out), ("conv_w", conv_w), ("norm_w", norm_w)):
        if t.dtype != torch.bfloat16 or t.stride(-1) != 1:
            raise TypeError(f"{name} must be bf16 with a contiguous last dimension")
    L = GdnLayer()
    L.w_in, L.ld_w_in = w_in.data_ptr(), w_in.stride(0)
    L.w_out, L.ld_w_out = w_out.data_ptr(), w_out.stride(0)
    L.conv_w, L.A_log, L.norm_w = conv_w.data_ptr(), A_log.data_ptr(), norm_w.data_ptr()
    L.H_k, L.H_v, L.hidden = int(H_k), int(H_v), int(w_in.shape[1])
    L.scale, L.schedule = float(scale), int(schedule)
    L.devices = {t.device for t in (w_in, w_out, conv_w, A_log, norm_w)}
    return L


def layer_workspace_size(H_k, H_v, B, T) -> int:
    return int(load().gdn_layer_workspace_size(H_k, H_v, B, T))


def layer_prefill(L: GdnLayer, B: int, T: int, x, state_in=None, conv_in=None, *, want_state=True, want_conv=True,
                  y=None, state_out=None, conv_out=None, workspace=None, err=None):
    """gdn_layer_prefill: y = out_proj(mixer(in_proj(x))) for B sequences of T tokens.
    Returns (y, state_out, conv_out)."""
    lib = load()
    dev = x.device
    _, state_out, conv_out = _outputs(dev, 0, L.H_k, L.H_v, B, want_state, want_conv, torch.empty(0), state_out,
                                      conv_out)
    if y is None:
        y = torch.empty(B * T, L.hidden, dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = torch.empty(layer_workspace_size(L.H_k, L.H_v, B, T), dtype=torch.uint8, device=dev)
    _check(lib.gdn_layer_prefill(ctypes.byref(L), B, T, _ptr(x), x.stride(0), _ptr(state_in), _ptr(state_out),
                                 _ptr(conv_in), _ptr(conv_out), _ptr(y), y.stride(0), _ptr(workspace),
                                 workspace.numel(), _ptr(err), _stream()), "gdn_layer_prefill")
    return y, state_out, conv_out


def layer_decode(L: GdnLayer, N: int, T: int, x, state, conv_state, state_slot=None, n_slots=None, *, y=None,
                 workspace=None, err=None):
    """gdn_layer_decode: T new tokens for each of N sequences (x [N*T][hidden]); state and
    conv_state (the pool, or one slot per sequence) are updated in place.  Returns y."""
    lib = load()
    if y is None:
        y = torch.empty(N * T, L.hidden, dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(int(lib.gdn_layer_decode_workspace_size(L.H_k, L.H_v, N, T)), dtype=torch.uint8,
                                device=x.device)
    if n_slots is None:
        n_slots = state.shape[0]
    _check(lib.gdn_layer_decode(ctypes.byref(L), N, T, _ptr(x), x.stride(0), _ptr(state), _ptr(conv_state),
                                _ptr(state_slot), int(n_slots), _ptr(y), y.stride(0), _ptr(workspace),
                                workspace.numel(), _ptr(err), _stream()), "gdn_layer_decode")
    return y


def make_attn_layer(w_in, w_out, q_norm_w, k_norm_w) -> GdnAttnLayer:
    """gdn_attn_layer from device tensors: w_in bf16 [ATTN_N_IN][hidden], w_out bf16 [hidden][24*256]."""
    for name, t in (("w_in", w_in), ("w_out", w_out), ("q_norm_w", q_norm_w), ("k_norm_w", k_norm_w)):
        if t.dtype != torch.bfloat16 or t.stride(-1) != 1:
            raise TypeError(f"{name} must be bf16 with a contiguous last dimension")
    L = GdnAttnLayer()
    L.w_in, L.ld_w_in = w_in.data_ptr(), w_in.stride(0)
    L.w_out, L.ld_w_out = w_out.data_ptr(), w_out.stride(0)
    L.q_norm_w, L.k_norm_w = q_norm_w.data_ptr(), k_norm_w.data_ptr()
    L.hidden = int(w_in.shape[1])
    L.devices = {t.device for t in (w_in, w_out, q_norm_w, k_norm_w)}
    return L


def attn_layer_prefill(L: GdnAttnLayer, B: int, T: int, x, *, y=None, k_cache=None, v_cache=None, cache_cap=0,
                       workspace=None, err=None):
    """gdn_attn_layer_prefill.  Caches are [B][cache_cap or T][4][256].  Returns (y, k_cache, v_cache)."""
    lib = load()
    dev = x.device
    cap = cache_cap or T
    if y is None:
        y = torch.empty(B * T, L.hidden, dtype=torch.bfloat16, device=dev)
    if k_cache is None:
        k_cache = torch.empty(B, cap, ATTN_KV_HEADS, ATTN_HEAD_DIM, dtype=torch.bfloat16, device=dev)
    if v_cache is None:
        v_cache = torch.empty(B, cap, ATTN_KV_HEADS, ATTN_HEAD_DIM, dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = torch.empty(int(lib.gdn_attn_layer_workspace_size(B, T)), dtype=torch.uint8, device=dev)
    _check(lib.gdn_attn_layer_prefill(ctypes.byref(L), B, T, _ptr(x), x.stride(0), _ptr(k_cache), _ptr(v_cache),
                                      int(cache_cap), _ptr(y), y.stride(0), _ptr(workspace), workspace.numel(),
                                      _ptr(err), _stream()), "gdn_attn_layer_prefill")
    return y, k_cache, v_cache


def attn_layer_decode_step(L: GdnAttnLayer, x, k_cache, v_cache, cache_len, *, y=None, workspace=None, err=None):
    """gdn_attn_layer_decode_step: one new token per sequence (x [N][hidden]); the caches
    [N][cap][4][256] and cache_len (device int32 [N]) are updated in place.  Returns y."""
    lib = load()
    N, cap = x.shape[0], k_cache.shape[1]
    if y is None:
        y = torch.empty(N, L.hidden, dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(int(lib.gdn_attn_decode_workspace_size(N, cap)), dtype=torch.uint8, device=x.device)
    _check(lib.gdn_attn_layer_decode_step(ctypes.byref(L), N, _ptr(x), x.stride(0), _ptr(k_cache), _ptr(v_cache),
                                          cap, _ptr(cache_len), _ptr(y), y.stride(0), _ptr(workspace),
                                          workspace.numel(), _ptr(err), _stream()), "gdn_attn_layer_decode_step")
    return y


def attention_prefill(q_hat, k, v, g, B: int, T: int, out=None, err=None):
    """gdn_attention_prefill on device tensors q_hat [B*T,24,256], k, v [B*T,4,256], g (rows of >= 24*256)."""
    lib = load()
    if out is None:
        out = torch.empty(B * T, ATTN_Q_HEADS * ATTN_HEAD_DIM, dtype=torch.bfloat16, device=q_hat.device)
    g2 = g.reshape(g.shape[0], -1) if g.dim() == 3 else g
    _check(lib.gdn_attention_prefill(_ptr(q_hat), _ptr(k), _ptr(v), _ptr(g2), g2.stride(0), B, T, _ptr(out),
                                     _ptr(err), _stream()), "gdn_attention_prefill")
    return out


# ------------------------------------------------------------------ trees of drafted tokens

# These bindings run once per layer and step on small tensors, where the host's time is the call's: pointers go
# over as plain integers, shapes and strides are read once, and the device is switched only when it has to be.

def _addr(t):
    return None if t is None else t.data_ptr()


def _run_on(device, name, *args):
    """Call entry point `name` on `device` and its current stream (which comes last)."""
    fn = getattr(_lib or load(), name)
    index = device.index
    if index == torch.cuda.current_device():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != 0:
        raise GdnError(status, name)


def _want(name, t, dtype, shape=None, device=None):
    """A contiguous tensor of this type (and shape) on this device, or None."""
    if t is None:
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _want_made(made, device, tokens=0):
    """The tensors of an input descriptor or a layer, as far as it knows them."""
    if made.devices is not None and made.devices != {device}:
        raise ValueError(f"the {type(made).__name__}'s tensors are on {sorted(map(str, made.devices))}, not on {device}")
    if tokens > 0 and made.tokens is not None and made.tokens < tokens:
        raise ValueError(f"the inputs hold {made.tokens} tokens, not {tokens}")


def _want_err(err, device):
    if err is not None and (err.dtype is not torch.int32 or err.numel() < 1 or err.device != device):
        raise ValueError(f"err must be an int32 on {device}, not {err.dtype} on {err.device}")


def _workspace_bytes(workspace, device):
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, not on {device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.numel() * workspace.element_size()


def _matrix(name, t, rows, cols, device):
    """Row stride of a bf16 matrix of at least rows x cols, of which those are used."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bf16, not {t.dtype}")
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] < cols or (cols > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [{rows}][{cols}] with rows side by side, not {tuple(t.shape)} by {t.stride()}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t.stride(0) if rows > 1 else cols


def _rows(name, t, tokens, heads, dim, device):
    """Token stride of a bf16 [tokens][heads][dim] tensor whose tokens' heads lie side by side."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bf16, not {t.dtype}")
    if shape != (tokens, heads, dim):
        raise ValueError(f"{name} must be {(tokens, heads, dim)}, not {tuple(shape)}")
    if stride[2] != 1 or (heads > 1 and stride[1] != dim):
        raise ValueError(f"{name} must have its heads side by side, not strides {stride}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if tokens <= 1 and (stride[0] < heads * dim or stride[0] % 8):  # a single row's stride may be anything
        return heads * dim
    return stride[0]


def _want_pool(H_k, H_v, state, conv_state):
    slots, dev = state.shape[0], state.device
    _want("state", state, torch.float32, (slots, H_v, HEAD_DIM, HEAD_DIM))
    _want("conv_state", conv_state, torch.bfloat16, (slots, 3, (2 * H_k + H_v) * HEAD_DIM), dev)
    return slots, dev


def decode_tree(inp: GdnInputs, N: int, T: int, parent, state, conv_state, state_slot=None, out=None, err=None):
    """gdn_decode_tree: the outputs of T tree nodes per sequence (node n*T + t), each after its own path.

    parent: device int32 [N][T] (-1 a child of the last committed token, an earlier node, or -2 for no
    node), None for a chain.  state and conv_state (the pools) are read.  Returns out [N*T][H_v][128] bf16."""
    slots, dev = _want_pool(inp.H_k, inp.H_v, state, conv_state)
    _want_made(inp, dev, N * T)
    _want("parent", parent, torch.int32, (N, T), dev)
    _want("state_slot", state_slot, torch.int32, (N,), dev)
    if out is None:
        out = torch.empty((N * T, inp.H_v, HEAD_DIM), dtype=torch.bfloat16, device=dev)
    else:
        _want("out", out, torch.bfloat16, (N * T, inp.H_v, HEAD_DIM), dev)
    _want_err(err, dev)
    _run_on(dev, "gdn_decode_tree", inp, N, T, _addr(parent), _addr(state), _addr(conv_state),
            _addr(state_slot), slots, _addr(out), _addr(err))
    return out


def decode_tree_commit(inp: GdnInputs, N: int, T: int, parent, accepted, state, conv_state, state_slot=None, *,
                       state_out=None, conv_out=None, err=None):
    """gdn_decode_tree_commit: state and conv_state advanced along each sequence's path to node accepted[n]
    (device int32 [N], -1: none), in place unless state_out / conv_out are given.  `inp`'s q, k, v, a and b hold what
    they held at decode_tree (the last raw rows become the conv state).  Returns both."""
    slots, dev = _want_pool(inp.H_k, inp.H_v, state, conv_state)
    _want_made(inp, dev, N * T)
    if state_out is None:
        state_out = state
    else:
        _want("state_out", state_out, torch.float32, state.shape, dev)
    if conv_out is None:
        conv_out = conv_state
    else:
        _want("conv_out", conv_out, torch.bfloat16, conv_state.shape, dev)
    _want("parent", parent, torch.int32, (N, T), dev)
    _want("accepted", accepted, torch.int32, (N,), dev)
    _want("state_slot", state_slot, torch.int32, (N,), dev)
    _want_err(err, dev)
    _run_on(dev, "gdn_decode_tree_commit", inp, N, T, _addr(parent), _addr(accepted), _addr(state),
            _addr(state_out), _addr(conv_state), _addr(conv_out), _addr(state_slot), slots, _addr(err))
    return state_out, conv_out


def make_rope(head_dim: int, rotary_dim: int | None = None, *, base: float = 1e7, interleaved: bool = False,
              scaling: str = "none", factor: float = 1.0, original_len: int = 0, beta_fast: float = 32.0,
              beta_slow: float = 1.0, eps: float = 1e-6) -> GdnRope:
    """gdn_rope_init: the table of a rotary embedding on the first rotary_dim dims of each head (default all),
    scaling "none", "linear", "ntk" or "yarn"; eps is the norms'.  Made once and kept; `amplitude`, the factor on
    cosine and sine, may be set on the result."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, not {scaling!r}")
    rope = GdnRope()
    _check(load().gdn_rope_init(ctypes.byref(rope), head_dim, head_dim if rotary_dim is None else rotary_dim,
                                ROPE_INTERLEAVED if interleaved else ROPE_HALF, ROPE_SCALINGS[scaling], base, factor,
                                original_len, beta_fast, beta_slow, eps), "gdn_rope_init")
    return rope


def qk_norm_rope(rope: GdnRope, q, k=None, v=None, *, q_norm_w=None, k_norm_w=None, positions=None, rows=None,
                 q_out=None, k_out=None, v_out=None, err=None):
    """gdn_qk_norm_rope on q [tokens][H_q][D] and k, v [tokens][H_kv][D] (token-strided views are fine; q or k
    may be None): norm per head (None weights: no norm), rotation by positions (device int32, None: 0, 1, ..),
    k and v stored at `rows` (device int64, negative: not stored) of k_out, v_out [n_rows][H_kv][D].
    Returns (q_out, k_out, v_out)."""
    lead = q if q is not None else k
    if lead is None or lead.dim() != 3:
        raise ValueError("q or k is needed, [tokens][heads][head_dim]")
    dev, n_tok, D = lead.device, lead.shape[0], rope.head_dim
    H_q = H_kv = n_rows = ld_q = ld_k = ld_v = ld_qo = ld_ko = ld_vo = 0
    if q is not None:
        H_q = q.shape[1]
        ld_q = _rows("q", q, n_tok, H_q, D, dev)
        if q_out is None:
            q_out, ld_qo = torch.empty((n_tok, H_q, D), dtype=torch.bfloat16, device=dev), H_q * D
        else:
            ld_qo = _rows("q_out", q_out, n_tok, H_q, D, dev)
    if k is not None:
        H_kv = k.shape[1]
        ld_k = _rows("k", k, n_tok, H_kv, D, dev)
        if rows is not None and (k_out is None or (v is not None and v_out is None)):
            raise ValueError("rows needs k_out and v_out")
        if k_out is None:
            k_out = torch.empty((n_tok, H_kv, D), dtype=torch.bfloat16, device=dev)
        n_rows = k_out.shape[0]
        ld_ko = _rows("k_out", k_out, n_rows, H_kv, D, dev)
        if v is not None:
            ld_v = _rows("v", v, n_tok, H_kv, D, dev)
            if v_out is None:
                v_out = torch.empty((n_rows, H_kv, D), dtype=torch.bfloat16, device=dev)
            ld_vo = _rows("v_out", v_out, n_rows, H_kv, D, dev)
    elif v is not None:
        raise ValueError("v needs k")
    _want("q_norm_w", q_norm_w, torch.bfloat16, (D,), dev)
    _want("k_norm_w", k_norm_w, torch.bfloat16, (D,), dev)
    _want("positions", positions, torch.int32, (n_tok,), dev)
    _want("rows", rows, torch.int64, (n_tok,), dev)
    _want_err(err, dev)
    _run_on(dev, "gdn_qk_norm_rope", rope, n_tok, H_q, H_kv, _addr(q), ld_q, _addr(k), ld_k, _addr(v), ld_v,
            _addr(q_norm_w), _addr(k_norm_w), _addr(positions), _addr(rows), n_rows,
            None if q is None else q_out.data_ptr(), ld_qo, None if k is None else k_out.data_ptr(), ld_ko,
            None if v is None else v_out.data_ptr(), ld_vo, _addr(err))
    return q_out, k_out, v_out


def attention_tree(q_hat, k_tree, v_tree, k_cache, v_cache, cache_len, parent=None, T: int | None = None, *, g=None,
                   scale=None, out=None, workspace=None, err=None):
    """gdn_attention_tree: q_hat [N*T][H_q][D] over the caches [N][cap][H_kv][D] (cache_len device int32 [N] rows
    of each) and the nodes' own k_tree, v_tree [N*T][H_kv][D]; parent device int32 [N][T] (None: a chain,
    then T is needed unless N*T tells it), g the gate [N*T][H_q][D] or None.  scale defaults to D ** -0.5.
    Returns out [N*T][H_q*D] bf16."""
    N, cap, H_kv, D = k_cache.shape
    dev = k_cache.device
    T = T if T is not None else parent.shape[1] if parent is not None else q_hat.shape[0] // N if N else 1
    H_q = q_hat.shape[1]
    _want("k_cache", k_cache, torch.bfloat16, None, dev)
    _want("v_cache", v_cache, torch.bfloat16, k_cache.shape, dev)
    _want("cache_len", cache_len, torch.int32, (N,), dev)
    _want("parent", parent, torch.int32, (N, T), dev)
    n_tok = N * T
    ld_q = _rows("q_hat", q_hat, n_tok, H_q, D, dev)
    ld_kt = _rows("k_tree", k_tree, n_tok, H_kv, D, dev)
    ld_vt = _rows("v_tree", v_tree, n_tok, H_kv, D, dev)
    ld_g = 0 if g is None else _rows("g", g, n_tok, H_q, D, dev)
    if out is None:
        out = torch.empty((n_tok, H_q * D), dtype=torch.bfloat16, device=dev)
    else:
        _want("out", out, torch.bfloat16, (n_tok, H_q * D), dev)
    if workspace is None:
        workspace = torch.empty(attention_tree_workspace_size(H_q, H_kv, D, N, T), dtype=torch.uint8, device=dev)
    nbytes = _workspace_bytes(workspace, dev)
    _want_err(err, dev)
    _run_on(dev, "gdn_attention_tree", _addr(q_hat), ld_q, _addr(k_tree), ld_kt, _addr(v_tree), ld_vt, _addr(k_cache),
            _addr(v_cache), cap, _addr(cache_len), _addr(parent), _addr(g), ld_g, H_q, H_kv, D,
            D ** -0.5 if scale is None else scale, N, T, _addr(out), _addr(workspace), nbytes, _addr(err))
    return out


def attention_tree_workspace_size(H_q: int, H_kv: int, head_dim: int, N: int, T: int) -> int:
    return int(load().gdn_attention_tree_workspace_size(H_q, H_kv, head_dim, N, T))


def attn_tree_commit(k_tree, v_tree, T: int, parent, accepted, k_cache, v_cache, cache_len, *, cache_len_out=None,
                     err=None):
    """gdn_attn_tree_commit: the accepted paths' rows of k_tree, v_tree [N*T][H_kv][D] appended to the caches;
    cache_len_out (default cache_len itself) becomes the new lengths.  Returns it."""
    N, cap, H_kv, D = k_cache.shape
    dev = k_cache.device
    _want("k_cache", k_cache, torch.bfloat16, None, dev)
    _want("v_cache", v_cache, torch.bfloat16, k_cache.shape, dev)
    _want("parent", parent, torch.int32, (N, T), dev)
    _want("accepted", accepted, torch.int32, (N,), dev)
    _want("cache_len", cache_len, torch.int32, (N,), dev)
    if cache_len_out is None:
        cache_len_out = cache_len
    else:
        _want("cache_len_out", cache_len_out, torch.int32, (N,), dev)
    ld_kt = _rows("k_tree", k_tree, N * T, H_kv, D, dev)
    ld_vt = _rows("v_tree", v_tree, N * T, H_kv, D, dev)
    _want_err(err, dev)
    _run_on(dev, "gdn_attn_tree_commit", _addr(k_tree), ld_kt, _addr(v_tree), ld_vt, H_kv, D, N, T, _addr(parent),
            _addr(accepted), _addr(k_cache), _addr(v_cache), cap, _addr(cache_len), _addr(cache_len_out), _addr(err))
    return cache_len_out


def _want_slots(N, slots, state_slot):
    """Without slots sequence n has slot n, so the pool needs N (the layer's entry points are not told how many it has)."""
    if state_slot is None and slots < N:
        raise ValueError(f"{N} sequences need {N} slots (or state_slot), not {slots}")


def layer_tree_workspace(L: GdnLayer, N: int, T: int, device):
    """The workspace of layer_decode_tree, kept until layer_tree_commit."""
    return torch.empty(int(load().gdn_layer_tree_workspace_size(L.H_k, L.H_v, N, T)), dtype=torch.uint8, device=device)


def layer_decode_tree(L: GdnLayer, N: int, T: int, parent, x, state, conv_state, workspace, state_slot=None, *, y=None,
                      err=None):
    """gdn_layer_decode_tree: x [N*T][hidden] -> y; state and conv_state are read, `workspace` keeps the projection
    for layer_tree_commit.  Returns y."""
    slots, dev = _want_pool(L.H_k, L.H_v, state, conv_state)
    _want_made(L, dev)
    _want_slots(N, slots, state_slot)
    _want("parent", parent, torch.int32, (N, T), dev)
    _want("state_slot", state_slot, torch.int32, (N,), dev)
    ldx = _matrix("x", x, N * T, L.hidden, dev)
    if y is None:
        y = torch.empty(N * T, L.hidden, dtype=torch.bfloat16, device=dev)
    ldy = _matrix("y", y, N * T, L.hidden, dev)
    nbytes = _workspace_bytes(workspace, dev)
    _want_err(err, dev)
    _run_on(dev, "gdn_layer_decode_tree", L, N, T, _addr(parent), _addr(x), ldx, _addr(state),
            _addr(conv_state), _addr(state_slot), slots, _addr(y), ldy, _addr(workspace), nbytes,
            _addr(err))
    return y


def layer_tree_commit(L: GdnLayer, N: int, T: int, parent, accepted, state, conv_state, workspace, state_slot=None, *,
                      err=None):
    """gdn_layer_tree_commit: state and conv_state advanced in place along the accepted paths of the
    layer_decode_tree call that left `workspace`."""
    slots, dev = _want_pool(L.H_k, L.H_v, state, conv_state)
    _want_made(L, dev)
    _want_slots(N, slots, state_slot)
    _want("parent", parent, torch.int32, (N, T), dev)
    _want("accepted", accepted, torch.int32, (N,), dev)
    _want("state_slot", state_slot, torch.int32, (N,), dev)
    nbytes = _workspace_bytes(workspace, dev)
    _want_err(err, dev)
    _run_on(dev, "gdn_layer_tree_commit", L, N, T, _addr(parent), _addr(accepted), _addr(state),
            _addr(conv_state), _addr(state_slot), slots, _addr(workspace), nbytes, _addr(err))


def attn_layer_tree_workspace(N: int, T: int, device):
    """The workspace of attn_layer_decode_tree, kept until attn_layer_tree_commit."""
    return torch.empty(int(load().gdn_attn_layer_tree_workspace_size(N, T)), dtype=torch.uint8, device=device)


def _want_attn_cache(N, k_cache, v_cache, cache_len):
    shape = (N, k_cache.shape[1], ATTN_KV_HEADS, ATTN_HEAD_DIM)
    _want("k_cache", k_cache, torch.bfloat16, shape)
    _want("v_cache", v_cache, torch.bfloat16, shape, k_cache.device)
    _want("cache_len", cache_len, torch.int32, (N,), k_cache.device)
    return k_cache.device, shape[1]


def attn_layer_decode_tree(L: GdnAttnLayer, N: int, T: int, parent, x, k_cache, v_cache, cache_len, workspace, *, y=None,
                           err=None):
    """gdn_attn_layer_decode_tree: x [N*T][hidden] -> y; the caches and cache_len are read, `workspace` keeps the
    nodes' keys and values for attn_layer_tree_commit.  Returns y."""
    dev, cap = _want_attn_cache(N, k_cache, v_cache, cache_len)
    _want_made(L, dev)
    _want("parent", parent, torch.int32, (N, T), dev)
    ldx = _matrix("x", x, N * T, L.hidden, dev)
    if y is None:
        y = torch.empty(N * T, L.hidden, dtype=torch.bfloat16, device=dev)
    ldy = _matrix("y", y, N * T, L.hidden, dev)
    nbytes = _workspace_bytes(workspace, dev)
    _want_err(err, dev)
    _run_on(dev, "gdn_attn_layer_decode_tree", L, N, T, _addr(parent), _addr(x), ldx, _addr(k_cache),
            _addr(v_cache), cap, _addr(cache_len), _addr(y), ldy, _addr(workspace), nbytes, _addr(err))
    return y


def attn_layer_tree_commit(N: int, T: int, parent, accepted, k_cache, v_cache, cache_len, workspace, *, err=None):
    """gdn_attn_layer_tree_commit: the accepted paths appended to the caches, cache_len advanced in place."""
    dev, cap = _want_attn_cache(N, k_cache, v_cache, cache_len)
    _want("parent", parent, torch.int32, (N, T), dev)
    _want("accepted", accepted, torch.int32, (N,), dev)
    nbytes = _workspace_bytes(workspace, dev)
    _want_err(err, dev)
    _run_on(dev, "gdn_attn_layer_tree_commit", N, T, _addr(parent), _addr(accepted), _addr(k_cache), _addr(v_cache), cap,
            _addr(cache_len), _addr(workspace), nbytes, _addr(err))


def status_string(status: int) -> str:
    return load().gdn_status_string(status).decode()


def err_status(err_word: int) -> int:
    """gdn_err_status: the gdn_status an error word read back from the device stands for."""
    return load().gdn_err_status(int(err_word))
