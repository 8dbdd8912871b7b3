"""Thin ctypes binding of the C ABI in ``include/attn.h`` (argument marshalling only).

Every function here has the name of the C entry point it calls.  Tensors are
torch tensors on a CUDA device; the binding checks dtypes, shapes and
contiguity, allocates outputs the caller did not pass (torch supplies device
memory), and hands raw pointers plus the current torch stream to the library.
All computation happens in the library's CUDA kernels.  If the library has not
been built, the first call raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libattn_gb300.so")

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_ALIGNMENT = 3
ATTN_ERR_CUDA = 4
ATTN_ERR_DEVICE_TIMEOUT = 5
ATTN_ERR_DEVICE_BOUNDS = 6
ATTN_ERR_SCRATCH_TOO_SMALL = 7
ATTN_ERR_DEVICE_POOL = 8
ATTN_DTYPE_BF16 = 0
ATTN_DTYPE_F32 = 1

# Every symbol include/attn.h declares.
EXPORTED = (
    "attn_fwd",
    "attn_fwd_ex",
    "attn_decode",
    "attn_decode_ex",
    "attn_decode_noalloc",
    "attn_decode_paged",
    "attn_decode_multi",
    "attn_decode_workspace_bytes",
    "attn_page_step",
    "attn_qk_norm_rope",
    "attn_kv_q4_page_bytes",
    "attn_kv_append_q4",
    "attn_kv_gather_q4",
    "attn_decode_q4",
    "attn_decode_q4_workspace_bytes",
    "attn_rope_tables",
    "attn_kv_append_paged",
    "attn_decode_multi_paged",
    "attn_decode_multi_paged_workspace_bytes",
    "attn_verify_drafts",
    "attn_get_device_status",
    "attn_status_string",
    "attn_release_workspace",
    "attn_selftest_wait_timeout",
    "attn_version",
)


ATTN_ROPE_NONE = 0
ATTN_ROPE_HALF = 1
ATTN_ROPE_INTERLEAVED = 2
_ROPE_STYLES = {"half": ATTN_ROPE_HALF, "interleaved": ATTN_ROPE_INTERLEAVED}
ATTN_ROPE_SCALE_NONE = 0
ATTN_ROPE_SCALE_LINEAR = 1
ATTN_ROPE_SCALE_BASE = 2
ATTN_ROPE_SCALE_TURNS = 3
ATTN_ROPE_SCALE_INDEX = 4


class attn_rope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("max_pos", ctypes.c_int), ("style", ctypes.c_int),
                ("k_out", ctypes.c_void_p)]


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class attn_fwd_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
        ("Lq", ctypes.c_int), ("Lkv", ctypes.c_int), ("D", ctypes.c_int),
        ("scale", ctypes.c_float), ("causal", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
        ("total_q", ctypes.c_int), ("total_k", ctypes.c_int),
        ("stream", ctypes.c_void_p),
        ("rope", attn_rope),
    ]


class attn_decode_paged_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("kpages", ctypes.c_void_p), ("vpages", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
        ("scale", ctypes.c_float), ("out_dtype", ctypes.c_int), ("chunk", ctypes.c_int),
        ("stream", ctypes.c_void_p),
        ("rope", attn_rope),
    ]


class attn_decode_multi_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("kcache", ctypes.c_void_p), ("vcache", ctypes.c_void_p),
        ("kv_lens", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("Lq", ctypes.c_int),
        ("Lmax", ctypes.c_int), ("D", ctypes.c_int),
        ("scale", ctypes.c_float), ("out_dtype", ctypes.c_int),
        ("stream", ctypes.c_void_p),
        ("rope", attn_rope),
    ]


class attn_decode_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("kcache", ctypes.c_void_p), ("vcache", ctypes.c_void_p),
        ("kv_lens", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
        ("Lmax", ctypes.c_int), ("D", ctypes.c_int),
        ("scale", ctypes.c_float), ("out_dtype", ctypes.c_int), ("chunk", ctypes.c_int),
        ("stream", ctypes.c_void_p),
        ("rope", attn_rope),
    ]


class attn_page_step_params(ctypes.Structure):
    _fields_ = [
        ("kv_lens", ctypes.c_void_p), ("keep_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p),
        ("cu_new", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("B", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
        ("max_tokens", ctypes.c_int),
        ("stream", ctypes.c_void_p),
    ]


# The stride arrays and the rope member of the next two are spelled out field by field (the same layout): filling a
# nested member from Python costs as much as ten plain ones.
class attn_qk_norm_rope_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("B", ctypes.c_int), ("L", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("eps", ctypes.c_float),
        *((f"{t}_{axis}_stride", ctypes.c_longlong) for t in ("q", "k", "q_out", "k_out")
          for axis in ("sequence", "token", "head")),
        ("rope_cos", ctypes.c_void_p), ("rope_sin", ctypes.c_void_p), ("rope_max_pos", ctypes.c_int),
        ("rope_style", ctypes.c_int), ("rope_k_out", ctypes.c_void_p),
        ("stream", ctypes.c_void_p),
    ]


class attn_kv_append_q4_params(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pool", ctypes.c_void_p), ("slots", ctypes.c_void_p),
        ("T", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int), ("page_size", ctypes.c_int),
        ("num_pages", ctypes.c_int),
        *((f"{t}_{axis}_stride", ctypes.c_longlong) for t in ("k", "v") for axis in ("token", "head")),
        ("stream", ctypes.c_void_p),
    ]


class attn_kv_gather_q4_params(ctypes.Structure):
    _fields_ = [
        ("pool", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("cu_k", ctypes.c_void_p),
        ("kv_starts", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("B", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int), ("page_size", ctypes.c_int),
        ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int), ("total_k", ctypes.c_int),
        ("stream", ctypes.c_void_p),
    ]


class attn_decode_q4_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("pool", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("kv_lens", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("Lq", ctypes.c_int), ("D", ctypes.c_int),
        ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
        ("scale", ctypes.c_float), ("out_dtype", ctypes.c_int), ("chunk", ctypes.c_int),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_ulonglong),
        ("stream", ctypes.c_void_p),
    ]


class attn_rope_tables_params(ctypes.Structure):
    _fields_ = [
        ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p),
        ("rows", ctypes.c_int), ("start", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("scaling", ctypes.c_int),
        ("base", ctypes.c_double), ("factor", ctypes.c_double), ("context", ctypes.c_double), ("low", ctypes.c_double),
        ("high", ctypes.c_double), ("amplitude", ctypes.c_double),
        ("stream", ctypes.c_void_p),
    ]


class attn_kv_append_paged_params(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("kpages", ctypes.c_void_p), ("vpages", ctypes.c_void_p),
        ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
        ("k_out", ctypes.c_void_p),
        ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int), ("rotary_dim", ctypes.c_int),
        *((f"{t}_{axis}_stride", ctypes.c_longlong) for t in ("k", "v", "q", "q_out", "k_out")
          for axis in ("token", "head")),
        ("rope_cos", ctypes.c_void_p), ("rope_sin", ctypes.c_void_p), ("rope_max_pos", ctypes.c_int),
        ("rope_style", ctypes.c_int), ("rope_k_out", ctypes.c_void_p),
        ("stream", ctypes.c_void_p),
    ]


class attn_decode_multi_paged_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("kpages", ctypes.c_void_p), ("vpages", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("cu_new", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("max_new", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
        ("num_pages", ctypes.c_int), ("scale", ctypes.c_float), ("out_dtype", ctypes.c_int),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_ulonglong),
        ("stream", ctypes.c_void_p),
    ]


class attn_verify_drafts_params(ctypes.Structure):
    _fields_ = [
        ("draft_tokens", ctypes.c_void_p), ("target_probs", ctypes.c_void_p), ("draft_probs", ctypes.c_void_p),
        ("uniforms", ctypes.c_void_p), ("cu_target", ctypes.c_void_p), ("draft_lens", ctypes.c_void_p),
        ("kv_lens", ctypes.c_void_p), ("tokens", ctypes.c_void_p), ("accepted", ctypes.c_void_p),
        ("keep_lens", ctypes.c_void_p),
        ("B", ctypes.c_int), ("K", ctypes.c_int), ("V", ctypes.c_int), ("total", ctypes.c_int), ("dtype", ctypes.c_int),
        *((f"{t}_{axis}_stride", ctypes.c_longlong) for t in ("target", "draft") for axis in ("sequence", "row")),
        ("stream", ctypes.c_void_p),
    ]


_lib = None
_lock = threading.Lock()


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library once (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"attention library not built: {path} is missing (run __graft_entry__.build())")
        lib = ctypes.CDLL(path)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, P]
        lib.attn_fwd.restype = I
        lib.attn_fwd_ex.argtypes = [ctypes.POINTER(attn_fwd_params)]
        lib.attn_fwd_ex.restype = I
        lib.attn_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, P]
        lib.attn_decode.restype = I
        lib.attn_decode_ex.argtypes = [ctypes.POINTER(attn_decode_params)]
        lib.attn_decode_ex.restype = I
        lib.attn_decode_noalloc.argtypes = [ctypes.POINTER(attn_decode_params)]
        lib.attn_decode_noalloc.restype = I
        lib.attn_decode_paged.argtypes = [ctypes.POINTER(attn_decode_paged_params)]
        lib.attn_decode_paged.restype = I
        lib.attn_decode_multi.argtypes = [ctypes.POINTER(attn_decode_multi_params)]
        lib.attn_decode_multi.restype = I
        lib.attn_decode_workspace_bytes.argtypes = [I, I, I, I, I, I]
        lib.attn_decode_workspace_bytes.restype = ctypes.c_ulonglong
        lib.attn_page_step.argtypes = [ctypes.POINTER(attn_page_step_params)]
        lib.attn_page_step.restype = I
        lib.attn_qk_norm_rope.argtypes = [ctypes.POINTER(attn_qk_norm_rope_params)]
        lib.attn_qk_norm_rope.restype = I
        lib.attn_kv_q4_page_bytes.argtypes = [I, I, I]
        lib.attn_kv_q4_page_bytes.restype = ctypes.c_ulonglong
        lib.attn_kv_append_q4.argtypes = [ctypes.POINTER(attn_kv_append_q4_params)]
        lib.attn_kv_append_q4.restype = I
        lib.attn_kv_gather_q4.argtypes = [ctypes.POINTER(attn_kv_gather_q4_params)]
        lib.attn_kv_gather_q4.restype = I
        lib.attn_decode_q4.argtypes = [ctypes.POINTER(attn_decode_q4_params)]
        lib.attn_decode_q4.restype = I
        lib.attn_decode_q4_workspace_bytes.argtypes = [I, I, I, I]
        lib.attn_decode_q4_workspace_bytes.restype = ctypes.c_ulonglong
        for name, cls in (("attn_rope_tables", attn_rope_tables_params),
                          ("attn_kv_append_paged", attn_kv_append_paged_params),
                          ("attn_decode_multi_paged", attn_decode_multi_paged_params),
                          ("attn_verify_drafts", attn_verify_drafts_params)):
            lib[name].argtypes, lib[name].restype = [ctypes.POINTER(cls)], I
            setattr(lib, name, lib[name])
        lib.attn_decode_multi_paged_workspace_bytes.argtypes = [I, I, I, I]
        lib.attn_decode_multi_paged_workspace_bytes.restype = ctypes.c_ulonglong
        lib.attn_get_device_status.argtypes = [P]
        lib.attn_get_device_status.restype = I
        lib.attn_status_string.argtypes = [I]
        lib.attn_status_string.restype = ctypes.c_char_p
        lib.attn_release_workspace.argtypes = []
        lib.attn_release_workspace.restype = None
        lib.attn_selftest_wait_timeout.argtypes = [ctypes.c_uint, P]
        lib.attn_selftest_wait_timeout.restype = I
        lib.attn_version.argtypes = []
        lib.attn_version.restype = I
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().attn_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != ATTN_OK:
        raise AttnError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype, ndim, shape=None, device=None):
    """Check a tensor argument; ``shape`` and ``device``, when given, must match exactly (outputs are written
    by the kernels over their full extent, so a smaller buffer must never reach the library)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _set_rope(p, rope, D, device, k_shape=None):
    """rope = (cos, sin, style) or (cos, sin, style, k_out): fp32 device tables [max_pos, D/2], "half" or
    "interleaved", and for prefill an optional bf16 tensor shaped like k receiving the rotated keys (None: off)."""
    if rope is None:
        return
    cos, sin, style = rope[:3]
    k_out = rope[3] if len(rope) > 3 else None
    if k_out is not None:
        if k_shape is None:
            raise ValueError("rope k_out is taken by prefill calls only")
        _need(k_out, "rope k_out", torch.bfloat16, len(k_shape), k_shape, device)
        p.rope.k_out = _ptr(k_out)
    for t, name in ((cos, "rope cos"), (sin, "rope sin")):
        _need(t, name, torch.float32, 2)
        if t.device != device or t.shape[1] != D // 2:
            raise ValueError(f"{name} must be [max_pos, D/2] on {device}")
    if cos.shape != sin.shape:
        raise ValueError("rope cos and sin tables differ in shape")
    if style not in _ROPE_STYLES:
        raise ValueError("rope style must be 'half' or 'interleaved'")
    p.rope.cos, p.rope.sin = _ptr(cos), _ptr(sin)
    p.rope.max_pos = cos.shape[0]
    p.rope.style = _ROPE_STYLES[style]


def attn_fwd(q, k, v, out=None, lse=None, causal=True, scale=None, out_dtype=torch.bfloat16,
             want_lse=True, stream=None, rope=None):
    """Dense prefill: q [B,Hq,Lq,D], k/v [B,Hkv,Lkv,D] bf16 -> (out [B,Hq,Lq,D], lse [B,Hq,Lq] fp32).

    ``rope = (cos, sin, style)`` rotates q and k inside the call (fp32 device tables [max_pos, D/2];
    style "half" or "interleaved"); every call that takes ``rope`` takes the same argument."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 4, device=q.device)
    _need(v, "v", torch.bfloat16, 4, device=q.device)
    B, Hq, Lq, D = q.shape
    Hkv, Lkv = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, Hkv, Lkv, D) or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"k/v shapes {tuple(k.shape)} {tuple(v.shape)} do not match q {tuple(q.shape)}")
    if out is None:
        out = torch.empty((B, Hq, Lq, D), dtype=out_dtype, device=q.device)
    _need(out, "out", out_dtype, 4, (B, Hq, Lq, D), q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 3, (B, Hq, Lq), q.device)
    p = attn_fwd_params()
    p.q, p.k, p.v, p.out, p.lse = (_ptr(t) for t in (q, k, v, out, lse))
    p.B, p.Hq, p.Hkv, p.Lq, p.Lkv, p.D = B, Hq, Hkv, Lq, Lkv, D
    p.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    p.causal = int(bool(causal))
    p.out_dtype = ATTN_DTYPE_F32 if out_dtype == torch.float32 else ATTN_DTYPE_BF16
    p.stream = _stream_handle(stream, q.device)
    _set_rope(p, rope, D, q.device, tuple(k.shape))
    _check(load().attn_fwd_ex(ctypes.byref(p)), "attn_fwd")
    return out, lse


def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, out=None, lse=None,
                    causal=True, scale=None, out_dtype=torch.bfloat16, want_lse=True, stream=None, rope=None):
    """Packed prefill: q [total_q,Hq,D], k/v [total_k,Hkv,D] bf16, cu_seqlens int32 [B+1] on the device."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, 3, device=q.device)
    _need(v, "v", torch.bfloat16, 3, device=q.device)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1, device=q.device)
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1, device=q.device)
    total_q, Hq, D = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    B = cu_seqlens_q.shape[0] - 1
    if cu_seqlens_k.shape[0] != B + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    if out is None:
        out = torch.empty((total_q, Hq, D), dtype=out_dtype, device=q.device)
    _need(out, "out", out_dtype, 3, (total_q, Hq, D), q.device)
    if lse is None and want_lse:
        lse = torch.empty((total_q, Hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2, (total_q, Hq), q.device)
    p = attn_fwd_params()
    p.q, p.k, p.v, p.out, p.lse = (_ptr(t) for t in (q, k, v, out, lse))
    p.B, p.Hq, p.Hkv, p.Lq, p.Lkv, p.D = B, Hq, Hkv, int(max_seqlen_q), int(max_seqlen_k), D
    p.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    p.causal = int(bool(causal))
    p.out_dtype = ATTN_DTYPE_F32 if out_dtype == torch.float32 else ATTN_DTYPE_BF16
    p.cu_seqlens_q, p.cu_seqlens_k = _ptr(cu_seqlens_q), _ptr(cu_seqlens_k)
    p.total_q, p.total_k = total_q, total_k
    p.stream = _stream_handle(stream, q.device)
    _set_rope(p, rope, D, q.device, tuple(k.shape))
    _check(load().attn_fwd_ex(ctypes.byref(p)), "attn_fwd_ex")
    return out, lse


def attn_decode(q, kcache, vcache, kv_lens, out=None, lse=None, scale=None, chunk=0,
                out_dtype=torch.bfloat16, want_lse=True, stream=None, rope=None):
    """Decode: q [B,Hq,D], caches [B,Hkv,Lmax,D] bf16, kv_lens int32 [B] -> (out [B,Hq,D], lse [B,Hq])."""
    _need(q, "q", torch.bfloat16, 3)
    _need(kcache, "kcache", torch.bfloat16, 4, device=q.device)
    _need(vcache, "vcache", torch.bfloat16, 4, device=q.device)
    _need(kv_lens, "kv_lens", torch.int32, 1, device=q.device)
    B, Hq, D = q.shape
    Hkv, Lmax = kcache.shape[1], kcache.shape[2]
    if tuple(kcache.shape) != (B, Hkv, Lmax, D) or tuple(vcache.shape) != tuple(kcache.shape):
        raise ValueError("cache shapes do not match q")
    if kv_lens.shape[0] != B:
        raise ValueError("kv_lens must have B entries")
    if out is None:
        out = torch.empty((B, Hq, D), dtype=out_dtype, device=q.device)
    _need(out, "out", out_dtype, 3, (B, Hq, D), q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2, (B, Hq), q.device)
    p = attn_decode_params()
    p.q, p.kcache, p.vcache, p.kv_lens, p.out, p.lse = (_ptr(t) for t in (q, kcache, vcache, kv_lens, out, lse))
    p.B, p.Hq, p.Hkv, p.Lmax, p.D = B, Hq, Hkv, Lmax, D
    p.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    p.out_dtype = ATTN_DTYPE_F32 if out_dtype == torch.float32 else ATTN_DTYPE_BF16
    p.chunk = int(chunk)
    p.stream = _stream_handle(stream, q.device)
    _set_rope(p, rope, D, q.device)
    _check(load().attn_decode_ex(ctypes.byref(p)), "attn_decode")
    return out, lse


def attn_decode_paged(q, kpages, vpages, block_table, kv_lens, out=None, lse=None, scale=None, chunk=0,
                      out_dtype=torch.bfloat16, want_lse=True, stream=None, rope=None):
    """Decode over a paged cache: pages [num_pages,Hkv,page_size,D] bf16, block_table int32 [B,max_pages]."""
    _need(q, "q", torch.bfloat16, 3)
    _need(kpages, "kpages", torch.bfloat16, 4, device=q.device)
    _need(vpages, "vpages", torch.bfloat16, 4, device=q.device)
    _need(block_table, "block_table", torch.int32, 2, device=q.device)
    _need(kv_lens, "kv_lens", torch.int32, 1, device=q.device)
    B, Hq, D = q.shape
    num_pages, Hkv, page_size = kpages.shape[0], kpages.shape[1], kpages.shape[2]
    if tuple(kpages.shape) != (num_pages, Hkv, page_size, D) or tuple(vpages.shape) != tuple(kpages.shape):
        raise ValueError("page pool shapes do not match q")
    if block_table.shape[0] != B or kv_lens.shape[0] != B:
        raise ValueError("block_table and kv_lens must have B rows")
    if out is None:
        out = torch.empty((B, Hq, D), dtype=out_dtype, device=q.device)
    _need(out, "out", out_dtype, 3, (B, Hq, D), q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2, (B, Hq), q.device)
    p = attn_decode_paged_params()
    p.q, p.kpages, p.vpages = _ptr(q), _ptr(kpages), _ptr(vpages)
    p.block_table, p.kv_lens, p.out, p.lse = _ptr(block_table), _ptr(kv_lens), _ptr(out), _ptr(lse)
    p.B, p.Hq, p.Hkv, p.D = B, Hq, Hkv, D
    p.page_size, p.max_pages, p.num_pages = page_size, block_table.shape[1], num_pages
    p.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    p.out_dtype = ATTN_DTYPE_F32 if out_dtype == torch.float32 else ATTN_DTYPE_BF16
    p.chunk = int(chunk)
    p.stream = _stream_handle(stream, q.device)
    _set_rope(p, rope, D, q.device)
    _check(load().attn_decode_paged(ctypes.byref(p)), "attn_decode_paged")
    return out, lse


def attn_decode_multi(q, kcache, vcache, kv_lens, out=None, lse=None, scale=None, out_dtype=torch.bfloat16,
                      want_lse=True, stream=None, rope=None):
    """Multi-token decode: q [B,Hq,Lq,D], caches [B,Hkv,Lmax,D] bf16, kv_lens int32 [B] counting the new tokens'
    own keys -> (out [B,Hq,Lq,D], lse [B,Hq,Lq])."""
    _need(q, "q", torch.bfloat16, 4)
    _need(kcache, "kcache", torch.bfloat16, 4, device=q.device)
    _need(vcache, "vcache", torch.bfloat16, 4, device=q.device)
    _need(kv_lens, "kv_lens", torch.int32, 1, device=q.device)
    B, Hq, Lq, D = q.shape
    Hkv, Lmax = kcache.shape[1], kcache.shape[2]
    if tuple(kcache.shape) != (B, Hkv, Lmax, D) or tuple(vcache.shape) != tuple(kcache.shape):
        raise ValueError("cache shapes do not match q")
    if kv_lens.shape[0] != B:
        raise ValueError("kv_lens must have B entries")
    if out is None:
        out = torch.empty((B, Hq, Lq, D), dtype=out_dtype, device=q.device)
    _need(out, "out", out_dtype, 4, (B, Hq, Lq, D), q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 3, (B, Hq, Lq), q.device)
    p = attn_decode_multi_params()
    p.q, p.kcache, p.vcache, p.kv_lens, p.out, p.lse = (_ptr(t) for t in (q, kcache, vcache, kv_lens, out, lse))
    p.B, p.Hq, p.Hkv, p.Lq, p.Lmax, p.D = B, Hq, Hkv, Lq, Lmax, D
    p.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    p.out_dtype = ATTN_DTYPE_F32 if out_dtype == torch.float32 else ATTN_DTYPE_BF16
    p.stream = _stream_handle(stream, q.device)
    _set_rope(p, rope, D, q.device)
    _check(load().attn_decode_multi(ctypes.byref(p)), "attn_decode_multi")
    return out, lse


def attn_decode_noalloc(q, kcache, vcache, kv_lens, out, lse=None, scale=None, chunk=0, stream=None, rope=None):
    """Decode through the entry point that allocates no device memory.

    For callers that cannot allocate (inside CUDA graph capture, engines that
    hand all of HBM to their own pool, latency paths that cannot take
    cudaMalloc's synchronisation).  ``out`` (and ``lse`` if wanted) must be
    passed in; the split-KV partials go to a fixed 4 MiB buffer inside the
    library, shared by every call on the device, so calls that may overlap on
    the GPU must be ordered on one stream.  The first call on a device does a
    one-time address lookup and should not be inside a stream capture.
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(kcache, "kcache", torch.bfloat16, 4, device=q.device)
    _need(vcache, "vcache", torch.bfloat16, 4, device=q.device)
    _need(kv_lens, "kv_lens", torch.int32, 1, device=q.device)
    B, Hq, D = q.shape
    Hkv, Lmax = kcache.shape[1], kcache.shape[2]
    if tuple(kcache.shape) != (B, Hkv, Lmax, D) or tuple(vcache.shape) != tuple(kcache.shape):
        raise ValueError("cache shapes do not match q")
    if kv_lens.shape[0] != B:
        raise ValueError("kv_lens must have B entries")
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be bf16 or fp32")
    _need(out, "out", out.dtype, 3, (B, Hq, D), q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2, (B, Hq), q.device)
    p = attn_decode_params()
    p.q, p.kcache, p.vcache, p.kv_lens, p.out, p.lse = (_ptr(t) for t in (q, kcache, vcache, kv_lens, out, lse))
    p.B, p.Hq, p.Hkv, p.Lmax, p.D = B, Hq, Hkv, Lmax, D
    p.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    p.out_dtype = ATTN_DTYPE_F32 if out.dtype == torch.float32 else ATTN_DTYPE_BF16
    p.chunk = int(chunk)
    p.stream = _stream_handle(stream, q.device)
    _set_rope(p, rope, D, q.device)
    _check(load().attn_decode_noalloc(ctypes.byref(p)), "attn_decode_noalloc")
    return out, lse


# The raw handle of a device's current stream without building a Stream object (2 us of a small call on the host), and
# the current device without asking whether CUDA is set up (the arguments are CUDA tensors).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(stream, index):
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


_CODES = {ctypes.c_void_p: "P", ctypes.c_int: "i", ctypes.c_longlong: "q", ctypes.c_ulonglong: "Q", ctypes.c_float: "f",
          ctypes.c_double: "d"}
_entries = {}


def _entry(name, cls):
    """Entry point `name` as a call that takes its parameters' bytes, and their packing: all fields of the structure cls
    in order (native alignment), with 0 for a null pointer.  Filling a structure takes 0.4 to 1.1 us longer."""
    fn = load()[name]
    fn.argtypes, fn.restype = [ctypes.c_char_p], ctypes.c_int
    layout = struct.Struct("@" + "".join(_CODES[t] for _, t in cls._fields_) + "0P")
    assert layout.size == ctypes.sizeof(cls)
    _entries[name] = entry = (layout.pack, fn)
    return entry


def _call(name, cls, index, *fields):
    """Run one entry point with device `index` current."""
    pack, fn = _entries.get(name) or _entry(name, cls)
    try:
        p = pack(*fields)
    except (struct.error, OverflowError) as e:  # a number that does not fit its field, or none
        raise ValueError(f"{name}: {e}") from None
    if index == _current_device():
        status = fn(p)
    else:
        with torch.cuda.device(index):
            status = fn(p)
    if status != ATTN_OK:
        raise AttnError(status, name)


def _fit(t, name, dtype, shape, index):
    """The address of a contiguous tensor of just this type and shape on device `index` (_need, told shortly: a decode
    step's calls take microseconds, and so may their checks)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0 and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:  # not a tensor: told below
        pass
    _need(t, name, dtype, len(shape), shape, torch.device("cuda", max(index, 0)))
    raise ValueError(f"{name}: not a contiguous CUDA tensor of shape {tuple(shape)}")


def _rows(t, name, ndim, index=None):
    """A bf16 CUDA tensor (on device `index`) whose rows (the last axis) are contiguous; the other axes may have any
    stride that is a multiple of 8 elements.  Returns its strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    st = t.stride()
    if len(st) != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    at = t.get_device()
    if at < 0 or (index is not None and at != index):
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on cuda:{index}" if index is not None else ""))
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return st


def _written_once(t, name):
    """A tensor to be written: no two of its elements may share memory."""
    need = 1
    for n, st in sorted(((n, st) for n, st in zip(t.shape, t.stride()) if n > 1), key=lambda a: a[1]):
        if st < need:
            raise ValueError(f"{name}: elements overlap")
        need = st * (n - 1) + need


def attn_page_step(kv_lens, block_table, free_pages, free_count, page_size, new_lens=None, keep_lens=None, slots=None,
                   positions=None, cu_new=None, stream=None):
    """Pages and slots of a serving step, on the GPU (all int32): row b keeps keep_lens[b] (default: all) of its
    kv_lens[b] keys and gets new_lens[b] (default: 0) tokens.  kv_lens [B], block_table [B,max_pages],
    free_pages [num_pages] (a stack) and free_count [1] are updated in place; slots and positions [max_tokens] and
    cu_new [B+1], where given, are written.  -> (slots, positions, cu_new)"""
    i32 = torch.int32
    _need(kv_lens, "kv_lens", i32, 1)
    at = kv_lens.get_device()
    B = kv_lens.shape[0]
    width = block_table.shape[-1] if isinstance(block_table, torch.Tensor) and block_table.dim() else 0
    pages = free_pages.shape[0] if isinstance(free_pages, torch.Tensor) and free_pages.dim() else 0
    rooms = [t.shape[0] for t in (slots, positions) if isinstance(t, torch.Tensor) and t.dim()]
    room = rooms[0] if rooms else 0
    if len(rooms) == 2 and rooms[1] != room:
        raise ValueError("slots and positions must have the same length")
    _call("attn_page_step", attn_page_step_params, at,
          kv_lens.data_ptr(),
          0 if keep_lens is None else _fit(keep_lens, "keep_lens", i32, (B,), at),
          0 if new_lens is None else _fit(new_lens, "new_lens", i32, (B,), at),
          _fit(block_table, "block_table", i32, (B, width), at),
          _fit(free_pages, "free_pages", i32, (pages,), at),
          _fit(free_count, "free_count", i32, (1,), at),
          0 if cu_new is None else _fit(cu_new, "cu_new", i32, (B + 1,), at),
          # (a list without room has no address of its own, and is none the less a list: any other stands for it)
          0 if slots is None else _fit(slots, "slots", i32, (room,), at) or kv_lens.data_ptr(),
          0 if positions is None else _fit(positions, "positions", i32, (room,), at) or kv_lens.data_ptr(),
          B, int(page_size), width, pages, room, _stream_of(stream, at))
    return slots, positions, cu_new


def attn_qk_norm_rope(q, k, q_weight=None, k_weight=None, rope=None, positions=None, eps=1e-6, q_out=None, k_out=None,
                      stream=None):
    """RMS norm of every q and k head and its rotation, in one pass: q [T,Hq,D] and k [T,Hkv,D] (packed), or
    [B,H,L,D] (dense), bf16 with any strides over contiguous rows (k may be None); weights bf16 [D] or None;
    rope = (cos, sin, style); positions int32 [T] or [B,L], -1 for padded rows, which are left as they were.
    q_out/k_out may be q/k themselves.  -> (q_out, k_out)"""
    dense = isinstance(q, torch.Tensor) and q.dim() == 4
    ndim = 4 if dense else 3
    sq = _rows(q, "q", ndim)
    at = q.get_device()
    if dense:
        B, Hq, L, D = q.shape
    else:
        B, (L, Hq, D) = 1, q.shape
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    sqo = _out_rows(q_out, "q_out", q, ndim, at)
    if k is None:
        if k_out is not None or k_weight is not None:
            raise ValueError("k_out and k_weight go with k")
        Hkv, sk, sko, kp, kop = 0, sq, sqo, 0, 0
    else:
        sk = _rows(k, "k", ndim, at)
        Hkv = k.shape[1]
        if k.shape != ((B, Hkv, L, D) if dense else (L, Hkv, D)):
            raise ValueError(f"k shape {tuple(k.shape)} does not match q {tuple(q.shape)}")
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=k.device)
        sko = _out_rows(k_out, "k_out", k, ndim, at)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    # as sequence, token, head
    if dense:
        strides = tuple(st[i] for st in (sq, sk, sqo, sko) for i in (0, 2, 1))
    else:
        strides = (0, sq[0], sq[1], 0, sk[0], sk[1], 0, sqo[0], sqo[1], 0, sko[0], sko[1])
    if rope is None:
        r = _NO_ROPE
    else:
        if len(rope) > 3 and rope[3] is not None:
            raise ValueError("rope k_out is taken by prefill calls only")
        cos, sin, style = rope[:3]
        if style not in _ROPE_STYLES:
            raise ValueError("rope style must be 'half' or 'interleaved'")
        tab = (cos.shape[0] if isinstance(cos, torch.Tensor) and cos.dim() else 0, D // 2)
        if tab[0] == 0:
            raise ValueError("rope tables must have rows")
        r = (_fit(cos, "rope cos", torch.float32, tab, at), _fit(sin, "rope sin", torch.float32, tab, at), tab[0],
             _ROPE_STYLES[style], 0)
    _call("attn_qk_norm_rope", attn_qk_norm_rope_params, at,
          q.data_ptr(), kp, q_out.data_ptr(), kop,
          0 if q_weight is None else _fit(q_weight, "q_weight", torch.bfloat16, (D,), at),
          0 if k_weight is None else _fit(k_weight, "k_weight", torch.bfloat16, (D,), at),
          0 if positions is None else _fit(positions, "positions", torch.int32, (B, L) if dense else (L,), at),
          B, L, Hq, Hkv, D, eps, *strides, *r, _stream_of(stream, at))
    return q_out, k_out


_NO_ROPE = (0, 0, 0, ATTN_ROPE_NONE, 0)


def _out_rows(out, name, like, ndim, at):
    """The strides of an output shaped like `like` whose rows are written once each."""
    try:
        if out.dtype is torch.bfloat16 and out.shape == like.shape and out.get_device() == at and out.is_contiguous():
            return out.stride()
    except AttributeError:  # not a tensor: told below
        pass
    st = _rows(out, name, ndim, at)
    if out.shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(out.shape)}")
    _written_once(out, name)
    return st


def _pool_q4(pool, D=None):
    """Check a 4-bit cache pool, uint8 [num_pages,Hkv,page_size/16,18*D] -> num_pages, Hkv, page_size, D, device."""
    if not (isinstance(pool, torch.Tensor) and pool.dtype == torch.uint8 and pool.dim() == 4 and pool.is_cuda
            and pool.is_contiguous()):
        _need(pool, "pool", torch.uint8, 4)
    num_pages, Hkv, tiles, tile = pool.shape
    if tile not in (18 * 64, 18 * 128) or (D is not None and tile != 18 * D):
        raise ValueError(f"pool tiles must have 18 * D bytes, got {tile}")
    return num_pages, Hkv, 16 * tiles, tile // 18, pool.get_device()


def attn_kv_q4_pool(num_pages, Hkv, page_size, D, device="cuda"):
    """A new 4-bit cache pool, uint8 [num_pages,Hkv,page_size/16,18*D], all zeros."""
    if attn_kv_q4_page_bytes(page_size, Hkv, D) == 0:
        raise AttnError(ATTN_ERR_INVALID_ARG, "attn_kv_q4_pool")
    return torch.zeros((num_pages, Hkv, page_size // 16, 18 * D), dtype=torch.uint8, device=device)


def attn_kv_q4_page_bytes(page_size, Hkv, D) -> int:
    return int(load().attn_kv_q4_page_bytes(page_size, Hkv, D))


def attn_kv_append_q4(k, v, pool, slots, stream=None):
    """Quantise k and v [T,Hkv,D] bf16 (any strides over contiguous rows) into the 4-bit pool at slots int32 [T]
    (-1: not written; the others must differ)."""
    num_pages, Hkv, page_size, D, at = _pool_q4(pool)
    sk, sv = _rows(k, "k", 3, at), _rows(v, "v", 3, at)
    T = k.shape[0]
    if k.shape != (T, Hkv, D) or v.shape != k.shape:
        raise ValueError(f"k/v shapes {tuple(k.shape)} {tuple(v.shape)} do not match the pool {tuple(pool.shape)}")
    _call("attn_kv_append_q4", attn_kv_append_q4_params, at,
          k.data_ptr(), v.data_ptr(), pool.data_ptr(),
          _fit(slots, "slots", torch.int32, (T,), at), T, Hkv, D, page_size, num_pages,
          sk[0], sk[1], sv[0], sv[1], _stream_of(stream, at))


def attn_kv_gather_q4(pool, block_table, cu_k, total_k, kv_starts=None, k_out=None, v_out=None, stream=None):
    """Read rows of the 4-bit pool back as packed bf16 k and v [total_k,Hkv,D]: keys kv_starts[b] (default 0) and on of
    sequence b become rows cu_k[b] .. cu_k[b+1]-1 (cu_k int32 [B+1]); rows past cu_k[B] stay as they were.
    -> (k, v)"""
    num_pages, Hkv, page_size, D, at = _pool_q4(pool)
    i32 = torch.int32
    B, width = block_table.shape if isinstance(block_table, torch.Tensor) and block_table.dim() == 2 else (0, 0)
    shape = (int(total_k), Hkv, D)
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=pool.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=torch.bfloat16, device=pool.device)
    _call("attn_kv_gather_q4", attn_kv_gather_q4_params, at,
          pool.data_ptr(), _fit(block_table, "block_table", i32, (B, width), at), _fit(cu_k, "cu_k", i32, (B + 1,), at),
          0 if kv_starts is None else _fit(kv_starts, "kv_starts", i32, (B,), at),
          _fit(k_out, "k_out", torch.bfloat16, shape, at), _fit(v_out, "v_out", torch.bfloat16, shape, at),
          B, Hkv, D, page_size, width, num_pages, shape[0], _stream_of(stream, at))
    return k_out, v_out


def attn_decode_q4(q, pool, block_table, kv_lens, out=None, lse=None, scale=None, chunk=0, out_dtype=torch.bfloat16,
                   want_lse=True, workspace=None, stream=None):
    """Decode over the 4-bit pool: q [B,Hq,D], or [B,Hq,Lq,D] for Lq new tokens, bf16 (already rotated); block_table
    int32 [B,max_pages], kv_lens int32 [B] counting the new tokens' own keys.  ``workspace`` is a buffer from
    attn_decode_q4_workspace; without one the library's is used, as by attn_decode.  -> (out, lse) shaped like q"""
    many = isinstance(q, torch.Tensor) and q.dim() == 4
    _need(q, "q", torch.bfloat16, 4 if many else 3)
    qs = q.shape
    B, Hq, D = qs[0], qs[1], qs[-1]
    num_pages, Hkv, page_size, _, at = _pool_q4(pool, D)
    if q.get_device() != at:
        raise ValueError(f"q must be on cuda:{at}, got {q.device}")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be bf16 or fp32")
    width = block_table.shape[-1] if isinstance(block_table, torch.Tensor) and block_table.dim() else 0
    if out is None:
        out = torch.empty(qs, dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(qs[:-1], dtype=torch.float32, device=q.device)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1, device=q.device)
    _call("attn_decode_q4", attn_decode_q4_params, at,
          q.data_ptr(), pool.data_ptr(), _fit(block_table, "block_table", torch.int32, (B, width), at),
          _fit(kv_lens, "kv_lens", torch.int32, (B,), at), _fit(out, "out", out_dtype, qs, at),
          0 if lse is None else _fit(lse, "lse", torch.float32, qs[:-1], at),
          B, Hq, Hkv, qs[2] if many else 1, D, page_size, width, num_pages,
          1.0 / math.sqrt(D) if scale is None else scale,
          ATTN_DTYPE_F32 if out_dtype == torch.float32 else ATTN_DTYPE_BF16, int(chunk),
          0 if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.shape[0],
          _stream_of(stream, at))
    return out, lse


def attn_decode_q4_workspace_bytes(Hq, Hkv, Lq, D) -> int:
    return int(load().attn_decode_q4_workspace_bytes(Hq, Hkv, Lq, D))


def attn_decode_q4_workspace(Hq, Hkv, D, Lq=1, device="cuda"):
    """A workspace of attn_decode_q4 of one's own (uint8, zeroed), for calls or captured graphs that may overlap others
    on the GPU."""
    device = torch.device(device)
    with torch.cuda.device(device):
        n = attn_decode_q4_workspace_bytes(Hq, Hkv, Lq, D)
        if n == 0:
            raise AttnError(ATTN_ERR_INVALID_ARG, "attn_decode_q4_workspace")
        return torch.zeros(n, dtype=torch.uint8, device=device)


_SCALINGS = {"linear": (ATTN_ROPE_SCALE_LINEAR, 1), "base": (ATTN_ROPE_SCALE_BASE, 1), "turns": (ATTN_ROPE_SCALE_TURNS, 4),
             "index": (ATTN_ROPE_SCALE_INDEX, 4)}


def attn_rope_tables(rows, rotary_dim, base=10000.0, scaling=None, amplitude=1.0, start=0, cos=None, sin=None,
                     device="cuda", stream=None):
    """Rotary tables, fp32 [rows, rotary_dim/2] of positions start and on: amplitude times cos and sin of position times
    base^(-2i/rotary_dim), scaled for long contexts by ``scaling``: ("linear", factor), ("base", factor),
    ("turns", factor, context, low, high) or ("index", factor, context, low, high).  -> (cos, sin), what ``rope`` takes"""
    kind, numbers = ATTN_ROPE_SCALE_NONE, ()
    if scaling is not None:
        if scaling[0] not in _SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling[0]!r}")
        kind, count = _SCALINGS[scaling[0]]
        numbers = tuple(scaling[1:])
        if len(numbers) != count:
            raise ValueError(f"scaling {scaling[0]!r} takes {count} numbers, got {len(numbers)}")
    rows, rotary_dim, start = int(rows), int(rotary_dim), int(start)
    if rows < 0 or rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rope tables of {rows} rows and {rotary_dim} dims")
    shape = (rows, rotary_dim // 2)
    if cos is None:
        cos = torch.empty(shape, dtype=torch.float32, device=device if sin is None else sin.device)
    if sin is None:
        sin = torch.empty(shape, dtype=torch.float32, device=cos.device)
    at = cos.get_device() if isinstance(cos, torch.Tensor) else -1
    _call("attn_rope_tables", attn_rope_tables_params, at,
          _fit(cos, "cos", torch.float32, shape, at), _fit(sin, "sin", torch.float32, shape, at),
          rows, start, rotary_dim, kind, base, *(numbers + (1.0,) * (4 - len(numbers))), amplitude,
          _stream_of(stream, at))
    return cos, sin


def attn_kv_append_paged(k, v, kpages, vpages, slots, rope=None, positions=None, q=None, q_out=None, k_out=None,
                         want_k=False, stream=None):
    """Rows k and v [T,Hkv,D] bf16 (any strides over contiguous rows) into the pages [num_pages,Hkv,page_size,D] at slots
    int32 [T] (-1: not written; the others must differ), k rotated by rope = (cos, sin, style) with tables
    [max_pos, R/2], R <= D, at positions int32 [T] (-1: a padded token, left out), and q [T,Hq,D], where given, rotated
    alike.  k_out (made where ``want_k``) takes the rotated k packed.  q_out/k_out may be q/k themselves.
    -> (q_out, k_out)"""
    sk, at = _rows(k, "k", 3), k.get_device()
    shape = k.shape
    sv = _rows(v, "v", 3, at)
    T, Hkv, D = shape
    if v.shape != shape:
        raise ValueError(f"k/v shapes {tuple(shape)} {tuple(v.shape)} differ")
    pool = _pool_pages(kpages, Hkv, D)
    R = Hq = qp = qop = kop = 0
    sq = sqo = sko = (0, 0)
    r = _NO_ROPE
    if rope is None:
        if q is not None or q_out is not None or k_out is not None or want_k:
            raise ValueError("q and k_out go with a rotation")
    else:
        cos, sin, style = rope if len(rope) == 3 else _rope3(rope)
        try:
            max_pos, pairs = tab = cos.shape
        except (AttributeError, ValueError):
            raise ValueError("rope tables must be tensors [max_pos, R/2]") from None
        if max_pos == 0 or pairs == 0:
            raise ValueError("rope tables must have rows")
        if style not in _ROPE_STYLES:
            raise ValueError("rope style must be 'half' or 'interleaved'")
        R = 2 * pairs
        r = (_fit(cos, "rope cos", torch.float32, tab, at), _fit(sin, "rope sin", torch.float32, tab, at), max_pos,
             _ROPE_STYLES[style], 0)
        if q is not None:
            sq = _rows(q, "q", 3, at)
            Hq = q.shape[1]
            if q.shape != (T, Hq, D) or Hq == 0:
                raise ValueError(f"q shape {tuple(q.shape)} does not match k {tuple(shape)}")
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
            sqo = _out_rows(q_out, "q_out", q, 3, at)
            qp, qop = q.data_ptr(), q_out.data_ptr()
        elif q_out is not None:
            raise ValueError("q_out goes with q")
        if k_out is None and want_k:
            k_out = torch.empty(shape, dtype=torch.bfloat16, device=k.device)
        if k_out is not None:
            sko = _out_rows(k_out, "k_out", k, 3, at)
            kop = k_out.data_ptr()
    _call("attn_kv_append_paged", attn_kv_append_paged_params, at,
          k.data_ptr(), v.data_ptr(), _fit(kpages, "kpages", torch.bfloat16, pool, at),
          _fit(vpages, "vpages", torch.bfloat16, pool, at), _fit(slots, "slots", torch.int32, (T,), at),
          0 if positions is None else _fit(positions, "positions", torch.int32, (T,), at), qp, qop, kop,
          T, Hq, Hkv, D, pool[2], pool[0], R,
          sk[0], sk[1], sv[0], sv[1], sq[0], sq[1], sqo[0], sqo[1], sko[0], sko[1], *r, _stream_of(stream, at))
    return q_out, k_out


def _rope3(rope):
    if len(rope) > 3 and rope[3] is not None:
        raise ValueError("rope k_out is taken by prefill calls only")
    return rope[:3]


def _pool_pages(pages, Hkv, D):
    """The shape of a pool [num_pages,Hkv,page_size,D] (Hkv, D where they are given)."""
    try:
        n, heads, size, dim = pages.shape
    except (AttributeError, ValueError):
        raise ValueError("kpages must be a tensor [num_pages,Hkv,page_size,D]") from None
    return n, heads if Hkv is None else Hkv, size, dim if D is None else D


def attn_decode_multi_paged(q, kpages, vpages, block_table, kv_lens, cu_new, max_new, out=None, lse=None, scale=None,
                            out_dtype=torch.bfloat16, want_lse=True, workspace=None, stream=None):
    """Decode of several new tokens of each sequence over pages [num_pages,Hkv,page_size,D] bf16: q [T,Hq,D] bf16 (already
    rotated), packed by cu_new int32 [B+1] with at most max_new tokens a sequence; block_table int32 [B,max_pages],
    kv_lens int32 [B] counting the new tokens' own keys.  ``workspace`` is a buffer from
    attn_decode_multi_paged_workspace; without one the library's is used.  Rows of no sequence stay as they were.
    -> (out [T,Hq,D], lse [T,Hq])"""
    _need(q, "q", torch.bfloat16, 3)
    at = q.get_device()
    T, Hq, D = shape = q.shape
    num_pages, Hkv, page_size, _ = pool = _pool_pages(kpages, None, D)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be bf16 or fp32")
    try:
        B, width = block_table.shape
    except (AttributeError, ValueError):
        raise ValueError("block_table must be a tensor [B,max_pages]") from None
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1, device=q.device)
    i32 = torch.int32
    _call("attn_decode_multi_paged", attn_decode_multi_paged_params, at,
          q.data_ptr(), _fit(kpages, "kpages", torch.bfloat16, pool, at),
          _fit(vpages, "vpages", torch.bfloat16, pool, at), _fit(block_table, "block_table", i32, (B, width), at),
          _fit(kv_lens, "kv_lens", i32, (B,), at), _fit(cu_new, "cu_new", i32, (B + 1,), at),
          _fit(out, "out", out_dtype, shape, at), 0 if lse is None else _fit(lse, "lse", torch.float32, (T, Hq), at),
          B, T, Hq, Hkv, D, int(max_new), page_size, width, num_pages, 1.0 / math.sqrt(D) if scale is None else scale,
          ATTN_DTYPE_F32 if out_dtype == torch.float32 else ATTN_DTYPE_BF16,
          0 if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.shape[0],
          _stream_of(stream, at))
    return out, lse


def attn_decode_multi_paged_workspace_bytes(Hq, Hkv, max_new, D) -> int:
    return int(load().attn_decode_multi_paged_workspace_bytes(Hq, Hkv, max_new, D))


def attn_decode_multi_paged_workspace(Hq, Hkv, D, max_new, device="cuda"):
    """A workspace of attn_decode_multi_paged of one's own (uint8, zeroed), for calls or captured graphs that may overlap
    others on the GPU."""
    device = torch.device(device)
    with torch.cuda.device(device):
        n = attn_decode_multi_paged_workspace_bytes(Hq, Hkv, max_new, D)
        if n == 0:
            raise AttnError(ATTN_ERR_INVALID_ARG, "attn_decode_multi_paged_workspace")
        return torch.zeros(n, dtype=torch.uint8, device=device)


def _prob_rows(t, name, dtype, shape, at):
    """The strides of a tensor of probabilities whose rows (the last axis) are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != at or at < 0:
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on cuda:{at}" if at >= 0 else ""))
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the probabilities of a row must be contiguous")
    return st


def attn_verify_drafts(draft_tokens, target_probs, uniforms, draft_probs=None, cu_target=None, draft_lens=None,
                       kv_lens=None, tokens=None, accepted=None, keep_lens=None, stream=None):
    """Which of the drafts [B,K] int32 stand, and the token that follows them.  target_probs, bf16 or fp32: [total,V]
    packed by cu_target int32 [B+1] (a sequence's drafts and one more row), or [B,K+1,V] with draft_lens int32 [B]
    (default K); draft_probs [B,K,V] of the same type, or None for drafts that were not drawn; uniforms fp32 [B,K+1] in
    [0, 1).  tokens [B,K+1] become the standing drafts, the next token, then -1; accepted [B] their number; keep_lens
    [B], where kv_lens [B] is given, what attn_page_step keeps.  -> (tokens, accepted, keep_lens)"""
    i32 = torch.int32
    _need(draft_tokens, "draft_tokens", i32, 2)
    at = draft_tokens.get_device()
    B, K = draft_tokens.shape
    dtype = target_probs.dtype if isinstance(target_probs, torch.Tensor) else None
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("target_probs must be a bf16 or fp32 tensor")
    if target_probs.dim() == 0:
        raise ValueError("target_probs must have rows")
    V = target_probs.shape[-1]
    if cu_target is not None:
        if draft_lens is not None:
            raise ValueError("draft_lens goes without cu_target")
        total = target_probs.shape[0]
        ts = (0, _prob_rows(target_probs, "target_probs", dtype, (total, V), at)[0])
    else:
        total = 0
        ts = _prob_rows(target_probs, "target_probs", dtype, (B, K + 1, V), at)[:2]
    ds = (0, 0) if draft_probs is None else _prob_rows(draft_probs, "draft_probs", dtype, (B, K, V), at)[:2]
    if tokens is None:
        tokens = torch.empty((B, K + 1), dtype=i32, device=draft_tokens.device)
    if accepted is None:
        accepted = torch.empty((B,), dtype=i32, device=draft_tokens.device)
    if keep_lens is None and kv_lens is not None:
        keep_lens = torch.empty((B,), dtype=i32, device=draft_tokens.device)
    if keep_lens is not None and kv_lens is None:
        raise ValueError("keep_lens goes with kv_lens")
    _call("attn_verify_drafts", attn_verify_drafts_params, at,
          draft_tokens.data_ptr(), target_probs.data_ptr(), 0 if draft_probs is None else draft_probs.data_ptr(),
          _fit(uniforms, "uniforms", torch.float32, (B, K + 1), at),
          0 if cu_target is None else _fit(cu_target, "cu_target", i32, (B + 1,), at),
          0 if draft_lens is None else _fit(draft_lens, "draft_lens", i32, (B,), at),
          0 if kv_lens is None else _fit(kv_lens, "kv_lens", i32, (B,), at),
          _fit(tokens, "tokens", i32, (B, K + 1), at), _fit(accepted, "accepted", i32, (B,), at),
          0 if keep_lens is None else _fit(keep_lens, "keep_lens", i32, (B,), at),
          B, K, V, total, ATTN_DTYPE_F32 if dtype == torch.float32 else ATTN_DTYPE_BF16, *ts, *ds,
          _stream_of(stream, at))
    return tokens, accepted, keep_lens


def attn_decode_workspace_bytes(B, Hq, Hkv, Lmax, D, chunk=0) -> int:
    return int(load().attn_decode_workspace_bytes(B, Hq, Hkv, Lmax, D, chunk))


def attn_get_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    h = None if stream is None else ctypes.c_void_p(stream.cuda_stream)
    return int(load().attn_get_device_status(h))


def attn_release_workspace():
    load().attn_release_workspace()


def attn_version() -> int:
    return int(load().attn_version())


def attn_selftest_wait_timeout(limit_us=1000, stream=None):
    """Run the bounded-wait timeout path on the current device (no fault): afterwards the device status word
    holds ATTN_ERR_DEVICE_TIMEOUT."""
    dev = torch.device("cuda", torch.cuda.current_device())
    _check(load().attn_selftest_wait_timeout(int(limit_us), _stream_handle(stream, dev)), "attn_selftest_wait_timeout")
