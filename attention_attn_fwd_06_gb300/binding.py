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


class attn_qk_norm_rope_params(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("B", ctypes.c_int), ("L", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("eps", ctypes.c_float),
        ("q_stride", ctypes.c_longlong * 3), ("k_stride", ctypes.c_longlong * 3),
        ("q_out_stride", ctypes.c_longlong * 3), ("k_out_stride", ctypes.c_longlong * 3),
        ("rope", attn_rope),
        ("stream", ctypes.c_void_p),
    ]


class attn_kv_append_q4_params(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pool", ctypes.c_void_p), ("slots", ctypes.c_void_p),
        ("T", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int), ("page_size", ctypes.c_int),
        ("num_pages", ctypes.c_int),
        ("k_stride", ctypes.c_longlong * 2), ("v_stride", ctypes.c_longlong * 2),
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


_lib = None
_lock = threading.Lock()


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library once (raises if it has not been built)."""
    global _lib
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
    style "half" or "interleaved"); every call of this module takes the same argument."""
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


def _call(fn, p, device, stream, where):
    """Run one entry point on `device` (made current for the call) and its stream."""
    p.stream = (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream
    if device.index == torch.cuda.current_device():
        status = fn(ctypes.byref(p))
    else:
        with torch.cuda.device(device):
            status = fn(ctypes.byref(p))
    if status != ATTN_OK:
        raise AttnError(status, where)


def _rows(t, name, ndim, device):
    """A bf16 tensor whose rows (the last axis) are contiguous; the other axes may have any stride that is a multiple
    of 8 elements.  Returns its strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on {device}" if device is not None else ""))
    st = t.stride()
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
    _need(kv_lens, "kv_lens", torch.int32, 1)
    dev = kv_lens.device
    B = kv_lens.shape[0]
    _need(block_table, "block_table", torch.int32, 2, device=dev)
    if block_table.shape[0] != B:
        raise ValueError("block_table must have B rows")
    _need(free_pages, "free_pages", torch.int32, 1, device=dev)
    _need(free_count, "free_count", torch.int32, 1, (1,), dev)
    p = attn_page_step_params()
    p.max_tokens = -1
    for t, name, shape in ((new_lens, "new_lens", (B,)), (keep_lens, "keep_lens", (B,)), (cu_new, "cu_new", (B + 1,)),
                           (slots, "slots", None), (positions, "positions", None)):
        if t is None:
            continue
        _need(t, name, torch.int32, 1, shape, dev)
        setattr(p, name, t.data_ptr())
        if shape is None:
            if p.max_tokens not in (-1, t.shape[0]):
                raise ValueError("slots and positions must have the same length")
            p.max_tokens = t.shape[0]
    p.max_tokens = max(p.max_tokens, 0)
    p.kv_lens, p.block_table = kv_lens.data_ptr(), block_table.data_ptr()
    p.free_pages, p.free_count = free_pages.data_ptr(), free_count.data_ptr()
    p.B, p.page_size, p.max_pages, p.num_pages = B, int(page_size), block_table.shape[1], free_pages.shape[0]
    _call(load().attn_page_step, p, dev, stream, "attn_page_step")
    return slots, positions, cu_new


def attn_qk_norm_rope(q, k, q_weight=None, k_weight=None, rope=None, positions=None, eps=1e-6, q_out=None, k_out=None,
                      stream=None):
    """RMS norm of every q and k head and its rotation, in one pass: q [T,Hq,D] and k [T,Hkv,D] (packed), or
    [B,H,L,D] (dense), bf16 with any strides over contiguous rows (k may be None); weights bf16 [D] or None;
    rope = (cos, sin, style); positions int32 [T] or [B,L], -1 for padded rows, which are left as they were.
    q_out/k_out may be q/k themselves.  -> (q_out, k_out)"""
    dense = isinstance(q, torch.Tensor) and q.dim() == 4
    _rows(q, "q", 4 if dense else 3, None)
    p = attn_qk_norm_rope_params()
    dev = q.device
    shapes = []
    for x, out, w, name in ((q, q_out, q_weight, "q"), (k, k_out, k_weight, "k")):
        if x is None:
            if name == "q" or out is not None or w is not None:
                raise ValueError("q is needed; k_out and k_weight go with k")
            shapes.append(None)
            continue
        st = _rows(x, name, 4 if dense else 3, dev)
        if out is None:
            out = torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
        elif out is not x:
            _rows(out, name + "_out", 4 if dense else 3, dev)
            if out.shape != x.shape:
                raise ValueError(f"{name}_out must have shape {tuple(x.shape)}, got {tuple(out.shape)}")
        if not out.is_contiguous():
            _written_once(out, name + "_out")
        if w is not None:
            _need(w, name + "_weight", torch.bfloat16, 1, (x.shape[-1],), dev)
            setattr(p, name + "_weight", w.data_ptr())
        so = out.stride()
        setattr(p, name, x.data_ptr())
        setattr(p, name + "_out", out.data_ptr())
        # sequence, token, head
        setattr(p, name + "_stride", (st[0], st[2], st[1]) if dense else (0, st[0], st[1]))
        setattr(p, name + "_out_stride", (so[0], so[2], so[1]) if dense else (0, so[0], so[1]))
        shapes.append(x.shape)
        if name == "q":
            q_out = out
        else:
            k_out = out
    sq, sk = shapes
    if dense:
        p.B, p.Hq, p.L, p.D = sq
        if sk is not None and (sk[0], sk[2], sk[3]) != (sq[0], sq[2], sq[3]):
            raise ValueError(f"k shape {tuple(sk)} does not match q {tuple(sq)}")
    else:
        p.B, (p.L, p.Hq, p.D) = 1, sq
        if sk is not None and (sk[0], sk[2]) != (sq[0], sq[2]):
            raise ValueError(f"k shape {tuple(sk)} does not match q {tuple(sq)}")
    p.Hkv = 0 if sk is None else sk[1]
    p.eps = float(eps)
    if positions is not None:
        _need(positions, "positions", torch.int32, 2 if dense else 1, (p.B, p.L) if dense else (p.L,), dev)
        p.positions = positions.data_ptr()
    if rope is not None and len(rope) > 3:
        raise ValueError("rope k_out is taken by prefill calls only")
    _set_rope(p, rope, p.D, dev)
    _call(load().attn_qk_norm_rope, p, dev, stream, "attn_qk_norm_rope")
    return q_out, k_out


def _pool_q4(pool, p, device, D=None):
    """Check a 4-bit cache pool, uint8 [num_pages,Hkv,page_size/16,18*D], and note its sizes."""
    _need(pool, "pool", torch.uint8, 4, device=device)
    num_pages, Hkv, tiles, tile = pool.shape
    if tile not in (18 * 64, 18 * 128) or (D is not None and tile != 18 * D):
        raise ValueError(f"pool tiles must have 18 * D bytes, got {tile}")
    p.pool = pool.data_ptr()
    p.num_pages, p.Hkv, p.page_size, p.D = num_pages, Hkv, 16 * tiles, tile // 18


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
    p = attn_kv_append_q4_params()
    sk = _rows(k, "k", 3, None)
    dev = k.device
    sv = _rows(v, "v", 3, dev)
    _pool_q4(pool, p, dev)
    T = k.shape[0]
    if tuple(k.shape) != (T, p.Hkv, p.D) or v.shape != k.shape:
        raise ValueError(f"k/v shapes {tuple(k.shape)} {tuple(v.shape)} do not match the pool {tuple(pool.shape)}")
    _need(slots, "slots", torch.int32, 1, (T,), dev)
    p.k, p.v, p.slots, p.T = k.data_ptr(), v.data_ptr(), slots.data_ptr(), T
    p.k_stride, p.v_stride = sk[:2], sv[:2]
    _call(load().attn_kv_append_q4, p, dev, stream, "attn_kv_append_q4")


def attn_kv_gather_q4(pool, block_table, cu_k, total_k, kv_starts=None, k_out=None, v_out=None, stream=None):
    """Read rows of the 4-bit pool back as packed bf16 k and v [total_k,Hkv,D]: keys kv_starts[b] (default 0) and on of
    sequence b become rows cu_k[b] .. cu_k[b+1]-1 (cu_k int32 [B+1]); rows past cu_k[B] stay as they were.
    -> (k, v)"""
    p = attn_kv_gather_q4_params()
    _pool_q4(pool, p, None)
    dev = pool.device
    _need(block_table, "block_table", torch.int32, 2, device=dev)
    B = block_table.shape[0]
    _need(cu_k, "cu_k", torch.int32, 1, (B + 1,), dev)
    if kv_starts is not None:
        _need(kv_starts, "kv_starts", torch.int32, 1, (B,), dev)
        p.kv_starts = kv_starts.data_ptr()
    shape = (int(total_k), p.Hkv, p.D)
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if v_out is None:
        v_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    _need(k_out, "k_out", torch.bfloat16, 3, shape, dev)
    _need(v_out, "v_out", torch.bfloat16, 3, shape, dev)
    p.block_table, p.cu_k, p.k, p.v = block_table.data_ptr(), cu_k.data_ptr(), k_out.data_ptr(), v_out.data_ptr()
    p.B, p.max_pages, p.total_k = B, block_table.shape[1], shape[0]
    _call(load().attn_kv_gather_q4, p, dev, stream, "attn_kv_gather_q4")
    return k_out, v_out


def attn_decode_q4(q, pool, block_table, kv_lens, out=None, lse=None, scale=None, chunk=0, out_dtype=torch.bfloat16,
                   want_lse=True, workspace=None, stream=None):
    """Decode over the 4-bit pool: q [B,Hq,D], or [B,Hq,Lq,D] for Lq new tokens, bf16 (already rotated); block_table
    int32 [B,max_pages], kv_lens int32 [B] counting the new tokens' own keys.  ``workspace`` is a buffer from
    attn_decode_q4_workspace; without one the library's is used, as by attn_decode.  -> (out, lse) shaped like q"""
    _need(q, "q", torch.bfloat16, 4 if isinstance(q, torch.Tensor) and q.dim() == 4 else 3)
    dev = q.device
    p = attn_decode_q4_params()
    B, Hq, D = q.shape[0], q.shape[1], q.shape[-1]
    Lq = q.shape[2] if q.dim() == 4 else 1
    _pool_q4(pool, p, dev, D)
    _need(block_table, "block_table", torch.int32, 2, device=dev)
    _need(kv_lens, "kv_lens", torch.int32, 1, (B,), dev)
    if block_table.shape[0] != B:
        raise ValueError("block_table must have B rows")
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=dev)
    else:
        _need(out, "out", out_dtype, q.dim(), q.shape, dev)
    if lse is None and want_lse:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev)
    elif lse is not None:
        _need(lse, "lse", torch.float32, q.dim() - 1, q.shape[:-1], dev)
    if lse is not None:
        p.lse = lse.data_ptr()
    p.q, p.block_table, p.kv_lens, p.out = q.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr(), out.data_ptr()
    p.B, p.Hq, p.Lq, p.max_pages = B, Hq, Lq, block_table.shape[1]
    p.scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be bf16 or fp32")
    p.out_dtype = ATTN_DTYPE_F32 if out_dtype == torch.float32 else ATTN_DTYPE_BF16
    p.chunk = int(chunk)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1, device=dev)
        p.workspace, p.workspace_bytes = workspace.data_ptr(), workspace.shape[0]
    _call(load().attn_decode_q4, p, dev, stream, "attn_decode_q4")
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
