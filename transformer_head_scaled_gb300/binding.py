"""ctypes binding of the C ABI in ``include/attn.h``.

Argument marshalling only: every step of the attention runs in the CUDA
library.  PyTorch is used for device buffers and streams.  The library must
have been built (``transformer_head_scaled_gb300.build.build()``); if it is
missing, :func:`load` raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

from .inputs import MASK_CAUSAL, MASK_KEY_PADDING, MASK_NONE  # noqa: F401

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build",
                        "libattn_gb300.so")

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = -1
ATTN_ERR_UNSUPPORTED = -2
ATTN_ERR_CUDA = -3
ATTN_ERR_TIMEOUT = -4
ATTN_ERR_SCRATCH_TOO_SMALL = -5
ATTN_ERR_WRONG_PLAN = -6
MASK_WINDOW = 3  # attn_fwd_strided: the window of attn_fwd_window
CACHE_BF16, CACHE_E4M3, CACHE_INT8 = 0, 1, 2  # attn_cache_format
_CACHE_FORMATS = {torch.bfloat16: CACHE_BF16, torch.float8_e4m3fn: CACHE_E4M3,
                  torch.int8: CACHE_INT8}
DECODE_NOALLOC_SCRATCH_BYTES = 1 << 20

# Every entry point declared in include/attn.h.
EXPORTS = ("attn_fwd", "attn_fwd_f32", "attn_fwd_window", "attn_fwd_strided", "attn_fwd_host",
           "attn_fwd_host_buffer_bytes", "attn_decode", "attn_decode_strided",
           "attn_decode_workspace_bytes", "attn_decode_window",
           "attn_decode_window_workspace_bytes", "attn_decode_noalloc", "attn_bwd", "attn_bwd_window", "attn_bwd_strided",
           "attn_bwd_workspace_bytes", "attn_cache_append", "attn_decode_scored",
           "attn_decode_scored_workspace_bytes", "attn_mask_plan", "attn_mask_plan_bytes",
           "attn_fwd_scored", "attn_bwd_scored", "attn_bwd_scored_workspace_bytes",
           "attn_check", "attn_status_string",
           "attn_last_cuda_error", "attn_set_wait_limit_ns", "attn_launch_count",
           "attn_diag_tile", "attn_diag_wait_timeout")

_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {status_string(status)} ({status})"
        if status == ATTN_ERR_CUDA and _lib is not None:
            msg += f", cudaError {_lib.attn_last_cuda_error()}"
        super().__init__(msg)


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (once) and declare the signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"CUDA library {path} is missing: build it with "
                "transformer_head_scaled_gb300.build.build()")
        lib = ctypes.CDLL(path)
        vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        for name in ("attn_fwd", "attn_fwd_f32"):
            fn = getattr(lib, name)
            fn.restype = i32
            fn.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp, vp]
        lib.attn_fwd_window.restype = i32
        lib.attn_fwd_window.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, i32,
                                        vp]
        lib.attn_fwd_strided.restype = i32
        lib.attn_fwd_strided.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp,
                                         vp, f32, i32, vp, i32, i32, vp]
        lib.attn_decode.restype = i32
        lib.attn_decode.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, vp,
                                    ctypes.c_size_t, vp]
        lib.attn_decode_noalloc.restype = i32
        lib.attn_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp,
                                            vp]
        lib.attn_decode_workspace_bytes.restype = ctypes.c_size_t
        lib.attn_decode_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        lib.attn_decode_window.restype = i32
        lib.attn_decode_window.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp,
                                           i32, vp, ctypes.c_size_t, vp]
        lib.attn_decode_window_workspace_bytes.restype = ctypes.c_size_t
        lib.attn_decode_window_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.attn_bwd.restype = i32
        lib.attn_bwd.argtypes = [vp] * 9 + [i32] * 5 + [f32, i32, vp, vp, ctypes.c_size_t, vp]
        lib.attn_decode_strided.restype = i32
        lib.attn_decode_strided.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, f32,
                                            vp, vp, ctypes.c_size_t, vp]
        lib.attn_fwd_host.restype = i32
        lib.attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp,
                                      i32, i32, vp, ctypes.c_size_t, vp]
        lib.attn_fwd_host_buffer_bytes.restype = ctypes.c_size_t
        lib.attn_fwd_host_buffer_bytes.argtypes = [i32, i32, i32, i32, i32]
        lib.attn_bwd_strided.restype = i32
        lib.attn_bwd_strided.argtypes = [vp] * 9 + [i32] * 5 + [vp, f32, i32, vp, i32, i32, vp,
                                                                 ctypes.c_size_t, vp]
        lib.attn_bwd_window.restype = i32
        lib.attn_bwd_window.argtypes = [vp] * 9 + [i32] * 5 + [f32, i32, i32, vp, ctypes.c_size_t,
                                                                vp]
        lib.attn_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.attn_bwd_workspace_bytes.argtypes = [i32, i32, i32, i32]
        lib.attn_cache_append.restype = i32
        lib.attn_cache_append.argtypes = [vp] * 6 + [i32] * 5 + [vp, i32, i32, vp, vp, vp]
        lib.attn_decode_scored.restype = i32
        lib.attn_decode_scored.argtypes = ([vp] * 7 + [i32] * 6 + [vp, i32, i32, f32, f32, vp, vp,
                                                                   i32, vp, ctypes.c_size_t, vp])
        lib.attn_decode_scored_workspace_bytes.restype = ctypes.c_size_t
        lib.attn_decode_scored_workspace_bytes.argtypes = [i32] * 8
        lib.attn_mask_plan.restype = i32
        lib.attn_mask_plan.argtypes = [i32] * 5 + [vp] * 4 + [ctypes.c_size_t, vp]
        lib.attn_mask_plan_bytes.restype = ctypes.c_size_t
        lib.attn_mask_plan_bytes.argtypes = [i32] * 3
        lib.attn_fwd_scored.restype = i32
        lib.attn_fwd_scored.argtypes = [vp] * 5 + [i32] * 6 + [vp, f32, f32, vp, vp,
                                                               ctypes.c_size_t, vp]
        lib.attn_bwd_scored.restype = i32
        lib.attn_bwd_scored.argtypes = [vp] * 9 + [i32] * 6 + [vp, f32, f32, vp, vp,
                                                               ctypes.c_size_t, vp,
                                                               ctypes.c_size_t, vp]
        lib.attn_bwd_scored_workspace_bytes.restype = ctypes.c_size_t
        lib.attn_bwd_scored_workspace_bytes.argtypes = [i32] * 6
        lib.attn_check.restype = i32
        lib.attn_check.argtypes = [vp]
        lib.attn_status_string.restype = ctypes.c_char_p
        lib.attn_status_string.argtypes = [i32]
        lib.attn_last_cuda_error.restype = i32
        lib.attn_last_cuda_error.argtypes = []
        lib.attn_set_wait_limit_ns.restype = ctypes.c_uint64
        lib.attn_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        lib.attn_launch_count.restype = ctypes.c_uint64
        lib.attn_launch_count.argtypes = []
        lib.attn_diag_tile.restype = i32
        lib.attn_diag_tile.argtypes = [vp, vp, vp, vp, vp, vp, vp]
        lib.attn_diag_wait_timeout.restype = i32
        lib.attn_diag_wait_timeout.argtypes = [ctypes.c_uint64, vp]
        _lib = lib
        return lib


def status_string(status: int) -> str:
    if _lib is None:
        return str(status)
    return _lib.attn_status_string(int(status)).decode()


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


def attn_fwd_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, n_k, d_k, scale, mask_kind,
                 key_lens_ptr, stream_ptr, f32: bool = False) -> int:
    """The C call itself, on raw device pointers; returns the status code."""
    lib = load()
    fn = lib.attn_fwd_f32 if f32 else lib.attn_fwd
    return fn(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, n_k, d_k, float(scale),
              mask_kind, key_lens_ptr, stream_ptr)


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None,
             mask: int = MASK_NONE, key_lens: torch.Tensor | None = None,
             out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
             with_lse: bool = True, stream=None):
    """O = softmax(Q K^T * scale + M) V on the GPU, q/k/v [B, h, n, d] CUDA tensors.

    bf16 inputs run on the tensor cores (d = 64), float32 inputs on the CUDA
    cores.  scale defaults to 1/sqrt(d).  Returns (o, lse); lse is None when
    with_lse is False and no lse buffer is given.
    """
    if not (q.is_cuda and k.is_cuda and v.is_cuda):
        raise ValueError("q, k, v must be CUDA tensors")
    if q.dtype != k.dtype or q.dtype != v.dtype or q.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("q, k, v must all be bfloat16 or all float32")
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, h, n, d]")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous")
    B, h, n_q, d = q.shape
    n_k = k.shape[2]
    if tuple(k.shape) != (B, h, n_k, d) or tuple(v.shape) != (B, h, n_k, d):
        raise ValueError("k and v must be [B, h, n_k, d] with q's B, h, d")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    kl = None
    if mask == MASK_KEY_PADDING:
        if key_lens is None:
            raise ValueError("key padding needs key_lens")
        kl = key_lens
        if kl.dtype != torch.int32 or not kl.is_cuda or kl.numel() != B or not kl.is_contiguous():
            raise ValueError("key_lens must be a contiguous int32 CUDA tensor of B entries")
    if out is None:
        out = torch.empty((B, h, n_q, d), dtype=q.dtype, device=q.device)
    if lse is None and with_lse:
        lse = torch.empty((B, h, n_q), dtype=torch.float32, device=q.device)
    rc = attn_fwd_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, h, n_q, n_k, d, scale,
                      int(mask), _ptr(kl), _stream_ptr(stream), f32=q.dtype == torch.float32)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd")
    return out, lse


def attn_fwd_window_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, n_k, d_k, scale, left,
                       right, stream_ptr) -> int:
    """The C call itself, on raw device pointers; returns the status code."""
    return load().attn_fwd_window(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, n_k, d_k,
                                  float(scale), int(left), int(right), stream_ptr)


def attn_fwd_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, left: int, right: int,
                    scale: float | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, with_lse: bool = True, stream=None):
    """Restricted self-attention on the GPU: query i sees keys i-left .. i+right.

    q, k, v: contiguous bf16 CUDA [B, h, n, d] tensors, d in {16, 32, 64, 128}.
    Returns (o, lse).
    """
    for t in (q, k, v):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous bf16 CUDA [B, h, n, d] tensors")
    B, h, n_q, d = q.shape
    n_k = k.shape[2]
    if tuple(k.shape) != (B, h, n_k, d) or tuple(v.shape) != (B, h, n_k, d):
        raise ValueError("k and v must be [B, h, n_k, d] with q's B, h, d")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and with_lse:
        lse = torch.empty((B, h, n_q), dtype=torch.float32, device=q.device)
    rc = attn_fwd_window_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, h, n_q, n_k, d,
                             scale, left, right, _stream_ptr(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_window")
    return out, lse


def attn_fwd_strided_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, n_k, d_k, strides, scale,
                        mask_kind, lens_ptr, left, right, stream_ptr) -> int:
    """The C call itself; ``strides`` = four (b, h, n) element-stride triples for q, k, v, o."""
    arrs = [(ctypes.c_int64 * 3)(*[int(x) for x in st]) for st in strides]
    return load().attn_fwd_strided(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, n_k, d_k,
                                   *[ctypes.cast(a, ctypes.c_void_p) for a in arrs],
                                   float(scale), int(mask_kind), lens_ptr, int(left), int(right),
                                   stream_ptr)


def attn_fwd_strided(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None,
                     mask: int = MASK_NONE, key_lens: torch.Tensor | None = None,
                     window: tuple[int, int] | None = None, out: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, with_lse: bool = True, stream=None):
    """attn_fwd on [B, h, n, d] bf16 views with any strides over the first three
    dimensions and a contiguous last one (e.g. ``x.view(B, n, h, d).transpose(1, 2)``).
    ``window=(left, right)`` selects restricted self-attention; ``out`` may be a
    strided view too (default: contiguous)."""
    for t in (q, k, v):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or t.stride(-1) != 1:
            raise ValueError("q, k, v must be bf16 CUDA [B, h, n, d] views with unit last stride")
    B, h, n_q, d = q.shape
    n_k = k.shape[2]
    if tuple(k.shape) != (B, h, n_k, d) or tuple(v.shape) != (B, h, n_k, d):
        raise ValueError("k and v must be [B, h, n_k, d] with q's B, h, d")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    kl, left, right = None, 0, 0
    if window is not None:
        mask, (left, right) = MASK_WINDOW, window
    if mask == MASK_KEY_PADDING:
        if key_lens is None:
            raise ValueError("key padding needs key_lens")
        kl = key_lens
        if kl.dtype != torch.int32 or not kl.is_cuda or kl.numel() != B or not kl.is_contiguous():
            raise ValueError("key_lens must be a contiguous int32 CUDA tensor of B entries")
    if out is None:
        out = torch.empty((B, h, n_q, d), dtype=q.dtype, device=q.device)
    if tuple(out.shape) != (B, h, n_q, d) or out.stride(-1) != 1:
        raise ValueError("out must be a [B, h, n_q, d] view with unit last stride")
    if lse is None and with_lse:
        lse = torch.empty((B, h, n_q), dtype=torch.float32, device=q.device)
    strides = [t.stride()[:3] for t in (q, k, v, out)]
    rc = attn_fwd_strided_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, h, n_q, n_k, d,
                              strides, scale, int(mask), _ptr(kl), left, right,
                              _stream_ptr(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_strided")
    return out, lse


def host_buffer_bytes(B: int, h: int, n_q: int, n_k: int, d: int = 64) -> int:
    """Device staging bytes attn_fwd_host needs (0 for unsupported sizes)."""
    return int(load().attn_fwd_host_buffer_bytes(B, h, n_q, n_k, d))


def attn_fwd_host_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, n_k, d_k, scale, mask_kind,
                      lens_ptr, left, right, buf_ptr, buf_bytes, stream_ptr) -> int:
    """The C call itself (host q, k, v, o, lse, lens; device staging); returns the status."""
    return load().attn_fwd_host(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, n_k, d_k,
                                float(scale), int(mask_kind), lens_ptr, int(left), int(right),
                                buf_ptr, int(buf_bytes), stream_ptr)


def attn_fwd_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None,
                  mask: int = MASK_NONE, key_lens: torch.Tensor | None = None,
                  window: tuple[int, int] | None = None, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, with_lse: bool = True,
                  buf: torch.Tensor | None = None, device=None, stream=None):
    """attn_fwd on host (CPU) bf16 [B, h, n, d] tensors, pinned for asynchronous copies:
    copies in, forward and copies out pipelined over batch slices on the device.
    Returns host (o, lse); they are complete once ``stream`` has reached the call's
    end (``check()`` synchronises)."""
    for t in (q, k, v):
        if t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous bf16 host [B, h, n, d] tensors")
    B, h, n_q, d = q.shape
    n_k = k.shape[2]
    if tuple(k.shape) != (B, h, n_k, d) or tuple(v.shape) != (B, h, n_k, d):
        raise ValueError("k and v must be [B, h, n_k, d] with q's B, h, d")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    kl, left, right = None, 0, 0
    if window is not None:
        mask, (left, right) = MASK_WINDOW, window
    if mask == MASK_KEY_PADDING:
        if key_lens is None:
            raise ValueError("key padding needs key_lens")
        kl = key_lens
        if kl.dtype != torch.int32 or kl.is_cuda or kl.numel() != B or not kl.is_contiguous():
            raise ValueError("key_lens must be a contiguous int32 host tensor of B entries")
    pin = q.is_pinned()
    if out is None:
        out = torch.empty((B, h, n_q, d), dtype=q.dtype, pin_memory=pin)
    if out.is_cuda or tuple(out.shape) != (B, h, n_q, d) or not out.is_contiguous():
        raise ValueError("out must be a contiguous host [B, h, n_q, d] tensor")
    if lse is None and with_lse:
        lse = torch.empty((B, h, n_q), dtype=torch.float32, pin_memory=pin)
    need = host_buffer_bytes(B, h, n_q, n_k, d)
    if buf is None or buf.numel() * buf.element_size() < need:
        dev = torch.device("cuda") if device is None else torch.device(device)
        buf = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    rc = attn_fwd_host_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, h, n_q, n_k, d,
                           scale, int(mask), _ptr(kl), left, right, _ptr(buf),
                           buf.numel() * buf.element_size(), _stream_ptr(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_host")
    return out, lse


def attn_fwd_f32(q, k, v, **kw):
    """Float32 path (same as attn_fwd with float32 tensors)."""
    if q.dtype != torch.float32:
        raise ValueError("attn_fwd_f32 takes float32 tensors")
    return attn_fwd(q, k, v, **kw)


def decode_workspace_bytes(B: int, h: int, n_q: int, L_max: int, d: int = 64,
                           window: int | None = None) -> int:
    """Scratch bytes attn_decode (attn_decode_window when `window` is given)
    needs on the current device (0: none)."""
    if window is not None:
        return int(load().attn_decode_window_workspace_bytes(B, h, n_q, L_max, d, int(window)))
    return int(load().attn_decode_workspace_bytes(B, h, n_q, L_max, d))


def attn_decode_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, L_max, d, scale,
                    lens_ptr, ws_ptr, ws_bytes, stream_ptr) -> int:
    """The C call itself, on raw device pointers; returns the status code."""
    return load().attn_decode(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, L_max, d,
                              float(scale), lens_ptr, ws_ptr, int(ws_bytes), stream_ptr)


def attn_decode_window_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, L_max, d, scale,
                           lens_ptr, window, ws_ptr, ws_bytes, stream_ptr) -> int:
    """attn_decode_window on raw device pointers; returns the status code."""
    return load().attn_decode_window(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, L_max, d,
                                     float(scale), lens_ptr, int(window), ws_ptr, int(ws_bytes),
                                     stream_ptr)


def attn_decode_strided_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, L_max, d, strides,
                            scale, lens_ptr, ws_ptr, ws_bytes, stream_ptr) -> int:
    """The C call itself; ``strides`` = four (b, h, n) element-stride triples for q, k_cache,
    v_cache, o."""
    flat = (ctypes.c_int64 * 12)(*[int(x) for st in strides for x in st])
    return load().attn_decode_strided(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, n_q, L_max, d,
                                      ctypes.cast(flat, ctypes.c_void_p), float(scale), lens_ptr,
                                      ws_ptr, int(ws_bytes), stream_ptr)


def attn_decode_strided(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        cache_lens: torch.Tensor | None = None, scale: float | None = None,
                        out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None):
    """attn_decode on [B, h, n, d] bf16 views with any strides over the first three
    dimensions and a contiguous last one (e.g. a [B, L_max, h, d] cache seen as
    ``cache.transpose(1, 2)``); ``out`` may be a strided view too."""
    for t in (q, k_cache, v_cache):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or t.stride(-1) != 1:
            raise ValueError("q, k_cache, v_cache must be bf16 CUDA [B, h, n, d] views with unit "
                             "last stride")
    B, h, n_q, d = q.shape
    L_max = k_cache.shape[2]
    if tuple(k_cache.shape) != (B, h, L_max, d) or tuple(v_cache.shape) != (B, h, L_max, d):
        raise ValueError("caches must be [B, h, L_max, d] with q's B, h, d")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if cache_lens is not None and (cache_lens.dtype != torch.int32 or not cache_lens.is_cuda
                                   or cache_lens.numel() != B or not cache_lens.is_contiguous()):
        raise ValueError("cache_lens must be a contiguous int32 CUDA tensor of B entries")
    if out is None:
        out = torch.empty((B, h, n_q, d), dtype=q.dtype, device=q.device)
    if tuple(out.shape) != (B, h, n_q, d) or out.stride(-1) != 1:
        raise ValueError("out must be a [B, h, n_q, d] view with unit last stride")
    if lse is None:
        lse = torch.empty((B, h, n_q), dtype=torch.float32, device=q.device)
    need = decode_workspace_bytes(B, h, n_q, L_max, d)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    strides = [t.stride()[:3] for t in (q, k_cache, v_cache, out)]
    rc = attn_decode_strided_raw(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse), B,
                                 h, n_q, L_max, d, strides, scale, _ptr(cache_lens),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream_ptr(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode_strided")
    return out, lse


def attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                cache_lens: torch.Tensor | None = None, scale: float | None = None,
                out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, with_lse: bool = True, stream=None,
                window: int | None = None):
    """n_q <= 8 new queries q [B,h,n_q,d] against bf16 caches [B,h,L_max,d];
    query i sees the first cache_lens[b] keys (all L_max when None), or with
    `window` (attn_decode_window) only keys cache_lens[b]-1-window ..
    cache_lens[b]-1.  Returns (o, lse)."""
    for t in (q, k_cache, v_cache):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError("q and the caches must be contiguous bf16 CUDA [B, h, n, d] tensors")
    B, h, n_q, d = q.shape
    L_max = k_cache.shape[2]
    if tuple(k_cache.shape) != (B, h, L_max, d) or tuple(v_cache.shape) != (B, h, L_max, d):
        raise ValueError("caches must be [B, h, L_max, d] with q's B, h, d")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if cache_lens is not None and (cache_lens.dtype != torch.int32 or not cache_lens.is_cuda
                                   or cache_lens.numel() != B or not cache_lens.is_contiguous()):
        raise ValueError("cache_lens must be a contiguous int32 CUDA tensor of B entries")
    if out is None:
        out = torch.empty((B, h, n_q, d), dtype=q.dtype, device=q.device)
    if lse is None and with_lse:
        lse = torch.empty((B, h, n_q), dtype=torch.float32, device=q.device)
    need = decode_workspace_bytes(B, h, n_q, L_max, d, window)
    if need > 0 and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if window is None:
        rc = attn_decode_raw(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse), B, h,
                             n_q, L_max, d, scale, _ptr(cache_lens), _ptr(workspace), ws_bytes,
                             _stream_ptr(stream))
    else:
        rc = attn_decode_window_raw(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse),
                                    B, h, n_q, L_max, d, scale, _ptr(cache_lens), window,
                                    _ptr(workspace), ws_bytes, _stream_ptr(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode" if window is None else "attn_decode_window")
    return out, lse


def bwd_workspace_bytes(B: int, h: int, n_q: int, d: int = 64) -> int:
    """Scratch bytes attn_bwd needs (0 for unsupported sizes)."""
    return int(load().attn_bwd_workspace_bytes(B, h, n_q, d))


def attn_bwd_raw(q_ptr, k_ptr, v_ptr, o_ptr, dout_ptr, lse_ptr, dq_ptr, dk_ptr, dv_ptr, B, h,
                 n_q, n_k, d, scale, mask_kind, lens_ptr, ws_ptr, ws_bytes, stream_ptr) -> int:
    """The C call itself, on raw device pointers; returns the status code."""
    return load().attn_bwd(q_ptr, k_ptr, v_ptr, o_ptr, dout_ptr, lse_ptr, dq_ptr, dk_ptr, dv_ptr,
                           B, h, n_q, n_k, d, float(scale), int(mask_kind), lens_ptr, ws_ptr,
                           int(ws_bytes), stream_ptr)


def attn_bwd_window_raw(q_ptr, k_ptr, v_ptr, o_ptr, dout_ptr, lse_ptr, dq_ptr, dk_ptr, dv_ptr, B,
                        h, n_q, n_k, d, scale, left, right, ws_ptr, ws_bytes, stream_ptr) -> int:
    """The C call itself, on raw device pointers; returns the status code."""
    return load().attn_bwd_window(q_ptr, k_ptr, v_ptr, o_ptr, dout_ptr, lse_ptr, dq_ptr, dk_ptr,
                                  dv_ptr, B, h, n_q, n_k, d, float(scale), int(left), int(right),
                                  ws_ptr, int(ws_bytes), stream_ptr)


def attn_bwd_strided_raw(q_ptr, k_ptr, v_ptr, o_ptr, dout_ptr, lse_ptr, dq_ptr, dk_ptr, dv_ptr, B,
                         h, n_q, n_k, d, strides, scale, mask_kind, lens_ptr, left, right, ws_ptr,
                         ws_bytes, stream_ptr) -> int:
    """The C call itself; ``strides`` = eight (b, h, n) element-stride triples for q, k, v, o,
    dout, dq, dk, dv."""
    flat = (ctypes.c_int64 * 24)(*[int(x) for st in strides for x in st])
    return load().attn_bwd_strided(q_ptr, k_ptr, v_ptr, o_ptr, dout_ptr, lse_ptr, dq_ptr, dk_ptr,
                                   dv_ptr, B, h, n_q, n_k, d, ctypes.cast(flat, ctypes.c_void_p),
                                   float(scale), int(mask_kind), lens_ptr, int(left), int(right),
                                   ws_ptr, int(ws_bytes), stream_ptr)


def attn_bwd_strided(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                     lse: torch.Tensor, dout: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor,
                     dv: torch.Tensor, scale: float | None = None, mask: int = MASK_NONE,
                     key_lens: torch.Tensor | None = None,
                     window: tuple[int, int] | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """attn_bwd on [B, h, n, d] bf16 views with any strides over the first three
    dimensions and a contiguous last one; the gradients are written into the
    given dq, dk, dv views (e.g. slices of one packed gradient buffer).
    ``window=(left, right)`` differentiates restricted self-attention."""
    for t in (q, k, v, o, dout, dq, dk, dv):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or t.stride(-1) != 1:
            raise ValueError("tensors must be bf16 CUDA [B, h, n, d] views with unit last stride")
    B, h, n_q, d = q.shape
    n_k = k.shape[2]
    for t in (k, v, dk, dv):
        if tuple(t.shape) != (B, h, n_k, d):
            raise ValueError("k, v, dk, dv must be [B, h, n_k, d] with q's B, h, d")
    for t in (o, dout, dq):
        if tuple(t.shape) != (B, h, n_q, d):
            raise ValueError("o, dout, dq must be shaped like q")
    if (lse is None or not lse.is_cuda or lse.dtype != torch.float32
            or tuple(lse.shape) != (B, h, n_q) or not lse.is_contiguous()):
        raise ValueError("lse must be the forward's contiguous float32 [B, h, n_q] CUDA tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    kl, left, right = None, 0, 0
    if window is not None:
        mask, (left, right) = MASK_WINDOW, window
    if mask == MASK_KEY_PADDING:
        if key_lens is None:
            raise ValueError("key padding needs key_lens")
        kl = key_lens
        if kl.dtype != torch.int32 or not kl.is_cuda or kl.numel() != B or not kl.is_contiguous():
            raise ValueError("key_lens must be a contiguous int32 CUDA tensor of B entries")
    need = bwd_workspace_bytes(B, h, n_q, d)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    strides = [t.stride()[:3] for t in (q, k, v, o, dout, dq, dk, dv)]
    rc = attn_bwd_strided_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                              _ptr(dk), _ptr(dv), B, h, n_q, n_k, d, strides, scale, int(mask),
                              _ptr(kl), left, right, _ptr(workspace), ws_bytes,
                              _stream_ptr(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd_strided")
    return dq, dk, dv


def attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
             lse: torch.Tensor, dout: torch.Tensor, scale: float | None = None,
             mask: int = MASK_NONE, key_lens: torch.Tensor | None = None,
             dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
             dv: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
             window: tuple[int, int] | None = None, stream=None):
    """Gradients (dq, dk, dv) of attn_fwd for dout = dLoss/dO.

    q, k, v, o, dout: contiguous bf16 CUDA [B, h, n, d] tensors, d in {16, 32,
    64}; o and lse are what attn_fwd returned for q, k, v with the same scale
    and mask.
    A workspace of bwd_workspace_bytes(...) is allocated when none is given.
    ``window=(left, right)`` differentiates attn_fwd_window instead (mask and
    key_lens ignored).
    """
    for t in (q, k, v, o, dout):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError("q, k, v, o, dout must be contiguous bf16 CUDA [B, h, n, d] tensors")
    B, h, n_q, d = q.shape
    n_k = k.shape[2]
    if tuple(k.shape) != (B, h, n_k, d) or tuple(v.shape) != (B, h, n_k, d):
        raise ValueError("k and v must be [B, h, n_k, d] with q's B, h, d")
    if tuple(o.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape):
        raise ValueError("o and dout must be shaped like q")
    if (lse is None or not lse.is_cuda or lse.dtype != torch.float32
            or tuple(lse.shape) != (B, h, n_q) or not lse.is_contiguous()):
        raise ValueError("lse must be the forward's contiguous float32 [B, h, n_q] CUDA tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    kl = None
    if mask == MASK_KEY_PADDING:
        if key_lens is None:
            raise ValueError("key padding needs key_lens")
        kl = key_lens
        if kl.dtype != torch.int32 or not kl.is_cuda or kl.numel() != B or not kl.is_contiguous():
            raise ValueError("key_lens must be a contiguous int32 CUDA tensor of B entries")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = bwd_workspace_bytes(B, h, n_q, d)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if window is not None:
        rc = attn_bwd_window_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                 _ptr(dq), _ptr(dk), _ptr(dv), B, h, n_q, n_k, d, scale,
                                 window[0], window[1], _ptr(workspace), ws_bytes,
                                 _stream_ptr(stream))
    else:
        rc = attn_bwd_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                          _ptr(dk), _ptr(dv), B, h, n_q, n_k, d, scale, int(mask), _ptr(kl),
                          _ptr(workspace), ws_bytes, _stream_ptr(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd_window" if window is not None else "attn_bwd")
    return dq, dk, dv


class _call_on:
    """Makes the tensors' device current for a call, and the call's stream too,
    so that what is allocated for it belongs to that stream; gives the stream's
    pointer.  Nothing has to be switched for a call on the current stream of the
    current device.  `stream`: a torch stream of the tensors' device, or a
    cudaStream_t as a number (0: the default stream)."""

    __slots__ = ("_device", "_stream")

    def __init__(self, device: torch.device, stream):
        self._device = None
        if stream is not None and getattr(stream, "device", device) != device:
            raise ValueError(f"stream must be one of the tensors' device, {device}")
        if stream is not None or device.index != torch.cuda.current_device():
            self._device = torch.cuda.device(device)
        self._stream = stream if self._device is not None else device.index

    def __enter__(self) -> int:
        if self._device is None:
            return torch._C._cuda_getCurrentRawStream(self._stream)
        self._device.__enter__()
        stream = self._stream
        if stream is None:
            stream = torch.cuda.current_stream()
        elif not hasattr(stream, "cuda_stream"):
            # (ExternalStream(0) would be a new stream)
            stream = (torch.cuda.ExternalStream(int(stream)) if int(stream)
                      else torch.cuda.default_stream())
        self._stream = torch.cuda.stream(stream)
        self._stream.__enter__()
        return int(stream.cuda_stream)

    def __exit__(self, *exc):
        if self._device is not None:
            self._stream.__exit__(*exc)
            self._device.__exit__(*exc)


def _views(what: str, dtype, *tensors) -> None:
    """[B, h, n, d] CUDA views of one dtype on one device with unit last stride."""
    device = tensors[0].device
    for t in tensors:
        if (t.dtype != dtype or t.dim() != 4 or t.device != device or not t.is_cuda
                or t.stride(3) != 1):
            raise ValueError(f"{what} must be {dtype} CUDA [B, h, n, d] views on one device with "
                             "unit last stride")


def _vector(name: str, t, dtype, count: int, device) -> None:
    if t is not None and (t.dtype != dtype or t.device != device or t.numel() != count
                          or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {count} entries on "
                         f"{device}")


_INT_MAX = 0x7fffffff  # what fits the C calls' sizes

_INT64S = {n: ctypes.c_int64 * n for n in (12, 24)}


def _strides_array(strides):
    """A host array of element strides (None: contiguous tensors)."""
    if strides is None or isinstance(strides, ctypes.Array):
        return strides
    return _INT64S[len(strides)](*strides)


@functools.lru_cache(maxsize=1024)
def _strides_of(layouts):
    flat = []
    for step, shape in layouts:
        if 1 in shape[:3]:
            room = -(-max(*step, shape[2] * shape[3]) // 16) * 16
            flat += [step[i] if shape[i] > 1 else room for i in range(3)]
        else:
            flat += step[:3]
    return _strides_array(flat)


def _strides(*tensors):
    """The (b, h, row) element strides of [B, h, n, d] views.  The stride of a
    dimension of one entry is never stepped over, whatever the view says.  None
    when all are contiguous, which needs no strides."""
    for t in tensors:
        if not t.is_contiguous():
            break
    else:
        return None
    return _strides_of(tuple([(t.stride(), t.shape) for t in tensors]))


def _workspace(need: int, given, device):
    """The caller's scratch when it is large enough, else a new one."""
    if need == 0:
        return None
    if given is not None:
        if given.device != device or not given.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {device}")
        if _nbytes(given) >= need:
            return given
    return torch.empty(need, dtype=torch.uint8, device=device)


def _contiguous_like(t):
    """A new contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def attn_cache_append_raw(k_new_ptr, v_new_ptr, k_ptr, v_ptr, ks_ptr, vs_ptr, B, h, n_new, L_max, d,
                          strides, cache_format, block_tokens, lens_ptr, new_lens_ptr,
                          stream_ptr) -> int:
    """The C call itself, on raw device pointers; ``strides`` = 12 element counts or None."""
    return load().attn_cache_append(
        k_new_ptr, v_new_ptr, k_ptr, v_ptr, ks_ptr, vs_ptr, B, h, n_new, L_max, d,
        _strides_array(strides), cache_format, block_tokens, lens_ptr, new_lens_ptr, stream_ptr)


def attn_cache_append(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                      cache_lens: torch.Tensor | None, block_tokens: int = 64,
                      new_lens: torch.Tensor | None = None, stream=None) -> None:
    """Writes bf16 k_new, v_new [B, h, n_new, d] behind the first cache_lens[b]
    tokens (None: empty) of 8-bit caches [B, h, L_max, d] (torch.float8_e4m3fn
    or torch.int8 codes), one float32 scale per block of block_tokens tokens and
    head in k_scale, v_scale [B, h, ceil(L_max / block_tokens)].  With new_lens
    only the first new_lens[b] new tokens.  cache_lens is not changed."""
    _views("k_new and v_new", torch.bfloat16, k_new, v_new)
    fmt = _CACHE_FORMATS.get(k_cache.dtype, CACHE_BF16)
    if fmt == CACHE_BF16:
        raise ValueError("the caches must hold torch.float8_e4m3fn or torch.int8 codes")
    _views("k_cache and v_cache", k_cache.dtype, k_cache, v_cache)
    B, h, n_new, d = k_new.shape
    L_max = k_cache.shape[2]
    if (v_new.shape != k_new.shape or tuple(k_cache.shape) != (B, h, L_max, d)
            or v_cache.shape != k_cache.shape or k_cache.device != k_new.device):
        raise ValueError("k_new, v_new must be [B, h, n_new, d] and the caches [B, h, L_max, d]")
    if n_new > _INT_MAX or L_max > _INT_MAX:
        raise ValueError("caches of 2^31 tokens and more are not supported")
    if block_tokens not in (16, 32, 64, 128):
        raise ValueError("block_tokens must be 16, 32, 64 or 128")
    dev = k_new.device
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _vector(name, t, torch.float32, B * h * -(-L_max // block_tokens), dev)
    _vector("cache_lens", cache_lens, torch.int32, B, dev)
    _vector("new_lens", new_lens, torch.int32, B, dev)
    with _call_on(dev, stream) as ptr:
        rc = attn_cache_append_raw(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(k_scale), _ptr(v_scale), B, h, n_new, L_max, d,
                                   _strides(k_new, v_new, k_cache, v_cache), fmt, block_tokens,
                                   _ptr(cache_lens), _ptr(new_lens), ptr)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_cache_append")


@functools.lru_cache(maxsize=256)
def _decode_scored_bytes(device: int, *sizes) -> int:
    """The workspace size follows from the sizes and the device alone."""
    return int(load().attn_decode_scored_workspace_bytes(*sizes))


def decode_scored_workspace_bytes(B: int, h: int, h_kv: int, n_q: int, L_max: int, d: int,
                                  cache_format: int = CACHE_BF16,
                                  window: int | None = None) -> int:
    """Scratch bytes attn_decode_scored needs on the current device (0: none)."""
    return int(load().attn_decode_scored_workspace_bytes(
        B, h, h_kv, n_q, L_max, d, cache_format,
        -1 if window is None else min(int(window), _INT_MAX)))


def attn_decode_scored_raw(q_ptr, k_ptr, v_ptr, ks_ptr, vs_ptr, o_ptr, lse_ptr, B, h, h_kv, n_q,
                           L_max, d, strides, cache_format, block_tokens, scale, softcap,
                           slopes_ptr, lens_ptr, window, ws_ptr, ws_bytes, stream_ptr) -> int:
    """The C call itself, on raw device pointers; ``strides`` = 12 element counts or None."""
    return load().attn_decode_scored(
        q_ptr, k_ptr, v_ptr, ks_ptr, vs_ptr, o_ptr, lse_ptr, B, h, h_kv, n_q, L_max, d,
        _strides_array(strides), cache_format, block_tokens, scale, softcap, slopes_ptr, lens_ptr,
        window, ws_ptr, ws_bytes, stream_ptr)


def attn_decode_scored(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       cache_lens: torch.Tensor | None = None,
                       k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                       block_tokens: int = 64, scale: float | None = None, softcap: float = 0.0,
                       slopes: torch.Tensor | None = None, window: int | None = None,
                       out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None):
    """n_q <= 8 newest queries q [B, h, n_q, d] (bf16) against a cache [B, h_kv,
    L_max, d] of bf16 rows or of 8-bit codes with scales (see attn_cache_append);
    query i stands at position cache_lens[b] - n_q + i and sees the keys up to
    there (with `window`: that key and the `window` before it).  softcap > 0
    caps the scores by a tanh, slopes [h] (float32) bias them by distance.
    Returns (o, lse)."""
    _views("q", torch.bfloat16, q)
    fmt = _CACHE_FORMATS.get(k_cache.dtype)
    if fmt is None:
        raise ValueError("the caches must be bf16, torch.float8_e4m3fn or torch.int8")
    _views("k_cache and v_cache", k_cache.dtype, k_cache, v_cache)
    B, h, n_q, d = q.shape
    h_kv, L_max = k_cache.shape[1:3]
    if (tuple(k_cache.shape) != (B, h_kv, L_max, d) or v_cache.shape != k_cache.shape
            or h_kv < 1 or h % h_kv != 0 or k_cache.device != q.device):
        raise ValueError("caches must be [B, h_kv, L_max, d] with q's B and d, h a multiple of h_kv")
    if L_max > _INT_MAX:
        raise ValueError("caches of 2^31 tokens and more are not supported")
    dev = q.device
    if fmt == CACHE_BF16:
        k_scale = v_scale = None
    else:
        if block_tokens not in (16, 32, 64, 128):
            raise ValueError("block_tokens must be 16, 32, 64 or 128")
        if k_scale is None or v_scale is None:
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _vector(name, t, torch.float32, B * h_kv * -(-L_max // block_tokens), dev)
    _vector("cache_lens", cache_lens, torch.int32, B, dev)
    _vector("slopes", slopes, torch.float32, h, dev)
    if window is not None and window < 0:
        raise ValueError("window must be >= 0 (None for none)")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _call_on(dev, stream) as ptr:
        if out is None:
            out = _contiguous_like(q)
        else:
            _views("q and out", torch.bfloat16, q, out)
            if out.shape != q.shape:
                raise ValueError("out must be shaped like q")
        if lse is None:
            lse = q.new_empty((B, h, n_q), dtype=torch.float32)
        else:
            _vector("lse", lse, torch.float32, B * h * n_q, dev)
        window = -1 if window is None else min(int(window), _INT_MAX)
        workspace = _workspace(
            _decode_scored_bytes(dev.index, B, h, h_kv, n_q, L_max, d, fmt, window), workspace, dev)
        rc = attn_decode_scored_raw(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(out),
            _ptr(lse), B, h, h_kv, n_q, L_max, d, _strides(q, k_cache, v_cache, out), fmt,
            block_tokens, scale, softcap, _ptr(slopes), _ptr(cache_lens),
            window, _ptr(workspace), _nbytes(workspace), ptr)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode_scored")
    return out, lse


def _not_negative(name: str, x: int) -> int:
    if x < 0:
        raise ValueError(f"{name} must be >= 0 (None: unbounded)")
    return min(int(x), _INT_MAX)


@functools.lru_cache(maxsize=256)
def mask_plan_bytes(B: int, n_q: int, n_k: int) -> int:
    """Bytes of a mask plan for these sizes (0 for unsupported sizes)."""
    return int(load().attn_mask_plan_bytes(B, n_q, n_k))


def attn_mask_plan_raw(B, n_q, n_k, left, right, lens_ptr, docs_ptr, prefix_ptr, plan_ptr,
                       plan_bytes, stream_ptr) -> int:
    """The C call itself, on raw device pointers; returns the status code."""
    return load().attn_mask_plan(B, n_q, n_k, left, right, lens_ptr, docs_ptr, prefix_ptr,
                                 plan_ptr, plan_bytes, stream_ptr)


def attn_mask_plan(B: int, n_q: int, n_k: int, left: int | None = None, right: int | None = None,
                   key_lens: torch.Tensor | None = None, doc_ids: torch.Tensor | None = None,
                   prefix_lens: torch.Tensor | None = None, plan: torch.Tensor | None = None,
                   device=None, stream=None) -> torch.Tensor:
    """The plan of a mask for attn_fwd_scored and attn_bwd_scored, a uint8 tensor
    (``plan`` when one is given): query i sees the keys i - left .. i + right
    (None: unbounded; right=0 is causal) and, with prefix_lens [B], the first
    prefix_lens[b] keys; of them those below key_lens[b] and, with doc_ids
    [B, n], those of its own run of equal ids (negative: no document)."""
    dev = device
    if dev is None:
        given = [t for t in (key_lens, doc_ids, prefix_lens, plan) if t is not None]
        dev = given[0].device if given else torch.device("cuda")
    elif not isinstance(dev, torch.device):
        dev = torch.device(dev)
    if dev.type != "cuda":
        raise ValueError("a mask plan lives on a CUDA device")
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    left = -1 if left is None else _not_negative("left", left)
    right = -1 if right is None else _not_negative("right", right)
    if key_lens is not None:
        _vector("key_lens", key_lens, torch.int32, B, dev)
    if prefix_lens is not None:
        _vector("prefix_lens", prefix_lens, torch.int32, B, dev)
        if left >= 0:
            raise ValueError("a prefix and a left bound leave a query two runs of keys")
    if doc_ids is not None:
        _vector("doc_ids", doc_ids, torch.int32, B * n_q, dev)
        if n_q != n_k:
            raise ValueError("documents need n_q == n_k")
    if max(B, n_q, n_k) > _INT_MAX:
        raise ValueError("sequences of 2^31 tokens and more are not supported")
    need = mask_plan_bytes(B, n_q, n_k)
    if plan is not None and (plan.device != dev or not plan.is_contiguous()
                             or _nbytes(plan) < need):
        raise ValueError(f"plan must be contiguous, on {dev} and of at least {need} bytes")
    with _call_on(dev, stream) as ptr:
        if plan is None:
            plan = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        rc = attn_mask_plan_raw(B, n_q, n_k, left, right, _ptr(key_lens), _ptr(doc_ids),
                                _ptr(prefix_lens), plan.data_ptr(), _nbytes(plan), ptr)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_mask_plan")
    return plan


def _scored_shapes(q, k, v, slopes, plan):
    """Sizes of a call with changed scores, checked: B, h, h_kv, n_q, n_k, d."""
    _views("q, k, v", torch.bfloat16, q, k, v)
    B, h, n_q, d = q.shape
    h_kv, n_k = k.shape[1:3]
    if (tuple(k.shape) != (B, h_kv, n_k, d) or v.shape != k.shape or h_kv < 1 or h % h_kv != 0):
        raise ValueError("k and v must be [B, h_kv, n_k, d] with q's B and d, h a multiple of h_kv")
    if n_q > _INT_MAX or n_k > _INT_MAX:
        raise ValueError("sequences of 2^31 tokens and more are not supported")
    _vector("slopes", slopes, torch.float32, h, q.device)
    if plan is not None and (plan.device != q.device or not plan.is_contiguous()
                             or _nbytes(plan) < mask_plan_bytes(B, n_q, n_k)):
        raise ValueError("plan must be attn_mask_plan's for these sizes and this device")
    return B, h, h_kv, n_q, n_k, d


def attn_fwd_scored_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, h_kv, n_q, n_k, d, strides,
                        scale, softcap, slopes_ptr, plan_ptr, plan_bytes, stream_ptr) -> int:
    """The C call itself, on raw device pointers; ``strides`` = 12 element counts or None."""
    return load().attn_fwd_scored(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, h, h_kv, n_q, n_k, d,
                                  _strides_array(strides), scale, softcap, slopes_ptr, plan_ptr,
                                  plan_bytes, stream_ptr)


def attn_fwd_scored(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    plan: torch.Tensor | None = None, scale: float | None = None,
                    softcap: float = 0.0, slopes: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    stream=None):
    """Attention with changed scores on bf16 views q [B, h, n_q, d] and k, v
    [B, h_kv, n_k, d] (h a multiple of h_kv): softcap > 0 caps them by a tanh,
    slopes [h] (float32) take slopes * |i - j| off.  ``plan``: the mask
    (attn_mask_plan; None: every query sees every key).  Returns (o, lse)."""
    B, h, h_kv, n_q, n_k, d = _scored_shapes(q, k, v, slopes, plan)
    dev = q.device
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _call_on(dev, stream) as ptr:
        if out is None:
            out = _contiguous_like(q)
        else:
            _views("q and out", torch.bfloat16, q, out)
            if out.shape != q.shape:
                raise ValueError("out must be shaped like q")
        if lse is None:
            lse = q.new_empty((B, h, n_q), dtype=torch.float32)
        else:
            _vector("lse", lse, torch.float32, B * h * n_q, dev)
        rc = attn_fwd_scored_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, h, h_kv, n_q,
                                 n_k, d, _strides(q, k, v, out), scale, softcap, _ptr(slopes),
                                 _ptr(plan), _nbytes(plan), ptr)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_scored")
    return out, lse


@functools.lru_cache(maxsize=256)
def bwd_scored_workspace_bytes(B: int, h: int, h_kv: int, n_q: int, n_k: int, d: int = 64) -> int:
    """Scratch bytes attn_bwd_scored needs (0 for unsupported sizes)."""
    return int(load().attn_bwd_scored_workspace_bytes(B, h, h_kv, n_q, n_k, d))


def attn_bwd_scored_raw(q_ptr, k_ptr, v_ptr, o_ptr, dout_ptr, lse_ptr, dq_ptr, dk_ptr, dv_ptr, B, h,
                        h_kv, n_q, n_k, d, strides, scale, softcap, slopes_ptr, plan_ptr,
                        plan_bytes, ws_ptr, ws_bytes, stream_ptr) -> int:
    """The C call itself, on raw device pointers; ``strides`` = 24 element counts or None."""
    return load().attn_bwd_scored(q_ptr, k_ptr, v_ptr, o_ptr, dout_ptr, lse_ptr, dq_ptr, dk_ptr,
                                  dv_ptr, B, h, h_kv, n_q, n_k, d, _strides_array(strides), scale,
                                  softcap, slopes_ptr, plan_ptr, plan_bytes, ws_ptr, ws_bytes,
                                  stream_ptr)


def attn_bwd_scored(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                    lse: torch.Tensor, dout: torch.Tensor, plan: torch.Tensor | None = None,
                    scale: float | None = None, softcap: float = 0.0,
                    slopes: torch.Tensor | None = None, dq: torch.Tensor | None = None,
                    dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None):
    """Gradients (dq, dk, dv) of attn_fwd_scored for dout = dLoss/dO, given its o
    and lse and the same plan, scale, softcap and slopes; d in {16, 32, 64}.
    All tensors but lse may be views of any strides with unit last stride."""
    B, h, h_kv, n_q, n_k, d = _scored_shapes(q, k, v, slopes, plan)
    dev = q.device
    _views("q, o, dout", torch.bfloat16, q, o, dout)
    if o.shape != q.shape or dout.shape != q.shape:
        raise ValueError("o and dout must be shaped like q")
    if lse is None:
        raise ValueError("lse must be the forward's")
    _vector("lse", lse, torch.float32, B * h * n_q, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None:
            _views(f"q and {name}", torch.bfloat16, q, t)
            if t.shape != like.shape:
                raise ValueError(f"{name} must be shaped like {name[1]}")
    with _call_on(dev, stream) as ptr:
        if dq is None:
            dq = _contiguous_like(q)
        if dk is None:
            dk = _contiguous_like(k)
        if dv is None:
            dv = _contiguous_like(v)
        workspace = _workspace(max(bwd_scored_workspace_bytes(B, h, h_kv, n_q, n_k, d), 16),
                               workspace, dev)
        rc = attn_bwd_scored_raw(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                 _ptr(dq), _ptr(dk), _ptr(dv), B, h, h_kv, n_q, n_k, d,
                                 _strides(q, k, v, o, dout, dq, dk, dv), scale, softcap,
                                 _ptr(slopes), _ptr(plan), _nbytes(plan), _ptr(workspace),
                                 _nbytes(workspace), ptr)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd_scored")
    return dq, dk, dv


def check(stream=None) -> None:
    """Synchronise and raise if a kernel recorded an error (bounded wait ran out)."""
    rc = load().attn_check(_stream_ptr(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_check")


def set_wait_limit_ns(limit_ns: int) -> int:
    return int(load().attn_set_wait_limit_ns(int(limit_ns)))


def launch_count() -> int:
    return int(load().attn_launch_count())


def diag_tile(q, k, p, v, stream=None):
    """Single-tile tensor-core products (see attn_diag_tile in include/attn.h).

    q, k: bf16 [128, 64]; p: bf16 [128, 128]; v: bf16 [128, 64].
    Returns (s = q k^T float32 [128,128], o = p v float32 [128, 64]).
    """
    for t, shp in ((q, (128, 64)), (k, (128, 64)), (p, (128, 128)), (v, (128, 64))):
        if tuple(t.shape) != shp or t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"diag_tile: expected contiguous bf16 CUDA {shp}")
    s = torch.empty((128, 128), dtype=torch.float32, device=q.device)
    o = torch.empty((128, 64), dtype=torch.float32, device=q.device)
    rc = load().attn_diag_tile(_ptr(q), _ptr(k), _ptr(p), _ptr(v), _ptr(s), _ptr(o),
                               _stream_ptr(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_diag_tile")
    return s, o


def diag_wait_timeout(limit_ns: int, stream=None) -> None:
    rc = load().attn_diag_wait_timeout(int(limit_ns), _stream_ptr(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_diag_wait_timeout")
