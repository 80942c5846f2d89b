"""Python binding of libattn_gb300.so (exact attention for GB300 / sm_103a).

The functions below only marshal arguments (torch tensors -> device pointers, sizes, the
current CUDA stream) and call the C ABI declared in ``include/attn.h``; every step of the
computation runs in the library's CUDA kernels.  There is no CPU or PyTorch fallback: if the
library is missing the import fails, and an unsupported request raises ``AttnError``.

What a call allocates, results and workspace, belongs to the stream it runs on (``stream``, or
torch's current one): another stream uses a result after waiting for that one.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os

__all__ = [
    "AttnError", "attn_fwd", "attn_fwd_window", "attn_fwd_block_sparse", "attn_fwd_fp8",
    "attn_fwd_fp8_workspace_bytes", "attn_fwd_fp8_workspace_offsets",
    "attn_fwd_window_sinks", "attn_bwd_window_sinks", "attn_bwd_window_sinks_workspace_bytes",
    "attn_fwd_paged", "attn_fwd_paged_workspace_bytes",
    "attn_cache_write_fp8", "attn_cache_read_fp8",
    "attn_decode_paged_fp8", "attn_decode_paged_fp8_workspace_bytes",
    "attn_bwd", "attn_bwd_workspace_bytes",
    "attn_decode_splitkv", "attn_decode_workspace_bytes", "attn_decode_paged",
    "attn_decode_splitkv_static", "attn_decode_static_scratch_bytes",
    "attn_poll_status", "attn_status_string", "attn_fwd_kv_tiles", "attn_fwd_kv_span",
    "attn_fwd_set_d64_kernel", "D64_AUTO", "D64_PAIR", "D64_SINGLE",
    "attn_bwd_kv_order", "attn_selftest_timeout",
    "attn_version", "library_path", "lib",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_PKG, "libattn_gb300.so")

if not os.path.exists(library_path):
    raise ImportError(
        f"{library_path} is missing: build it first (python exact_io_aware_09_gb300/build.py "
        "or __graft_entry__.build()); there is no fallback implementation")

lib = ctypes.CDLL(library_path)

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t
lib.attn_fwd.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _I]
lib.attn_fwd.restype = _I
lib.attn_bwd_workspace_bytes.argtypes = [_I, _I, _I]
lib.attn_bwd_workspace_bytes.restype = _SZ
lib.attn_bwd.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P,
                         _SZ, _P]
lib.attn_bwd.restype = _I
lib.attn_fwd_fp8_workspace_bytes.argtypes = [_I] * 6
lib.attn_fwd_fp8_workspace_bytes.restype = _SZ
lib.attn_fwd_fp8_workspace_offsets.argtypes = [_I] * 6 + [_P]
lib.attn_fwd_fp8_workspace_offsets.restype = _I
lib.attn_fwd_fp8.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _SZ, _P, _I]
lib.attn_fwd_fp8.restype = _I
lib.attn_fwd_window.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _I]
lib.attn_fwd_window.restype = _I
lib.attn_fwd_window_sinks.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P,
                                      _I]
lib.attn_fwd_window_sinks.restype = _I
lib.attn_bwd_window_sinks_workspace_bytes.argtypes = [_I] * 8
lib.attn_bwd_window_sinks_workspace_bytes.restype = _SZ
lib.attn_bwd_window_sinks.argtypes = [_P] * 9 + [_I] * 8 + [_F, _I, _P, _SZ, _P]
lib.attn_bwd_window_sinks.restype = _I
lib.attn_fwd_paged_workspace_bytes.argtypes = [_I] * 9
lib.attn_fwd_paged_workspace_bytes.restype = _SZ
lib.attn_fwd_paged.argtypes = [_P] * 6 + [_I] * 6 + [_P, _P] + [_I] * 6 + [_F, _I, _P, _SZ, _P]
lib.attn_fwd_paged.restype = _I
lib.attn_cache_write_fp8.argtypes = [_P] * 9 + [_I] * 8 + [_P]
lib.attn_cache_write_fp8.restype = _I
lib.attn_cache_read_fp8.argtypes = [_P] * 6 + [_I] * 3 + [_P, _P] + [_I] * 5 + [_P]
lib.attn_cache_read_fp8.restype = _I
lib.attn_decode_paged_fp8.argtypes = [_P] * 7 + [_I] * 4 + [_P, _P] + [_I] * 5 + [_F, _I, _P, _SZ,
                                                                              _P]
lib.attn_decode_paged_fp8.restype = _I
lib.attn_decode_paged_fp8_workspace_bytes.argtypes = [_I] * 6
lib.attn_decode_paged_fp8_workspace_bytes.restype = _SZ
lib.attn_fwd_block_sparse.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _F, _P,
                                      _I]
lib.attn_fwd_block_sparse.restype = _I
lib.attn_decode_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
lib.attn_decode_workspace_bytes.restype = _SZ
lib.attn_decode_splitkv.argtypes = [_P, _P, _P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I, _F, _I,
                                    _P, _SZ, _P]
lib.attn_decode_splitkv.restype = _I
lib.attn_decode_splitkv_static.argtypes = [_P, _P, _P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I,
                                           _F, _I, _P]
lib.attn_decode_splitkv_static.restype = _I
lib.attn_decode_paged.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _I, _I, _I, _I, _I, _F,
                                  _I, _P, _SZ, _P]
lib.attn_decode_paged.restype = _I
lib.attn_decode_static_scratch_bytes.argtypes = []
lib.attn_decode_static_scratch_bytes.restype = _SZ
lib.attn_poll_status.argtypes = [_P]
lib.attn_poll_status.restype = _I
lib.attn_status_string.argtypes = [_I]
lib.attn_status_string.restype = ctypes.c_char_p
lib.attn_fwd_kv_tiles.argtypes = [_I, _I, _I, _I, _I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)]
lib.attn_fwd_kv_tiles.restype = _I
lib.attn_fwd_set_d64_kernel.argtypes = [_I]
lib.attn_fwd_set_d64_kernel.restype = _I
lib.attn_bwd_kv_order.argtypes = [_I] * 7 + [ctypes.POINTER(ctypes.c_uint16), _I, ctypes.POINTER(_I)]
lib.attn_bwd_kv_order.restype = _I
lib.attn_fwd_kv_span.argtypes = [_I, _I, _I, _I, _I, _I, _I] + [ctypes.POINTER(_I)] * 4
lib.attn_fwd_kv_span.restype = _I
lib.attn_selftest_timeout.argtypes = [_I, _P]
lib.attn_selftest_timeout.restype = _I
lib.attn_version.argtypes = []
lib.attn_version.restype = ctypes.c_char_p

ATTN_F16, ATTN_BF16 = 0, 1


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {attn_status_string(status)} (status {status})")


def attn_status_string(status: int) -> str:
    return lib.attn_status_string(int(status)).decode()


def attn_version() -> str:
    return lib.attn_version().decode()


def _torch():
    import torch

    return torch


_NO_SWITCH = contextlib.nullcontext()


def _stream_handle(stream, device=None):
    """The raw handle of ``stream`` (a torch stream or an integer handle); None = torch's
    current stream of ``device`` (of the current device when that is None too).  A torch
    stream must belong to ``device``."""
    if stream is None:
        cuda = _torch()._C
        return cuda._cuda_getCurrentRawStream(cuda._cuda_getDevice() if device is None
                                              else device.index)
    if device is not None and getattr(stream, "device", device) != device:
        raise AttnError(-1, f"stream on {stream.device}, tensors on {device}")
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _allocating(stream, device):
    """A context in which torch allocates for ``stream``, the stream the call runs on: a workspace
    given back when the call returns is then reused behind the call's kernels and not beside them."""
    if stream is None or device.type != "cuda":  # (tensors off the GPU are refused later)
        return _NO_SWITCH
    handle = _stream_handle(stream, device)
    cuda = _torch().cuda
    if hasattr(stream, "cuda_stream"):
        return cuda.stream(stream)
    # handle 0, the legacy default stream, makes a stream of torch's pool of an ExternalStream
    return cuda.stream(cuda.ExternalStream(handle, device=device) if handle
                       else cuda.default_stream(device))


def _on_device(where, first, *others):
    """Checks that every given tensor sits on ``first``'s CUDA device and returns a context
    that makes that device current, so that the library's launches, its per-device state and
    torch's default stream all refer to the device that holds the data."""
    torch = _torch()
    if not first.is_cuda:
        raise AttnError(-1, f"{where}: tensors must be CUDA tensors")
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise AttnError(-1, f"{where}: tensors on {first.device} and {t.device}")
    if torch._C._cuda_getDevice() == index:
        return _NO_SWITCH  # entering a device context costs a microsecond
    return torch.cuda.device(first.device)


def _pointers(where, names, tensors):
    """The device index of the first tensor and every tensor's address (None for None), checked to
    be contiguous CUDA tensors of that device: one pass, since a call's host time is mostly this."""
    index = tensors[0].get_device()
    out = []
    for i, t in enumerate(tensors):
        if t is None:
            out.append(None)
        elif index < 0 or t.get_device() != index or not t.is_contiguous():
            raise AttnError(-1, f"{where}: {names[i]} must be a contiguous CUDA tensor"
                                + (f" on {tensors[0].device}" if index >= 0 else ""))
        else:
            out.append(t.data_ptr())
    return index, out


def _device(index):
    """A context with CUDA device ``index`` current; nothing to do where it is already."""
    torch = _torch()
    return _NO_SWITCH if torch._C._cuda_getDevice() == index else torch.cuda.device(index)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float16:
        return ATTN_F16
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    raise AttnError(-2, f"dtype {t.dtype}")


def _check(status: int, where: str):
    if status != 0:
        raise AttnError(status, where)


def _dev_ptr(t, name):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise AttnError(-1, f"{name} must be a contiguous CUDA tensor")
    return t.data_ptr()


def attn_fwd(q, k, v, o=None, lse=None, causal: bool = False, scale: float | None = None,
             stream=None):
    """Exact attention forward.  q [B,Hq,N_q,d], k/v [B,Hkv,N_kv,d] fp16/bf16 CUDA tensors.

    Returns (o [B,Hq,N_q,d] same dtype, lse [B,Hq,N_q] fp32).  Enqueued on ``stream``
    (default: torch's current stream); no synchronisation.
    """
    torch = _torch()
    B, Hq, N_q, d = q.shape
    _, Hkv, N_kv, _ = k.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != d or k.dtype != q.dtype or v.dtype != q.dtype:
        raise AttnError(-1, "attn_fwd: q/k/v shapes or dtypes disagree")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _allocating(stream, q.device):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq, N_q), device=q.device, dtype=torch.float32)
    with _on_device("attn_fwd", q, k, v, o, lse):
        st = lib.attn_fwd(_dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"), _dev_ptr(o, "o"),
                          _dev_ptr(lse, "lse"), B, Hq, Hkv, N_q, N_kv, d, int(bool(causal)),
                          float(scale), _stream_handle(stream, q.device), _dtype_code(q))
    _check(st, "attn_fwd")
    return o, lse


def _expect(where, t, name, dtype, shape):
    if t.dtype != dtype or t.shape != shape:
        raise AttnError(-1, f"{where}: {name} must be {dtype} {tuple(shape)}, "
                            f"got {t.dtype} {tuple(t.shape)}")


def _fwd_prep(q, k, v, o, lse, scale, stream):
    torch = _torch()
    B, Hq, N_q, d = q.shape
    _, Hkv, N_kv, _ = k.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != d or k.dtype != q.dtype or v.dtype != q.dtype:
        raise AttnError(-1, "attn_fwd: q/k/v shapes or dtypes disagree")
    with _allocating(stream, q.device):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq, N_q), device=q.device, dtype=torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    return B, Hq, Hkv, N_q, N_kv, d, o, lse, float(scale)


def attn_bwd_workspace_bytes(B: int, Hq: int, N_q: int) -> int:
    return int(lib.attn_bwd_workspace_bytes(B, Hq, N_q))


def attn_bwd(q, k, v, o, dout, lse, causal: bool = False, scale: float | None = None,
             dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of attn_fwd for the incoming gradient ``dout`` (shape of o).

    q/o/dout [B,Hq,N_q,d], k/v [B,Hkv,N_kv,d] 16-bit CUDA tensors, lse [B,Hq,N_q] fp32 as
    attn_fwd returns it.  Deterministic.
    """
    torch = _torch()
    B, Hq, N_q, d = q.shape
    _, Hkv, N_kv, _ = k.shape
    for t, nm in ((o, "o"), (dout, "dout")):
        if t.shape != q.shape or t.dtype != q.dtype:
            raise AttnError(-1, f"attn_bwd: {nm} must match q")
    if k.shape != v.shape or k.dtype != q.dtype or v.dtype != q.dtype or lse.dtype != torch.float32:
        raise AttnError(-1, "attn_bwd: k/v/lse shapes or dtypes disagree")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _allocating(stream, q.device):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        if workspace is None:
            workspace = torch.empty(max(int(lib.attn_bwd_workspace_bytes(B, Hq, N_q)), 1),
                                    device=q.device, dtype=torch.uint8)
    with _on_device("attn_bwd", q, k, v, o, dout, lse, dq, dk, dv, workspace):
        st = lib.attn_bwd(_dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"), _dev_ptr(o, "o"),
                          _dev_ptr(dout, "dout"), _dev_ptr(lse, "lse"), _dev_ptr(dq, "dq"),
                          _dev_ptr(dk, "dk"), _dev_ptr(dv, "dv"), B, Hq, Hkv, N_q, N_kv, d,
                          int(bool(causal)), float(scale), _dtype_code(q),
                          _dev_ptr(workspace, "workspace"), workspace.numel(),
                          _stream_handle(stream, q.device))
    _check(st, "attn_bwd")
    return dq, dk, dv


def attn_fwd_fp8_workspace_bytes(B, Hq, Hkv, N_q, N_kv, d) -> int:
    return int(lib.attn_fwd_fp8_workspace_bytes(B, Hq, Hkv, N_q, N_kv, d))


def attn_fwd_fp8_workspace_offsets(B, Hq, Hkv, N_q, N_kv, d):
    """Byte offsets of (Q codes, K codes, V^T codes, Q scales, K scales, V scales, scratch)."""
    off = (ctypes.c_size_t * 7)()
    _check(lib.attn_fwd_fp8_workspace_offsets(B, Hq, Hkv, N_q, N_kv, d, off),
           "attn_fwd_fp8_workspace_offsets")
    return list(off)


def attn_fwd_fp8(q, k, v, signs=None, o=None, lse=None, causal: bool = False,
                 scale: float | None = None, workspace=None, stream=None):
    """FP8 prefill with incoherent processing.  signs: int8 CUDA tensor [d] of +-1 (None: no
    rotation).  Shapes and return value as attn_fwd (d = 128)."""
    torch = _torch()
    B, Hq, Hkv, N_q, N_kv, d, o, lse, scale = _fwd_prep(q, k, v, o, lse, scale, stream)
    if signs is not None and (signs.dtype != torch.int8 or tuple(signs.shape) != (d,)):
        raise AttnError(-1, "attn_fwd_fp8: signs must be int8 [d]")
    if workspace is None:
        with _allocating(stream, q.device):
            workspace = torch.empty(max(1, attn_fwd_fp8_workspace_bytes(B, Hq, Hkv, N_q, N_kv, d)),
                                    device=q.device, dtype=torch.uint8)
    with _on_device("attn_fwd_fp8", q, k, v, o, lse, signs, workspace):
        st = lib.attn_fwd_fp8(_dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"),
                              _dev_ptr(o, "o"), _dev_ptr(lse, "lse"), B, Hq, Hkv, N_q, N_kv, d,
                              int(bool(causal)), scale,
                              _dev_ptr(signs, "signs") if signs is not None else None,
                              _dev_ptr(workspace, "workspace"), workspace.numel(),
                              _stream_handle(stream, q.device), _dtype_code(q))
    _check(st, "attn_fwd_fp8")
    return o, lse


def attn_fwd_window(q, k, v, window: int, o=None, lse=None, scale: float | None = None,
                    stream=None):
    """Sliding-window prefill: key j visible to row i iff 0 <= i + N_kv - N_q - j <= window.

    Shapes and return value as attn_fwd.
    """
    B, Hq, Hkv, N_q, N_kv, d, o, lse, scale = _fwd_prep(q, k, v, o, lse, scale, stream)
    with _on_device("attn_fwd_window", q, k, v, o, lse):
        st = lib.attn_fwd_window(_dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"),
                                 _dev_ptr(o, "o"), _dev_ptr(lse, "lse"), B, Hq, Hkv, N_q, N_kv, d,
                                 int(window), scale, _stream_handle(stream, q.device),
                                 _dtype_code(q))
    _check(st, "attn_fwd_window")
    return o, lse


def attn_fwd_window_sinks(q, k, v, window: int, sinks: int, o=None, lse=None,
                          scale: float | None = None, stream=None):
    """Sliding-window prefill whose first ``sinks`` keys stay visible: key j visible to row i,
    p = i + N_kv - N_q, iff j <= p and (p - j <= window or j < sinks).

    Shapes and return value as attn_fwd.
    """
    torch = _torch()
    where = "attn_fwd_window_sinks"
    if o is not None:
        _expect(where, o, "o", q.dtype, q.shape)
    if lse is not None:
        _expect(where, lse, "lse", torch.float32, q.shape[:3])
    B, Hq, Hkv, N_q, N_kv, d, o, lse, scale = _fwd_prep(q, k, v, o, lse, scale, stream)
    index, p = _pointers(where, ("q", "k", "v", "o", "lse"), (q, k, v, o, lse))
    with _device(index):
        st = lib.attn_fwd_window_sinks(*p, B, Hq, Hkv, N_q, N_kv, d, int(window), int(sinks), scale,
                                       _stream_handle(stream, q.device), _dtype_code(q))
    _check(st, where)
    return o, lse


def attn_bwd_window_sinks_workspace_bytes(B, Hq, Hkv, N_q, N_kv, d, window, sinks) -> int:
    return int(lib.attn_bwd_window_sinks_workspace_bytes(B, Hq, Hkv, N_q, N_kv, d, int(window),
                                                         int(sinks)))


def attn_bwd_window_sinks(q, k, v, o, dout, lse, window: int, sinks: int,
                          scale: float | None = None, dq=None, dk=None, dv=None, workspace=None,
                          stream=None):
    """Gradients (dq, dk, dv) of attn_fwd_window_sinks (sinks = 0: of attn_fwd_window) for the
    incoming gradient ``dout``.  Arguments as attn_bwd with the mask of the forward call; the
    workspace takes attn_bwd_window_sinks_workspace_bytes(...) bytes.  Deterministic.
    """
    torch = _torch()
    where = "attn_bwd_window_sinks"
    B, Hq, N_q, d = q.shape
    _, Hkv, N_kv, _ = k.shape
    for t, nm, like in ((o, "o", q), (dout, "dout", q), (v, "v", k), (dq, "dq", q), (dk, "dk", k),
                        (dv, "dv", k)):
        if t is not None and (t.shape != like.shape or t.dtype != q.dtype):
            raise AttnError(-1, f"{where}: {nm} must be {tuple(like.shape)} {q.dtype}")
    if k.shape[0] != B or k.shape[3] != d or k.dtype != q.dtype:
        raise AttnError(-1, f"{where}: q/k/v shapes or dtypes disagree")
    _expect(where, lse, "lse", torch.float32, (B, Hq, N_q))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _allocating(stream, q.device):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        if workspace is None:
            need = attn_bwd_window_sinks_workspace_bytes(B, Hq, Hkv, N_q, N_kv, d, window, sinks)
            workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    index, (*p, ws) = _pointers(
        where, ("q", "k", "v", "o", "dout", "lse", "dq", "dk", "dv", "workspace"),
        (q, k, v, o, dout, lse, dq, dk, dv, workspace))
    with _device(index):
        st = lib.attn_bwd_window_sinks(*p, B, Hq, Hkv, N_q, N_kv, d, int(window), int(sinks),
                                       float(scale), _dtype_code(q), ws, workspace.nbytes,
                                       _stream_handle(stream, q.device))
    _check(st, where)
    return dq, dk, dv


def attn_fwd_block_sparse(q, k, v, block_mask, causal: bool = False, o=None, lse=None,
                          scale: float | None = None, stream=None):
    """Block-sparse prefill.  block_mask: uint8 CUDA tensor [ceil(N_q/128), ceil(N_kv/128)],
    nonzero = compute that (query tile, key tile) block.  Shapes and return value as attn_fwd.
    """
    torch = _torch()
    B, Hq, Hkv, N_q, N_kv, d, o, lse, scale = _fwd_prep(q, k, v, o, lse, scale, stream)
    shape = ((N_q + 127) // 128, (N_kv + 127) // 128)
    if (block_mask.dtype != torch.uint8 or tuple(block_mask.shape) != shape
            or not block_mask.is_contiguous()):
        raise AttnError(-1, f"attn_fwd_block_sparse: block_mask must be contiguous uint8 {shape}")
    with _on_device("attn_fwd_block_sparse", q, k, v, o, lse, block_mask):
        st = lib.attn_fwd_block_sparse(_dev_ptr(q, "q"), _dev_ptr(k, "k"), _dev_ptr(v, "v"),
                                       _dev_ptr(o, "o"), _dev_ptr(lse, "lse"), B, Hq, Hkv, N_q,
                                       N_kv, d, int(bool(causal)),
                                       _dev_ptr(block_mask, "block_mask"), scale,
                                       _stream_handle(stream, q.device), _dtype_code(q))
    _check(st, "attn_fwd_block_sparse")
    return o, lse


def attn_fwd_kv_span(q_tile: int, block_m: int, block_n: int, N_q: int, N_kv: int,
                     causal: bool, window: int = -1):
    """(j_begin, j_end, lo_masked, hi_masked) of the prefill schedule for one query tile."""
    out = [_I(0) for _ in range(4)]
    _check(lib.attn_fwd_kv_span(q_tile, block_m, block_n, N_q, N_kv, int(bool(causal)),
                                int(window), *[ctypes.byref(x) for x in out]), "attn_fwd_kv_span")
    return tuple(x.value for x in out)


def attn_decode_paged(q, k_pages, v_pages, block_table, seqlens_k, max_seqlen_k: int, o=None,
                      lse=None, split_size: int = 512, scale: float | None = None, workspace=None,
                      stream=None):
    """One split-KV decode step over a paged cache.

    q [B,Hq,d]; k_pages/v_pages [num_pages, page_size, Hkv, d]; block_table int32 CUDA
    [B, max_pages_per_seq]; seqlens_k int32 CUDA [B].  Returns (o [B,Hq,d], lse [B,Hq] fp32).
    """
    torch = _torch()
    B, Hq, d = q.shape
    num_pages, page_size, Hkv, _ = k_pages.shape
    if v_pages.shape != k_pages.shape or k_pages.dtype != q.dtype or v_pages.dtype != q.dtype:
        raise AttnError(-1, "attn_decode_paged: page pools disagree with q")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B:
        raise AttnError(-1, "attn_decode_paged: block_table must be int32 [B, max_pages]")
    if seqlens_k.dtype != torch.int32 or tuple(seqlens_k.shape) != (B,):
        raise AttnError(-1, "attn_decode_paged: seqlens_k must be int32 [B]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = attn_decode_workspace_bytes(B, Hq, max_seqlen_k, split_size, d)
    with _allocating(stream, q.device):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
        if workspace is None:
            workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    with _on_device("attn_decode_paged", q, k_pages, v_pages, block_table, seqlens_k, o, lse,
                    workspace):
        st = lib.attn_decode_paged(_dev_ptr(q, "q"), _dev_ptr(k_pages, "k_pages"),
                                   _dev_ptr(v_pages, "v_pages"),
                                   _dev_ptr(block_table, "block_table"),
                                   _dev_ptr(seqlens_k, "seqlens_k"), num_pages, page_size,
                                   block_table.shape[1], int(max_seqlen_k), _dev_ptr(o, "o"),
                                   _dev_ptr(lse, "lse"), B, Hq, Hkv, d, int(split_size),
                                   float(scale), _dtype_code(q), _dev_ptr(workspace, "workspace"),
                                   workspace.numel(), _stream_handle(stream, q.device))
    _check(st, "attn_decode_paged")
    return o, lse


def attn_fwd_paged_workspace_bytes(total_q, B, Hq, Hkv, max_seqlen_q, max_seqlen_k, d, window=-1,
                                   sinks=0) -> int:
    return int(lib.attn_fwd_paged_workspace_bytes(total_q, B, Hq, Hkv, max_seqlen_q, max_seqlen_k,
                                                  window, sinks, d))


def attn_fwd_paged(q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q: int,
                   max_seqlen_k: int, window: int = -1, sinks: int = 0, o=None, lse=None,
                   scale: float | None = None, workspace=None, stream=None):
    """A chunk of new tokens of each sequence over its paged cache, causal; the new tokens' keys
    and values are the cache's last rows already.

    q [total_q,Hq,d] packed new tokens; cu_seqlens_q int32 CUDA [B+1]; k_pages/v_pages
    [num_pages, page_size, Hkv, d]; block_table int32 CUDA [B, max_pages_per_seq]; seqlens_k int32
    CUDA [B], the new tokens included.  window (-1: none) and sinks as attn_fwd_window_sinks, by
    cache position.  Returns (o [total_q,Hq,d], lse [total_q,Hq] fp32).
    """
    torch = _torch()
    where = "attn_fwd_paged"
    total_q, Hq, d = q.shape
    num_pages, page_size, Hkv, dk = k_pages.shape
    if (v_pages.shape != k_pages.shape or dk != d or k_pages.dtype != q.dtype
            or v_pages.dtype != q.dtype):
        raise AttnError(-1, f"{where}: page pools disagree with q")
    B = seqlens_k.shape[0]
    _expect(where, seqlens_k, "seqlens_k", torch.int32, (B,))
    _expect(where, cu_seqlens_q, "cu_seqlens_q", torch.int32, (B + 1,))
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B:
        raise AttnError(-1, f"{where}: block_table must be int32 [B, max_pages]")
    if o is not None:
        _expect(where, o, "o", q.dtype, q.shape)
    if lse is not None:
        _expect(where, lse, "lse", torch.float32, (total_q, Hq))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _allocating(stream, q.device):
        o = torch.empty_like(q) if o is None else o
        if lse is None:
            lse = torch.empty((total_q, Hq), device=q.device, dtype=torch.float32)
        if workspace is None:
            need = attn_fwd_paged_workspace_bytes(total_q, B, Hq, Hkv, max_seqlen_q, max_seqlen_k, d,
                                                  window, sinks)
            workspace = torch.empty(need, device=q.device, dtype=torch.uint8) if need else None
    index, (*p, op, lp, ws) = _pointers(
        where, ("q", "k_pages", "v_pages", "block_table", "cu_seqlens_q", "seqlens_k", "o", "lse",
                "workspace"),
        (q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens_k, o, lse, workspace))
    with _device(index):
        st = lib.attn_fwd_paged(*p, num_pages, page_size, block_table.shape[1], total_q,
                                int(max_seqlen_q), int(max_seqlen_k), op, lp, B, Hq, Hkv, d,
                                int(window), int(sinks), float(scale), _dtype_code(q), ws,
                                0 if workspace is None else workspace.nbytes,
                                _stream_handle(stream, q.device))
    _check(st, where)
    return o, lse


def _check_cache_fp8(where, k_pages, v_pages, k_scales, v_scales, block_table, B):
    """The (num_pages, page_size, Hkv, d) of a quantised cache, its tensors checked."""
    torch = _torch()
    shape = k_pages.shape
    num_pages, page_size, Hkv, d = shape
    rows = (num_pages, Hkv, page_size)
    if not (k_pages.dtype == v_pages.dtype == torch.float8_e4m3fn and v_pages.shape == shape
            and k_scales.dtype == v_scales.dtype == torch.float32
            and k_scales.shape == v_scales.shape == rows):
        raise AttnError(-1, f"{where}: the pools must be float8_e4m3fn [num_pages, page_size, Hkv, d]"
                            " and their scales float32 [num_pages, Hkv, page_size]")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B:
        raise AttnError(-1, f"{where}: block_table must be int32 [B, max_pages]")
    return num_pages, page_size, Hkv, d


def attn_cache_write_fp8(k, v, k_pages, v_pages, k_scales, v_scales, block_table, cu_seqlens_q,
                         seqlens_k, stream=None) -> None:
    """New tokens into a paged cache held in 8 bits.

    k/v [total,Hkv,d] packed new tokens (fp16/bf16), sequence b's rows cu_seqlens_q[b] ..
    cu_seqlens_q[b+1]-1 going to its last cache positions; k_pages/v_pages float8_e4m3fn
    [num_pages, page_size, Hkv, d] and k_scales/v_scales fp32 [num_pages, Hkv, page_size], written
    in place; block_table int32 CUDA [B, max_pages_per_seq]; seqlens_k int32 CUDA [B], the new
    tokens included.  Each (token, head) row gets the scale 2^e, the smallest that brings its
    largest magnitude to at most 448.
    """
    torch = _torch()
    where = "attn_cache_write_fp8"
    B = seqlens_k.shape[0]
    num_pages, page_size, Hkv, d = _check_cache_fp8(where, k_pages, v_pages, k_scales, v_scales,
                                                    block_table, B)
    total = k.shape[0]
    _expect(where, k, "k", k.dtype, (total, Hkv, d))
    _expect(where, v, "v", k.dtype, (total, Hkv, d))
    _expect(where, seqlens_k, "seqlens_k", torch.int32, (B,))
    _expect(where, cu_seqlens_q, "cu_seqlens_q", torch.int32, (B + 1,))
    index, p = _pointers(
        where, ("k", "v", "k_pages", "v_pages", "k_scales", "v_scales", "block_table",
                "cu_seqlens_q", "seqlens_k"),
        (k, v, k_pages, v_pages, k_scales, v_scales, block_table, cu_seqlens_q, seqlens_k))
    with _device(index):
        st = lib.attn_cache_write_fp8(*p, num_pages, page_size, block_table.shape[1], total, B, Hkv,
                                      d, _dtype_code(k), _stream_handle(stream, k.device))
    _check(st, where)


def attn_cache_read_fp8(k_pages, v_pages, k_scales, v_scales, block_table, cu_seqlens_k, total: int,
                        dtype=None, k=None, v=None, stream=None):
    """The first tokens of each sequence of a quantised cache as a packed 16-bit cache.

    Sequence b's tokens 0 .. cu_seqlens_k[b+1]-cu_seqlens_k[b]-1 go to rows cu_seqlens_k[b] ..
    of (k, v) [total,Hkv,d], allocated here in ``dtype`` (bfloat16 when omitted) unless given.
    The cache as attn_cache_write_fp8 takes it.  Returns (k, v).
    """
    torch = _torch()
    where = "attn_cache_read_fp8"
    B = cu_seqlens_k.shape[0] - 1
    num_pages, page_size, Hkv, d = _check_cache_fp8(where, k_pages, v_pages, k_scales, v_scales,
                                                    block_table, B)
    _expect(where, cu_seqlens_k, "cu_seqlens_k", torch.int32, (B + 1,))
    if dtype is None:
        dtype = k.dtype if k is not None else v.dtype if v is not None else torch.bfloat16
    total = int(total)
    with _allocating(stream, k_pages.device):
        if k is None:
            k = torch.empty((total, Hkv, d), device=k_pages.device, dtype=dtype)
        if v is None:
            v = torch.empty((total, Hkv, d), device=k_pages.device, dtype=dtype)
    _expect(where, k, "k", dtype, (total, Hkv, d))
    _expect(where, v, "v", dtype, (total, Hkv, d))
    index, (*p, kp, vp) = _pointers(
        where, ("k_pages", "v_pages", "k_scales", "v_scales", "block_table", "cu_seqlens_k", "k",
                "v"),
        (k_pages, v_pages, k_scales, v_scales, block_table, cu_seqlens_k, k, v))
    with _device(index):
        st = lib.attn_cache_read_fp8(*p, num_pages, page_size, block_table.shape[1], kp, vp, total,
                                     B, Hkv, d, _dtype_code(k), _stream_handle(stream, k.device))
    _check(st, where)
    return k, v


def attn_decode_paged_fp8_workspace_bytes(B, Hq, Hkv, max_seqlen_k, d, split_size: int = 0) -> int:
    return int(lib.attn_decode_paged_fp8_workspace_bytes(B, Hq, Hkv, max_seqlen_k, split_size, d))


def attn_decode_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k,
                          max_seqlen_k: int, o=None, lse=None, split_size: int = 0,
                          scale: float | None = None, workspace=None, stream=None):
    """One split-KV decode step over a quantised paged cache (written by attn_cache_write_fp8).

    Arguments and return value as attn_decode_paged, with float8_e4m3fn pools and their fp32
    power-of-two scales [num_pages, Hkv, page_size].  split_size 0: the library's choice; the
    workspace takes attn_decode_paged_fp8_workspace_bytes(...) bytes (none for few splits).
    """
    torch = _torch()
    where = "attn_decode_paged_fp8"
    B, Hq, d = q.shape
    num_pages, page_size, Hkv, dk = _check_cache_fp8(where, k_pages, v_pages, k_scales, v_scales,
                                                     block_table, B)
    if dk != d:
        raise AttnError(-1, f"{where}: page pools disagree with q")
    _expect(where, seqlens_k, "seqlens_k", torch.int32, (B,))
    if o is not None:
        _expect(where, o, "o", q.dtype, q.shape)
    if lse is not None:
        _expect(where, lse, "lse", torch.float32, (B, Hq))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _allocating(stream, q.device):
        o = torch.empty_like(q) if o is None else o
        if lse is None:
            lse = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
        if workspace is None:
            need = attn_decode_paged_fp8_workspace_bytes(B, Hq, Hkv, max_seqlen_k, d, split_size)
            workspace = torch.empty(need, device=q.device, dtype=torch.uint8) if need else None
    index, (*p, op, lp, ws) = _pointers(
        where, ("q", "k_pages", "v_pages", "k_scales", "v_scales", "block_table", "seqlens_k", "o",
                "lse", "workspace"),
        (q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, o, lse, workspace))
    with _device(index):
        st = lib.attn_decode_paged_fp8(*p, num_pages, page_size, block_table.shape[1],
                                       int(max_seqlen_k), op, lp, B, Hq, Hkv, d, int(split_size),
                                       float(scale), _dtype_code(q), ws,
                                       0 if workspace is None else workspace.nbytes,
                                       _stream_handle(stream, q.device))
    _check(st, where)
    return o, lse


def attn_decode_workspace_bytes(B: int, Hq: int, max_seqlen_k: int, split_size: int, d: int) -> int:
    return int(lib.attn_decode_workspace_bytes(B, Hq, max_seqlen_k, split_size, d))


def attn_decode_splitkv(q, k_cache, v_cache, cu_seqlens_k, max_seqlen_k: int, o=None, lse=None,
                        split_size: int = 512, scale: float | None = None, workspace=None,
                        stream=None):
    """One split-KV decode step.

    q [B,Hq,d]; k_cache/v_cache [capacity,Hkv,d]; cu_seqlens_k int32 CUDA [B+1].
    ``workspace``: a uint8 CUDA tensor of at least attn_decode_workspace_bytes(...) bytes
    (allocated here when omitted).  Returns (o [B,Hq,d], lse [B,Hq] fp32).
    """
    torch = _torch()
    B, Hq, d = q.shape
    cap, Hkv, _ = k_cache.shape
    if cu_seqlens_k.dtype != torch.int32 or cu_seqlens_k.numel() != B + 1:
        raise AttnError(-1, "attn_decode_splitkv: cu_seqlens_k must be int32 [B+1]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = attn_decode_workspace_bytes(B, Hq, max_seqlen_k, split_size, d)
    with _allocating(stream, q.device):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
        if workspace is None:
            workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    with _on_device("attn_decode_splitkv", q, k_cache, v_cache, cu_seqlens_k, o, lse,
                    workspace):
        st = lib.attn_decode_splitkv(_dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"),
                                     _dev_ptr(v_cache, "v_cache"),
                                     _dev_ptr(cu_seqlens_k, "cu_seqlens_k"), cap,
                                     int(max_seqlen_k), _dev_ptr(o, "o"), _dev_ptr(lse, "lse"), B,
                                     Hq, Hkv, d, int(split_size), float(scale), _dtype_code(q),
                                     _dev_ptr(workspace, "workspace"), workspace.numel(),
                                     _stream_handle(stream, q.device))
    _check(st, "attn_decode_splitkv")
    return o, lse


def attn_decode_static_scratch_bytes() -> int:
    return int(lib.attn_decode_static_scratch_bytes())


def attn_decode_splitkv_static(q, k_cache, v_cache, cu_seqlens_k, max_seqlen_k: int, o=None,
                               lse=None, split_size: int = 512, scale: float | None = None,
                               stream=None):
    """attn_decode_splitkv without a workspace, for callers that cannot allocate device memory
    during a decode step.

    The partial states go to a fixed 32 MiB scratch array owned by the library (one per GPU,
    kept until exit); requests needing more raise AttnError(ATTN_ERR_WORKSPACE).  All calls
    share that array, so calls must not overlap on the GPU.  The first call on each GPU looks
    the array up; make it before any stream capture.  ``o`` and ``lse`` are allocated here only
    when omitted -- pass them to keep the call allocation-free.
    """
    torch = _torch()
    B, Hq, d = q.shape
    cap, Hkv, _ = k_cache.shape
    if cu_seqlens_k.dtype != torch.int32 or cu_seqlens_k.numel() != B + 1:
        raise AttnError(-1, "attn_decode_splitkv_static: cu_seqlens_k must be int32 [B+1]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _allocating(stream, q.device):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
    with _on_device("attn_decode_splitkv_static", q, k_cache, v_cache, cu_seqlens_k, o, lse):
        st = lib.attn_decode_splitkv_static(_dev_ptr(q, "q"), _dev_ptr(k_cache, "k_cache"),
                                            _dev_ptr(v_cache, "v_cache"),
                                            _dev_ptr(cu_seqlens_k, "cu_seqlens_k"), cap,
                                            int(max_seqlen_k), _dev_ptr(o, "o"),
                                            _dev_ptr(lse, "lse"), B, Hq, Hkv, d, int(split_size),
                                            float(scale), _dtype_code(q),
                                            _stream_handle(stream, q.device))
    _check(st, "attn_decode_splitkv_static")
    return o, lse


def attn_poll_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(lib.attn_poll_status(_stream_handle(stream)))


def attn_fwd_kv_tiles(q_tile: int, block_m: int, block_n: int, N_q: int, N_kv: int, causal: bool):
    """(n_tiles, first_masked) of the prefill schedule for one query tile (host only)."""
    n = _I(0)
    fm = _I(0)
    _check(lib.attn_fwd_kv_tiles(q_tile, block_m, block_n, N_q, N_kv, int(bool(causal)),
                                 ctypes.byref(n), ctypes.byref(fm)), "attn_fwd_kv_tiles")
    return n.value, fm.value


D64_AUTO, D64_PAIR, D64_SINGLE = 0, 1, 2


def attn_fwd_set_d64_kernel(mode: int) -> int:
    """Choose the d = 64 prefill kernel for later calls (D64_AUTO, D64_PAIR: two query tiles per
    work item, D64_SINGLE: one); returns the previous mode."""
    r = int(lib.attn_fwd_set_d64_kernel(int(mode)))
    if r < 0:
        raise AttnError(r, "attn_fwd_set_d64_kernel")
    return r


def attn_bwd_kv_order(B: int, Hq: int, Hkv: int, N_q: int, N_kv: int, causal: bool, n_sm: int,
                      cap: int = 2048):
    """Launch order of attn_bwd's dK/dV blocks on n_sm SMs (host only): the job of every block,
    or an empty list when the default order (job = block index) stands."""
    buf = (ctypes.c_uint16 * max(cap, 1))()
    n = _I(0)
    _check(lib.attn_bwd_kv_order(B, Hq, Hkv, N_q, N_kv, int(bool(causal)), n_sm, buf, cap,
                                 ctypes.byref(n)), "attn_bwd_kv_order")
    return list(buf[:n.value])


def attn_selftest_timeout(limit_us: int, stream=None) -> None:
    _check(lib.attn_selftest_timeout(int(limit_us), _stream_handle(stream)), "attn_selftest_timeout")
