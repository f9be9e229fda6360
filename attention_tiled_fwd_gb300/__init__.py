"""Exact tiled attention on GB300: thin Python binding over libfa.so.

The functions here carry the C ABI's names (include/fa.h) and only marshal
arguments: they check tensor shapes and dtypes, allocate outputs with torch
when the caller passes none, hand raw device pointers and the current CUDA
stream to the library, and raise ``FAError`` on a non-zero status.  Every
step of the computation runs in the library's CUDA kernels; nothing falls
back to PyTorch or the CPU.

Layout: q, k, v, o, dO, dq, dk, dv are ``[B, H, N, D]`` contiguous CUDA
tensors; lse and delta are ``[B, H, N]`` float32.  The windowed and
shared-prefix calls take grouped heads: q, o, dO, dq with Hq heads, k, v, dk,
dv with Hkv heads, Hq a multiple of Hkv.  The paged calls read and write
``[n_pages, Hkv, page, D]`` pages through a table, in bf16 or in 4 bits.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct
from typing import Optional, Tuple

import torch

from . import _native
from ._native import FA_BF16, FA_F32, FA_INT4, FAError

__all__ = ["fa_forward", "fa_backward_dq", "fa_backward_dkdv", "fa_backward_atomic", "fa_decode", "fa_decode_workspace_bytes",
           "fa_decode_noalloc",
           "fa_window_forward", "fa_window_backward_dq", "fa_window_backward_dkdv", "fa_window_backward",
           "fa_window_backward_workspace_bytes",
           "fa_window_decode", "fa_window_decode_workspace_bytes", "fa_prefix_decode", "fa_prefix_decode_workspace_bytes",
           "fa_paged_append", "fa_paged_decode", "fa_paged_decode_workspace_bytes", "fa_paged_gather", "paged_cache",
           "rotation_table",
           "fa_device_status", "fa_selftest_timeout", "FAError", "FA_BF16", "FA_F32", "FA_INT4", "attention_flops",
           "attention", "window_attention"]

_DT = {torch.bfloat16: FA_BF16, torch.float32: FA_F32}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}; expected bfloat16 or float32")
    return _DT[t.dtype]


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _shape4(t: torch.Tensor, name: str):
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, H, N, D], got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return tuple(t.shape)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _scale(scale: Optional[float], D: int) -> float:
    return 1.0 / math.sqrt(D) if scale is None else float(scale)


def fa_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
               causal: bool = False, o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O = softmax(scale Q K^T) V and the natural log-sum-exp per row (fa_forward)."""
    shp = _shape4(q, "q")
    for t, n in ((k, "k"), (v, "v")):
        if _shape4(t, n) != shp or t.dtype != q.dtype:
            raise ValueError(f"{n} must match q in shape and dtype")
    B, H, N, D = shp
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    lib = _native.load()
    rc = lib.fa_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, D, _scale(scale, D),
                        int(bool(causal)), _dtype_code(q), _stream_ptr(stream))
    _native.check(rc, "fa_forward")
    return o, lse


def fa_backward_dq(q, k, v, o, dO, lse, scale: Optional[float] = None, causal: bool = False,
                   grad_dtype: torch.dtype = torch.float32, dq: Optional[torch.Tensor] = None,
                   delta: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """delta = rowsum(dO * O) and dQ (fa_backward_dq).  Returns (dq, delta)."""
    B, H, N, D = _shape4(q, "q")
    if dq is None:
        dq = torch.empty((B, H, N, D), dtype=grad_dtype, device=q.device)
    if delta is None:
        delta = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    lib = _native.load()
    rc = lib.fa_backward_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(delta), _ptr(dq),
                            B, H, N, D, _scale(scale, D), int(bool(causal)), _dtype_code(q),
                            _dtype_code(dq), _stream_ptr(stream))
    _native.check(rc, "fa_backward_dq")
    return dq, delta


def fa_backward_dkdv(q, k, v, dO, lse, delta, scale: Optional[float] = None, causal: bool = False,
                     grad_dtype: torch.dtype = torch.float32, dk: Optional[torch.Tensor] = None,
                     dv: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """dK and dV (fa_backward_dkdv).  Returns (dk, dv)."""
    B, H, N, D = _shape4(q, "q")
    if dk is None:
        dk = torch.empty((B, H, N, D), dtype=grad_dtype, device=q.device)
    if dv is None:
        dv = torch.empty((B, H, N, D), dtype=grad_dtype, device=q.device)
    if dk.dtype != dv.dtype:
        raise ValueError("dk and dv must share a dtype")
    lib = _native.load()
    rc = lib.fa_backward_dkdv(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(lse), _ptr(delta), _ptr(dk), _ptr(dv),
                              B, H, N, D, _scale(scale, D), int(bool(causal)), _dtype_code(q),
                              _dtype_code(dk), _stream_ptr(stream))
    _native.check(rc, "fa_backward_dkdv")
    return dk, dv


def fa_backward_atomic(q, k, v, o, dO, lse, scale: Optional[float] = None, causal: bool = False,
                       grad_dtype: torch.dtype = torch.float32, dq_accum: Optional[torch.Tensor] = None,
                       dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                       dv: Optional[torch.Tensor] = None, delta: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None):
    """The 5-GEMM comparator backward (fa_backward_atomic).  Returns (dq, dk, dv, delta).

    dq_accum is an fp32 CUDA tensor of at least B*H*N*D elements; outputs and dq_accum are
    allocated here when the caller passes none (dq, dk, dv in grad_dtype unless given)."""
    B, H, N, D = _shape4(q, "q")
    if dq is None:
        dq = torch.empty((B, H, N, D), dtype=grad_dtype, device=q.device)
    if dk is None:
        dk = torch.empty_like(dq)
    if dv is None:
        dv = torch.empty_like(dq)
    if not (dq.dtype == dk.dtype == dv.dtype):
        raise ValueError("dq, dk and dv must share a dtype")
    if delta is None:
        delta = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if dq_accum is None:
        dq_accum = torch.empty((B, H, N, D), dtype=torch.float32, device=q.device)
    lib = _native.load()
    rc = lib.fa_backward_atomic(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(delta), _ptr(dq),
                                _ptr(dk), _ptr(dv), _ptr(dq_accum), dq_accum.numel() * dq_accum.element_size(),
                                B, H, N, D, _scale(scale, D), int(bool(causal)), _dtype_code(q), _dtype_code(dq),
                                _stream_ptr(stream))
    _native.check(rc, "fa_backward_atomic")
    return dq, dk, dv, delta


def fa_decode_workspace_bytes(B: int, H: int, n_q: int, N: int, D: int) -> int:
    """Workspace bytes fa_decode needs (fa_decode_workspace_bytes)."""
    import ctypes
    out = ctypes.c_size_t(0)
    _native.check(_native.load().fa_decode_workspace_bytes(B, H, n_q, N, D, ctypes.byref(out)),
                  "fa_decode_workspace_bytes")
    return int(out.value)


def fa_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
              causal: bool = False, o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Decode: q [B, H, n_q, D] (the last n_q positions) against k, v [B, H, N, D] (fa_decode).

    The workspace is a CUDA uint8 tensor of at least fa_decode_workspace_bytes(...) bytes; one is
    allocated here when the caller passes none.  Returns (o, lse)."""
    B, H, nq, D = _shape4(q, "q")
    Bk, Hk, N, Dk = _shape4(k, "k")
    if (Bk, Hk, Dk) != (B, H, D) or _shape4(v, "v") != (B, H, N, D):
        raise ValueError("k and v must be [B, H, N, D] matching q's B, H, D")
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, nq), dtype=torch.float32, device=q.device)
    need = fa_decode_workspace_bytes(B, H, nq, N, D)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    lib = _native.load()
    rc = lib.fa_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, nq, N, D, _scale(scale, D),
                       int(bool(causal)), _ptr(workspace), workspace.numel() * workspace.element_size(),
                       _stream_ptr(stream))
    _native.check(rc, "fa_decode")
    return o, lse


def fa_decode_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                      scale: Optional[float] = None, causal: bool = False,
                      stream: Optional[torch.cuda.Stream] = None):
    """fa_decode with no workspace (fa_decode_noalloc): the partials go to the library's fixed
    per-device scratch, so the call allocates nothing; the caller passes the outputs o
    [B, H, n_q, D] bf16 and lse [B, H, n_q] fp32.  Calls that overlap in time on one device race on
    that scratch; sizes needing more than FA_DECODE_NOALLOC_SCRATCH_BYTES raise FAError
    (FA_ERR_SCRATCH_LIMIT).  Returns (o, lse)."""
    B, H, nq, D = _shape4(q, "q")
    Bk, Hk, N, Dk = _shape4(k, "k")
    if (Bk, Hk, Dk) != (B, H, D) or _shape4(v, "v") != (B, H, N, D):
        raise ValueError("k and v must be [B, H, N, D] matching q's B, H, D")
    if _shape4(o, "o") != (B, H, nq, D) or tuple(lse.shape) != (B, H, nq):
        raise ValueError("o must be [B, H, n_q, D] and lse [B, H, n_q]")
    rc = _native.load().fa_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, nq, N, D,
                                          _scale(scale, D), int(bool(causal)), _stream_ptr(stream))
    _native.check(rc, "fa_decode_noalloc")
    return o, lse


# The calls below run in 10-30 us on the device at their smallest, so the binding's own time counts: one comparison
# per tensor when all is well (_bad says what is not), the current stream's handle without a Stream object, and no
# size query when the caller brings the workspace.
def _bf16(t: torch.Tensor, name: str, shape, device: int) -> None:
    """t is a contiguous bf16 CUDA tensor of this shape on the current device."""
    if t.shape != shape or t.dtype is not torch.bfloat16 or t.get_device() != device or not t.is_contiguous():
        _bad(t, name, torch.bfloat16, shape)


def _tensor(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device: int) -> None:
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        _bad(t, name, dtype, shape)


def _bad(t: torch.Tensor, name: str, dtype: torch.dtype, shape, contiguous: bool = True) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on the current CUDA device, got {t.device}")


def _device() -> int:
    return torch.cuda.current_device()


def _stream_handle(stream: Optional[torch.cuda.Stream], device: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError(f"stream must belong to the current CUDA device, got {stream.device}")
    return stream.cuda_stream


def _no_c_int(where: str) -> None:
    """A size that the C interface's int cannot hold (ctypes would pass on its low 32 bits)."""
    raise FAError(_native.FA_ERR_SHAPE, where)


def _grouped(q: torch.Tensor, k: torch.Tensor):
    """Sizes (B, Hq, Nq, D, Hkv, rows of k) of grouped-head tensors."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"q and k must have 4 dimensions, got {list(q.shape)} and {list(k.shape)}")
    (B, Hq, Nq, D), (_, Hkv, rows, _) = q.shape, k.shape
    if (B | Hq | Nq | D | Hkv | rows) >> 31:
        _no_c_int("a size of q or k")
    if Hkv < 1 or Hq % Hkv != 0:
        raise ValueError(f"q's {Hq} heads must be a multiple of k's {Hkv}")
    return B, Hq, Nq, D, Hkv, rows


def _c_int(x: int) -> int:
    """A window or sink count as a C int (anything longer than every sequence is the same mask)."""
    return max(-1, min(int(x), (1 << 31) - 1))


def _empty(like: torch.Tensor, shape, dtype: torch.dtype, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """Memory of the stream that the call runs on, so that the allocator hands it on in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _empty_like(like: torch.Tensor, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    return torch.empty_like(like) if stream is None else _empty(like, like.shape, like.dtype, stream)


def _size_query(name: str, *sizes: int) -> int:
    for n in sizes:
        if n >> 31:
            _no_c_int(name)
    out = ctypes.c_size_t(0)
    _native.check(getattr(_native.load(), name)(*sizes, ctypes.byref(out)), name)
    return int(out.value)


@functools.lru_cache(maxsize=1024)
def _device_size_query(device: int, name: str, *sizes: int) -> int:
    """The same number every time: it depends on the sizes and on the current device's SM count alone."""
    return _size_query(name, *sizes)


def _workspace(workspace: Optional[torch.Tensor], like: torch.Tensor, stream, device: int, query: str, *sizes: int):
    """The caller's workspace, or a new one of the size that the library asks for; None when it asks for nothing."""
    if workspace is None:
        need = _device_size_query(device, query, *sizes)
        return _empty(like, (need,), torch.uint8, stream) if need else None
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the current CUDA device")
    return workspace


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def fa_window_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, sinks: int = 0,
                      scale: Optional[float] = None, kv_len: Optional[int] = None, o: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Windowed attention (fa_window_forward): q [B, Hq, Nq, D] are the last Nq of Nk positions; a row at position p
    sees key j iff j <= p and (j < sinks or j > p - window).

    k, v are [B, Hkv, rows, D]; the first kv_len rows (default: all) of each head are the Nk keys.  bf16.
    Returns (o, lse)."""
    B, Hq, Nq, D, Hkv, rows = _grouped(q, k)
    Nk = rows if kv_len is None else int(kv_len)
    if Nk >> 31:
        _no_c_int("kv_len")
    dev = _device()
    _bf16(q, "q", (B, Hq, Nq, D), dev)
    _bf16(k, "k", (B, Hkv, rows, D), dev)
    _bf16(v, "v", (B, Hkv, rows, D), dev)
    if o is None:
        o = _empty_like(q, stream)
    else:
        _bf16(o, "o", q.shape, dev)
    if lse is None:
        lse = _empty(q, (B, Hq, Nq), torch.float32, stream)
    else:
        _tensor(lse, "lse", torch.float32, (B, Hq, Nq), dev)
    rc = _native.load().fa_window_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq,
                                          Hkv, Nq, Nk, rows, D, _c_int(window), _c_int(sinks), _scale(scale, D),
                                          FA_BF16, _stream_handle(stream, dev))
    _native.check(rc, "fa_window_forward")
    return o, lse


def fa_window_backward_dq(q, k, v, o, dO, lse, window: int, sinks: int = 0, scale: Optional[float] = None,
                          grad_dtype: torch.dtype = torch.float32, dq: Optional[torch.Tensor] = None,
                          delta: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """delta = rowsum(dO * O) (the first 128 positions: sum P dP) and dQ of windowed attention (fa_window_backward_dq).
    Returns (dq, delta)."""
    B, Hq, Nq, D, Hkv, Nk = _grouped(q, k)
    dev = _device()
    rows, keys = (B, Hq, Nq, D), (B, Hkv, Nk, D)
    for t, n, shape in ((q, "q", rows), (k, "k", keys), (v, "v", keys), (o, "o", rows), (dO, "dO", rows)):
        _bf16(t, n, shape, dev)
    _tensor(lse, "lse", torch.float32, (B, Hq, Nq), dev)
    if dq is None:
        dq = _empty(q, q.shape, grad_dtype, stream)
    code = _dtype_code(dq)
    _tensor(dq, "dq", dq.dtype, q.shape, dev)
    if delta is None:
        delta = _empty(q, (B, Hq, Nq), torch.float32, stream)
    else:
        _tensor(delta, "delta", torch.float32, (B, Hq, Nq), dev)
    rc = _native.load().fa_window_backward_dq(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(),
                                              lse.data_ptr(), delta.data_ptr(), dq.data_ptr(), B, Hq, Hkv, Nq, Nk, D,
                                              _c_int(window), _c_int(sinks), _scale(scale, D), FA_BF16, code,
                                              _stream_handle(stream, dev))
    _native.check(rc, "fa_window_backward_dq")
    return dq, delta


def fa_window_backward_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, D: int, window: int,
                                       sinks: int) -> int:
    """Workspace bytes fa_window_backward_dkdv needs (may be 0)."""
    return _size_query("fa_window_backward_workspace_bytes", B, Hq, Hkv, Nq, Nk, D, _c_int(window),
                       _c_int(sinks))


def fa_window_backward_dkdv(q, k, v, dO, lse, delta, window: int, sinks: int = 0, scale: Optional[float] = None,
                            grad_dtype: torch.dtype = torch.float32, dk: Optional[torch.Tensor] = None,
                            dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None):
    """dK and dV of windowed attention, summed over each key head's query heads (fa_window_backward_dkdv).

    A workspace of fa_window_backward_workspace_bytes(...) bytes is allocated here when the caller passes none.
    Returns (dk, dv)."""
    B, Hq, Nq, D, Hkv, Nk = _grouped(q, k)
    dev = _device()
    rows, keys = (B, Hq, Nq, D), (B, Hkv, Nk, D)
    for t, n, shape in ((q, "q", rows), (k, "k", keys), (v, "v", keys), (dO, "dO", rows)):
        _bf16(t, n, shape, dev)
    _tensor(lse, "lse", torch.float32, (B, Hq, Nq), dev)
    _tensor(delta, "delta", torch.float32, (B, Hq, Nq), dev)
    if dk is None:
        dk = _empty(k, k.shape, grad_dtype, stream)
    if dv is None:
        dv = _empty(k, k.shape, grad_dtype, stream)
    code = _dtype_code(dk)
    _tensor(dk, "dk", dk.dtype, k.shape, dev)
    _tensor(dv, "dv", dk.dtype, k.shape, dev)
    window, sinks = _c_int(window), _c_int(sinks)
    workspace = _workspace(workspace, q, stream, dev, "fa_window_backward_workspace_bytes", B, Hq, Hkv, Nq, Nk, D, window,
                           sinks)
    rc = _native.load().fa_window_backward_dkdv(q.data_ptr(), k.data_ptr(), v.data_ptr(), dO.data_ptr(), lse.data_ptr(),
                                                delta.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Nq, Nk, D,
                                                window, sinks, _scale(scale, D), FA_BF16, code, _ptr(workspace),
                                                _nbytes(workspace), _stream_handle(stream, dev))
    _native.check(rc, "fa_window_backward_dkdv")
    return dk, dv


def fa_window_backward(q, k, v, o, dO, lse, window: int, sinks: int = 0, scale: Optional[float] = None,
                       grad_dtype: torch.dtype = torch.float32, dq: Optional[torch.Tensor] = None,
                       dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                       delta: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None):
    """fa_window_backward_dq and fa_window_backward_dkdv in one call (fa_window_backward).  Returns (dq, dk, dv, delta)."""
    B, Hq, Nq, D, Hkv, Nk = _grouped(q, k)
    dev = _device()
    rows, keys = (B, Hq, Nq, D), (B, Hkv, Nk, D)
    for t, n, shape in ((q, "q", rows), (k, "k", keys), (v, "v", keys), (o, "o", rows), (dO, "dO", rows)):
        _bf16(t, n, shape, dev)
    _tensor(lse, "lse", torch.float32, (B, Hq, Nq), dev)
    if dq is None:
        dq = _empty(q, q.shape, grad_dtype, stream)
    if dk is None:
        dk = _empty(k, k.shape, dq.dtype, stream)
    if dv is None:
        dv = _empty(k, k.shape, dq.dtype, stream)
    code = _dtype_code(dq)
    for t, n, shape in ((dq, "dq", rows), (dk, "dk", keys), (dv, "dv", keys)):
        _tensor(t, n, dq.dtype, shape, dev)
    if delta is None:
        delta = _empty(q, (B, Hq, Nq), torch.float32, stream)
    else:
        _tensor(delta, "delta", torch.float32, (B, Hq, Nq), dev)
    window, sinks = _c_int(window), _c_int(sinks)
    workspace = _workspace(workspace, q, stream, dev, "fa_window_backward_workspace_bytes", B, Hq, Hkv, Nq, Nk, D, window,
                           sinks)
    rc = _native.load().fa_window_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(),
                                           lse.data_ptr(), delta.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                           B, Hq, Hkv, Nq, Nk, D, window, sinks, _scale(scale, D), FA_BF16, code,
                                           _ptr(workspace), _nbytes(workspace), _stream_handle(stream, dev))
    _native.check(rc, "fa_window_backward")
    return dq, dk, dv, delta


def _rows_and_cache(q, k, v, lens, o, lse, stream):
    """(B, Hq, Hkv, n_q), N, D, the outputs and the device of a decode call, its tensors checked."""
    B, Hq, n_q, D, Hkv, N = _grouped(q, k)
    dev = _device()
    _bf16(q, "q", (B, Hq, n_q, D), dev)
    _bf16(k, "k", (B, Hkv, N, D), dev)
    _bf16(v, "v", (B, Hkv, N, D), dev)
    if lens is not None:
        _tensor(lens, "lens", torch.int32, (B,), dev)
    if o is None:
        o = _empty_like(q, stream)
    else:
        _bf16(o, "o", q.shape, dev)
    if lse is None:
        lse = _empty(q, (B, Hq, n_q), torch.float32, stream)
    else:
        _tensor(lse, "lse", torch.float32, (B, Hq, n_q), dev)
    return (B, Hq, Hkv, n_q), N, D, o, lse, dev


def fa_window_decode_workspace_bytes(B: int, Hq: int, Hkv: int, n_q: int, N: int, D: int, window: int,
                                     sinks: int) -> int:
    """Workspace bytes fa_window_decode needs (may be 0)."""
    return _size_query("fa_window_decode_workspace_bytes", B, Hq, Hkv, n_q, N, D, _c_int(window),
                       _c_int(sinks))


def fa_window_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, sinks: int = 0,
                     lens: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """The n_q <= 16 newest rows q [B, Hq, n_q, D] of each sequence against its cache k, v [B, Hkv, N, D], windowed
    (fa_window_decode).  lens: int32 CUDA tensor [B], the keys each sequence holds (default N).  Returns (o, lse)."""
    heads, N, D, o, lse, dev = _rows_and_cache(q, k, v, lens, o, lse, stream)
    window, sinks = _c_int(window), _c_int(sinks)
    workspace = _workspace(workspace, q, stream, dev, "fa_window_decode_workspace_bytes", *heads, N, D, window, sinks)
    rc = _native.load().fa_window_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(lens), o.data_ptr(),
                                         lse.data_ptr(), *heads, N, D, window, sinks, _scale(scale, D), _ptr(workspace),
                                         _nbytes(workspace), _stream_handle(stream, dev))
    _native.check(rc, "fa_window_decode")
    return o, lse


def fa_prefix_decode_workspace_bytes(B: int, Hq: int, Hkv: int, n_q: int, P: int, N: int, D: int) -> int:
    """Workspace bytes fa_prefix_decode needs."""
    return _size_query("fa_prefix_decode_workspace_bytes", B, Hq, Hkv, n_q, P, N, D)


def fa_prefix_decode(q: torch.Tensor, k_prefix: torch.Tensor, v_prefix: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     lens: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """The n_q <= 16 newest rows q [B, Hq, n_q, D] of each sequence against the prefix k_prefix, v_prefix [Hkv, P, D]
    that all sequences share, and against the sequence's own cache k, v [B, Hkv, N, D] behind it, of which lens[b]
    keys are held (int32 CUDA tensor; default N) (fa_prefix_decode).  Returns (o, lse)."""
    if k_prefix.dim() != 3:
        raise ValueError(f"k_prefix must be [Hkv, P, D], got {list(k_prefix.shape)}")
    P = k_prefix.shape[1]
    if P >> 31:
        _no_c_int("k_prefix's length")
    heads, N, D, o, lse, dev = _rows_and_cache(q, k, v, lens, o, lse, stream)
    _bf16(k_prefix, "k_prefix", (heads[2], P, D), dev)
    _bf16(v_prefix, "v_prefix", (heads[2], P, D), dev)
    workspace = _workspace(workspace, q, stream, dev, "fa_prefix_decode_workspace_bytes", *heads, P, N, D)
    rc = _native.load().fa_prefix_decode(q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), k.data_ptr(),
                                         v.data_ptr(), _ptr(lens), o.data_ptr(), lse.data_ptr(), *heads, P, N, D,
                                         _scale(scale, D), _ptr(workspace), _nbytes(workspace),
                                         _stream_handle(stream, dev))
    _native.check(rc, "fa_prefix_decode")
    return o, lse


# A paged cache: two tensors k_pages, v_pages of bf16 [n_pages, Hkv, page, D], or of bytes [n_pages, Hkv, page, 9 D / 16]
# (4 bits a value and a scale for 32 of them; include/fa.h has the order), a page table and the sequences' lengths.
def paged_cache(n_pages: int, heads: int, page: int, D: int, dtype: int = FA_BF16,
                device: Optional[torch.device] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Zeroed pages for the keys and the values of `heads` key heads: FA_BF16 or FA_INT4 (4 bits a value)."""
    if dtype not in (FA_BF16, FA_INT4):
        raise ValueError(f"dtype must be FA_BF16 or FA_INT4, got {dtype}")
    shape = (n_pages, heads, page, D if dtype == FA_BF16 else 9 * D // 16)
    kind = torch.bfloat16 if dtype == FA_BF16 else torch.uint8
    device = torch.device("cuda") if device is None else device
    return torch.zeros(shape, dtype=kind, device=device), torch.zeros(shape, dtype=kind, device=device)


def rotation_table(positions: int, rot: int, base: float = 10000.0,
                   device: Optional[torch.device] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """cos and sin [positions, rot / 2] fp32 of the angles p * base ** (-2 i / rot), taken in 64 bits."""
    if rot % 2 != 0:
        raise ValueError(f"rot must be even, got {rot}")
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * torch.pow(torch.tensor(base, dtype=torch.float64), -i / rot)
    device = torch.device("cuda") if device is None else device
    return angle.cos().float().to(device), angle.sin().float().to(device)


def _pages(k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor, lens: Optional[torch.Tensor], B: int,
           device: int):
    """D, Hkv, n_pages, page, slots and the type of a paged cache, its tensors checked."""
    shape = k_pages.shape
    if len(shape) != 4 or table.dim() != 2:
        raise ValueError(f"k_pages must have 4 dimensions and table 2, got {list(shape)} and {list(table.shape)}")
    n_pages, Hkv, page, row = shape
    slots = table.shape[1]
    if (n_pages | Hkv | page | row | slots | B) >> 31:
        _no_c_int("a size of the pages or the table")
    dtype = k_pages.dtype
    if dtype is torch.bfloat16:
        D, kind = row, FA_BF16
    elif dtype is torch.uint8:
        D, kind = row * 16 // 9, FA_INT4
        if row % 9 != 0:
            raise ValueError(f"4-bit pages have 9 D / 16 bytes a position, got {row}")
    else:
        raise TypeError(f"k_pages must be bfloat16, or uint8 for 4-bit pages, got {dtype}")
    if k_pages.get_device() != device or not k_pages.is_contiguous():
        _bad(k_pages, "k_pages", dtype, shape)
    if v_pages.shape != shape or v_pages.dtype is not dtype or v_pages.get_device() != device or not v_pages.is_contiguous():
        _bad(v_pages, "v_pages", dtype, shape)
    _tensor(table, "table", torch.int32, (B, slots), device)
    if lens is not None:
        _tensor(lens, "lens", torch.int32, (B,), device)
    return D, Hkv, n_pages, page, slots, kind


_NINE = struct.Struct("9q").pack  # nine strides as C's long long


def _rows(t: torch.Tensor, name: str, shape, device: int):
    """The strides between sequences, heads and rows of bf16 rows [B, H, n, D] whose D channels are neighbours."""
    if t.shape != shape or t.dtype is not torch.bfloat16 or t.get_device() != device:
        _bad(t, name, torch.bfloat16, shape, contiguous=False)
    strides = t.stride()
    if strides[3] != 1 and shape[3] > 1:
        raise ValueError(f"{name}'s channels must be neighbours, got strides {list(strides)}")
    return strides


def fa_paged_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
                    lens: torch.Tensor, q: Optional[torch.Tensor] = None, cos: Optional[torch.Tensor] = None,
                    sin: Optional[torch.Tensor] = None, interleaved: bool = False, counts: Optional[torch.Tensor] = None,
                    q_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """The n newest rows of each sequence into its pages, rotated by their positions (fa_paged_append).

    k, v [B, Hkv, n, D] and q [B, Hq, n, D] are bf16 views of any strides (multiples of 8) with neighbouring channels, such
    as parts of one projection's output.  lens: int32 [B], the keys each sequence holds with these rows; counts: int32 [B],
    how many of the n rows (the last ones) are new.  cos, sin: fp32 [positions, rot / 2] (rotation_table), None: no
    rotation.  Returns q rotated and contiguous (None without q)."""
    shape = k.shape
    if len(shape) != 4:
        raise ValueError(f"k must be [B, Hkv, n, D], got {list(shape)}")
    if lens is None:
        raise ValueError("lens is needed: it says where the rows go")
    B, Hkv, n, D = shape
    dev = _device()
    row, heads, n_pages, page, slots, kind = _pages(k_pages, v_pages, table, lens, B, dev)
    if row != D or heads != Hkv:
        raise ValueError(f"the pages hold {heads} heads of {row}, got k {list(shape)}")
    if (n | D) >> 31:
        _no_c_int("a size of k")
    ks, vs = _rows(k, "k", shape, dev), _rows(v, "v", shape, dev)
    if q is not None:
        if q.dim() != 4 or q.shape[1] < 1 or q.shape[1] >> 31:
            raise ValueError(f"q must be [B, Hq, n, D], got {list(q.shape)}")
        Hq = q.shape[1]
        qs, q_ptr = _rows(q, "q", (B, Hq, n, D), dev), q.data_ptr()
        if q_out is None:
            q_out = _empty(q, (B, Hq, n, D), torch.bfloat16, stream)
            out_ptr = q_out.data_ptr()
        else:
            _bf16(q_out, "q_out", (B, Hq, n, D), dev)
            out_ptr = q_out.data_ptr()
            if out_ptr == q_ptr:
                raise ValueError("q_out must not be q")
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    else:
        Hq, q_ptr, out_ptr, qs = 0, None, None, ks
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is not None:
        angles = cos.shape
        if len(angles) != 2:
            raise ValueError(f"cos must be [positions, rot / 2], got {list(angles)}")
        positions, rot = angles[0], 2 * angles[1]
        if (positions | rot) >> 31:
            _no_c_int("a size of cos")
        _tensor(cos, "cos", torch.float32, angles, dev)
        _tensor(sin, "sin", torch.float32, angles, dev)
        cos_ptr, sin_ptr = cos.data_ptr(), sin.data_ptr()
    else:
        positions = rot = 0
        cos_ptr = sin_ptr = None
    if counts is not None:
        _tensor(counts, "counts", torch.int32, (B,), dev)
    rc = _native.load().fa_paged_append(q_ptr, k.data_ptr(), v.data_ptr(), _NINE(*qs[:3], *ks[:3], *vs[:3]), cos_ptr, sin_ptr,
                                        table.data_ptr(), lens.data_ptr(), _ptr(counts), out_ptr, k_pages.data_ptr(),
                                        v_pages.data_ptr(), B, Hq, Hkv, n, D, rot, 1 if interleaved else 0, positions, n_pages,
                                        page, slots, kind, _stream_handle(stream, dev))
    if rc:
        _native.check(rc, "fa_paged_append")
    return q_out


def fa_paged_decode_workspace_bytes(B: int, Hq: int, Hkv: int, n_q: int, D: int, page: int, slots: int,
                                    dtype: int = FA_BF16) -> int:
    """Workspace bytes fa_paged_decode needs (may be 0; never more than 16 MB)."""
    return _size_query("fa_paged_decode_workspace_bytes", B, Hq, Hkv, n_q, D, page, slots, dtype)


def fa_paged_decode(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
                    lens: Optional[torch.Tensor] = None, window: Optional[int] = None, sinks: int = 0,
                    scale: Optional[float] = None, o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """The n_q <= 16 newest rows q [B, Hq, n_q, D] of each sequence against its pages (fa_paged_decode).

    table: int32 [B, slots], the sequences' pages; lens: int32 [B], the keys each holds (default: all its pages);
    window None: every earlier key.  Returns (o, lse)."""
    shape = q.shape
    if len(shape) != 4:
        raise ValueError(f"q must be [B, Hq, n_q, D], got {list(shape)}")
    B, Hq, n_q, D = shape
    dev = _device()
    row, Hkv, n_pages, page, slots, kind = _pages(k_pages, v_pages, table, lens, B, dev)
    if row != D or Hkv < 1 or Hq % Hkv != 0:
        raise ValueError(f"the pages hold {Hkv} heads of {row}, got q {list(shape)}")
    if (Hq | n_q) >> 31:
        _no_c_int("a size of q")
    _bf16(q, "q", shape, dev)
    if o is None:
        o = _empty_like(q, stream)
    else:
        _bf16(o, "o", shape, dev)
    if lse is None:
        lse = _empty(q, (B, Hq, n_q), torch.float32, stream)
    else:
        _tensor(lse, "lse", torch.float32, (B, Hq, n_q), dev)
    workspace = _workspace(workspace, q, stream, dev, "fa_paged_decode_workspace_bytes", B, Hq, Hkv, n_q, D, page, slots, kind)
    rc = _native.load().fa_paged_decode(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), _ptr(lens),
                                        o.data_ptr(), lse.data_ptr(), B, Hq, Hkv, n_q, D, n_pages, page, slots,
                                        slots * page if window is None else _c_int(window), _c_int(sinks) if sinks else 0,
                                        _scale(scale, D), kind, _ptr(workspace), _nbytes(workspace), _stream_handle(stream, dev))
    if rc:
        _native.check(rc, "fa_paged_decode")
    return o, lse


def fa_paged_gather(k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor, lens: Optional[torch.Tensor] = None,
                    rows: Optional[int] = None, k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None):
    """The sequences' rows out of their pages (fa_paged_gather): k, v [B, Hkv, rows, D] bf16 (rows: default all of a
    sequence's pages), of which the first min(lens[b], rows) are written.  Returns (k, v)."""
    if table.dim() != 2:
        raise ValueError(f"table must be [B, slots], got {list(table.shape)}")
    B = table.shape[0]
    dev = _device()
    D, Hkv, n_pages, page, slots, kind = _pages(k_pages, v_pages, table, lens, B, dev)
    if (k is None) != (v is None):
        raise ValueError("k and v come together")
    if k is None:
        shape = (B, Hkv, slots * page if rows is None else rows, D)
        k, v = (_empty(k_pages, shape, torch.bfloat16, stream) for _ in range(2))
    else:
        if k.dim() != 4 or (rows is not None and k.shape[2] != rows):
            raise ValueError(f"k must be [B, Hkv, rows, D], got {list(k.shape)}")
        shape = (B, Hkv, k.shape[2], D)
        _bf16(k, "k", shape, dev)
        _bf16(v, "v", shape, dev)
    if shape[2] >> 31:
        _no_c_int("rows")
    rc = _native.load().fa_paged_gather(k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), _ptr(lens), k.data_ptr(),
                                        v.data_ptr(), B, Hkv, shape[2], D, n_pages, page, slots, kind,
                                        _stream_handle(stream, dev))
    _native.check(rc, "fa_paged_gather")
    return k, v


def fa_device_status(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return _native.load().fa_device_status(_stream_ptr(stream))


def fa_selftest_timeout(limit_us: int, stream: Optional[torch.cuda.Stream] = None) -> None:
    _native.check(_native.load().fa_selftest_timeout(int(limit_us), _stream_ptr(stream)), "fa_selftest_timeout")


def attention_flops(B: int, H: int, N: int, D: int, causal: bool, pass_: str = "fwd") -> float:
    """Algorithmic FLOPs: forward 4 B H N^2 D (two N x N x D GEMMs); the split
    backward counted as its 7 GEMMs, 14 B H N^2 D; both halved when causal."""
    per = {"fwd": 4.0, "bwd": 14.0, "bwd_dq": 6.0, "bwd_dkdv": 8.0}[pass_]
    f = per * B * H * float(N) * N * D
    return f / 2 if causal else f


from .autograd import attention, window_attention  # noqa: E402  (differentiable wrapper over the functions above)
