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
dv with Hkv heads, Hq a multiple of Hkv.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

from . import _native
from ._native import FA_BF16, FA_F32, FAError

__all__ = ["fa_forward", "fa_backward_dq", "fa_backward_dkdv", "fa_backward_atomic", "fa_decode", "fa_decode_workspace_bytes",
           "fa_decode_noalloc",
           "fa_window_forward", "fa_window_backward_dq", "fa_window_backward_dkdv", "fa_window_backward",
           "fa_window_backward_workspace_bytes",
           "fa_window_decode", "fa_window_decode_workspace_bytes", "fa_prefix_decode", "fa_prefix_decode_workspace_bytes",
           "fa_device_status", "fa_selftest_timeout", "FAError", "FA_BF16", "FA_F32", "attention_flops",
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


def _bad(t: torch.Tensor, name: str, dtype: torch.dtype, shape) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
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
