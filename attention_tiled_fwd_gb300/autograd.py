"""Differentiable attention for PyTorch training code, built on the C ABI.

``attention(q, k, v, causal, scale)`` returns O = softmax(scale Q K^T) V and
records what the split backward needs: its ``backward`` runs fa_backward_dq
(delta = rowsum(dO * O) and dQ) and then fa_backward_dkdv (dK, dV) on the
current stream -- the training-step integration that the MLX port of
"Learning Metal with FlashAttention" lacks (its custom kernel has no
backward).  Inputs are ``[B, H, N, D]`` bf16 CUDA tensors, D any multiple of
8 up to 256; gradients come back in the inputs' dtype.  ``window_attention`` is
the same for windowed attention with grouped heads.  Nothing here computes attention:
every step runs in the library's kernels.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (FA_BF16, _c_int, _device, _device_size_query, _native, _scale, _stream_handle, fa_backward_dkdv,
               fa_backward_dq, fa_forward, fa_window_forward)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal: bool, scale: Optional[float]):
        q, k, v = (t.contiguous() for t in (q, k, v))
        o, lse = fa_forward(q, k, v, scale=scale, causal=causal)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.causal, ctx.scale = causal, scale
        return o

    @staticmethod
    def backward(ctx, dO):
        q, k, v, o, lse = ctx.saved_tensors
        dO = dO.to(q.dtype).contiguous()
        dq, delta = fa_backward_dq(q, k, v, o, dO, lse, scale=ctx.scale, causal=ctx.causal, grad_dtype=q.dtype)
        dk, dv = fa_backward_dkdv(q, k, v, dO, lse, delta, scale=ctx.scale, causal=ctx.causal,
                                  grad_dtype=q.dtype)
        return dq, dk, dv, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
              scale: Optional[float] = None) -> torch.Tensor:
    """O = softmax(scale Q K^T) V (scale defaults to 1/sqrt(D)), differentiable in q, k and v."""
    return _Attention.apply(q, k, v, bool(causal), scale)


class _WindowAttention(torch.autograd.Function):
    # The backward calls the library directly: its tensors were checked by the forward or are made here, and the
    # engine's thread runs this Python 2-3 times slower than the main thread does.
    @staticmethod
    def forward(ctx, q, k, v, window: int, sinks: int, scale: Optional[float]):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        o, lse = fa_window_forward(q, k, v, window, sinks, scale=scale)
        ctx.save_for_backward(q, k, v, o, lse)
        B, Hq, Nq, D = q.shape
        ctx.sizes = (B, Hq, k.shape[1], Nq, k.shape[2], D, _c_int(window), _c_int(sinks))
        ctx.scale = _scale(scale, D)
        if True in ctx.needs_input_grad:  # sizes that the backward refuses are refused here
            _device_size_query(_device(), "fa_window_backward_workspace_bytes", *ctx.sizes)
        return o

    @staticmethod
    def backward(ctx, dO):
        if torch.is_grad_enabled():  # the gradients would be constants in the graph that create_graph asks for
            raise RuntimeError("window_attention has no second derivatives: create_graph=True is not supported")
        q, k, v, o, lse = ctx.saved_tensors
        if dO.dtype is not q.dtype or not dO.is_contiguous():
            dO = dO.to(q.dtype).contiguous()
        if dO.data_ptr() % 16:  # a view into something else: the library reads 16-byte units
            dO = dO.clone()
        dev = _device()
        lib, stream = _native.load(), _stream_handle(None, dev)
        common = (*ctx.sizes, ctx.scale, FA_BF16, FA_BF16)
        dq = torch.empty_like(q)
        if not (ctx.needs_input_grad[1] or ctx.needs_input_grad[2]):
            delta = torch.empty_like(lse)
            rc = lib.fa_window_backward_dq(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(),
                                           lse.data_ptr(), delta.data_ptr(), dq.data_ptr(), *common, stream)
            _native.check(rc, "fa_window_backward_dq")
            return dq, None, None, None, None, None
        dk, dv = torch.empty_like(k), torch.empty_like(v)
        # delta, then the workspace, in one piece of memory
        head = (lse.numel() * 4 + 255) // 256 * 256
        need = _device_size_query(dev, "fa_window_backward_workspace_bytes", *ctx.sizes)
        scratch = torch.empty((head + need,), dtype=torch.uint8, device=q.device)  # (held until both launches are made)
        rc = lib.fa_window_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(), lse.data_ptr(),
                                    scratch.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *common,
                                    scratch.data_ptr() + head, need, stream)
        _native.check(rc, "fa_window_backward")
        return dq, dk, dv, None, None, None


def window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, sinks: int = 0,
                     scale: Optional[float] = None) -> torch.Tensor:
    """Windowed attention, differentiable in q, k and v: q [B, Hq, Nq, D] are the last Nq positions of k, v
    [B, Hkv, Nk, D] (bf16 CUDA tensors, Hq a multiple of Hkv); a row at position p sees key j iff j <= p and
    (j < sinks or j > p - window).  A row sees at most 2^21 keys, and at most 2^21 rows of a key head's query heads see a
    key in their window.  First derivatives only.  A backward pass can be captured into a CUDA graph while no
    other autograd graph of the same leaves is alive (torch synchronises with that one's stream, which ends a capture)."""
    return _WindowAttention.apply(q, k, v, int(window), int(sinks), scale)
