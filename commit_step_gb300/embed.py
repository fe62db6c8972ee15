"""The embedding of a canvas and its gradient (``dllm_embed_tokens``,
``dllm_embed_tokens_backward``)."""
from __future__ import annotations

from typing import Optional

import torch

from . import DLLM_BF16, DLLM_F32, _check, _lib, _need_cuda
from .cache import _raw_stream
from .head import _may_capture, _size, _stamp, _workspace


_DTYPES = {torch.bfloat16: DLLM_BF16, torch.float32: DLLM_F32}


def _dtype(t, name: str) -> int:
    code = _DTYPES.get(t.dtype) if torch.is_tensor(t) else None
    if code is None:
        raise TypeError(f"{name} must be a bfloat16 or float32 tensor")
    return code


def _canvas(tokens, index: int):
    """(B, L, row stride) of (T,) or (B, L) int32 tokens, unit stride over the last dimension."""
    if not torch.is_tensor(tokens) or tokens.dtype != torch.int32 or tokens.dim() not in (1, 2):
        raise TypeError("tokens must be a (T,) or (B, L) int32 tensor")
    if tokens.get_device() != index:
        raise ValueError(f"tokens are on {tokens.device}; the call runs on cuda:{index}")
    shape, strides = tokens.shape, tokens.stride()
    L = shape[-1]
    if L > 1 and strides[-1] != 1:
        raise ValueError("tokens need unit stride over their last dimension")
    if len(shape) == 1:
        return 1, L, L
    return shape[0], L, (strides[0] if shape[0] > 1 else L)


def _weight(t, name: str, V: int, d: int) -> int:
    """The row stride of a (V, d) tensor with unit column stride."""
    if t.dim() != 2 or t.shape != (V, d):
        raise ValueError(f"{name} must be (V, d) = ({V}, {d})")
    stride, unit = t.stride()
    if d > 1 and unit != 1:
        raise ValueError(f"{name} needs unit column stride")
    return stride if V > 1 else d


def embed_tokens(tokens: torch.Tensor, weight: torch.Tensor, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                 stream=None):
    """scale * weight[tokens]: (..., d) in weight's dtype, contiguous.

    ``tokens``: (T,) or (B, L) int32, rows at any stride (a window of a longer
    canvas); an id outside [0, V) gives zeros.  ``weight``: (V, d) bf16 or fp32.
    ``out``: preallocated."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return embed_tokens(tokens, weight, scale, out)
    dt, idx = _dtype(weight, "weight"), weight.get_device()
    if idx < 0:
        raise ValueError("device tensors are required")
    if weight.dim() != 2:
        raise ValueError("weight must be (V, d)")
    (V, d), (stride, unit) = weight.shape, weight.stride()
    if d > 1 and unit != 1:
        raise ValueError("weight needs unit column stride")
    B, L, t_stride = _canvas(tokens, idx)
    if out is None:
        out = torch.empty((*tokens.shape, d), dtype=weight.dtype, device=weight.device)
    elif (not torch.is_tensor(out) or out.dtype != weight.dtype or out.get_device() != idx
          or out.shape != (*tokens.shape, d) or not out.is_contiguous()):
        raise ValueError("out must be a contiguous (..., d) tensor of weight's dtype, on the same device")
    _check(_lib.dllm_embed_tokens(tokens.data_ptr(), B, L, t_stride, weight.data_ptr(), dt, V, d, stride if V > 1 else d,
                                  scale, out.data_ptr(), _raw_stream(None, idx)), "dllm_embed_tokens")
    return out


def embed_tokens_backward(tokens: torch.Tensor, grad: torch.Tensor, V: int, scale: float = 1.0,
                          out: Optional[torch.Tensor] = None, accumulate: bool = False,
                          ws: Optional[torch.Tensor] = None, stream=None):
    """The gradient of embed_tokens with respect to its weight, (V, d): scale
    times the sum of ``grad`` (..., d), bf16 or fp32, over each id's positions.
    ``out``: preallocated, bf16 or fp32 (by default of grad's dtype);
    ``accumulate`` adds to it, e.g. to the gradient of a head that shares the
    weight.  ``ws``: a workspace of the caller's, not in use by another call."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return embed_tokens_backward(tokens, grad, V, scale, out, accumulate, ws)
    _need_cuda(tokens, grad)
    dt = _dtype(grad, "grad")
    dev, idx, V = grad.device, grad.get_device(), int(V)
    B, L, t_stride = _canvas(tokens, idx)
    if grad.shape[:-1] != tokens.shape or not grad.is_contiguous():
        raise ValueError("grad must be a contiguous tensor of the tokens' shape and d")
    if not 0 < V < 1 << 31:
        raise ValueError(f"V: {V} is out of range")
    d = grad.shape[-1]
    if out is None:
        if accumulate:
            raise ValueError("accumulate adds to the gradient given as out")
        out = torch.empty((V, d), dtype=grad.dtype, device=dev)
    out_dt = _dtype(out, "out")
    if out.device != dev:
        raise ValueError(f"out is on {out.device}; grad is on {dev}")
    out_stride = _weight(out, "out", V, d)
    raw = _raw_stream(None, idx)
    ws = _workspace(ws, _size("dllm_embed_tokens_backward_workspace_size", B * L, V, d), dev, raw)
    _check(_lib.dllm_embed_tokens_backward(tokens.data_ptr(), B, L, t_stride, grad.data_ptr(), dt, V, d, scale,
                                           out.data_ptr(), out_dt, out_stride, 1 if accumulate else 0, ws.data_ptr(),
                                           ws.numel() * ws.element_size(), raw), "dllm_embed_tokens_backward")
    return out


class _EmbedGrad(torch.autograd.Function):
    """The gradient is linear in its input, but its derivative is not built."""

    @staticmethod
    def forward(ctx, tokens, grad, V, scale):
        return embed_tokens_backward(tokens, grad, V, scale)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("the gradient of embed_canvas cannot be differentiated again")


class _EmbedCanvas(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale):
        if torch.is_tensor(tokens) and tokens.dim() in (1, 2) and tokens.numel() > 0:
            L, (*rows, unit) = tokens.shape[-1], tokens.stride()
            if (L > 1 and unit != 1) or (rows and tokens.shape[0] > 1 and rows[0] < L):
                tokens = tokens.contiguous()
        ctx.V, ctx.scale = weight.shape[0], scale
        ctx.save_for_backward(tokens)
        return embed_tokens(tokens, weight, scale)

    @staticmethod
    def backward(ctx, g):
        tokens, = ctx.saved_tensors
        _may_capture(ctx)
        g = g.contiguous()
        if torch.is_grad_enabled():                                              # (under create_graph)
            return None, _EmbedGrad.apply(tokens, g, ctx.V, ctx.scale), None
        return None, embed_tokens_backward(tokens, g, ctx.V, ctx.scale), None


def embed_canvas(tokens: torch.Tensor, weight: torch.Tensor, scale: float = 1.0):
    """embed_tokens for training, of tokens of any strides: differentiable once with
    respect to ``weight`` through autograd, captured and watched (``kernel_fault``) as score_hidden is."""
    out = _EmbedCanvas.apply(tokens, weight, float(scale))
    _stamp(out)
    return out
