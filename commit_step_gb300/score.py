"""Log probabilities of given tokens, with the entropy and the top
alternatives, and their gradient (``dllm_token_logprobs``,
``dllm_token_logprobs_backward``)."""
from __future__ import annotations

import ctypes as C
from typing import Optional, Sequence

import torch

from . import _F32, _I32, _check, _dtype_code, _lib, _need_cuda
from .cache import _at, _at_or_none, _empty, _raw_stream

MAX_TOP = 32


def _rows(t: torch.Tensor, name: str):
    """(T, V, row stride) of (T, V) or (B, L, V) logits, unit stride over V."""
    if not torch.is_tensor(t) or t.dim() not in (2, 3):
        raise ValueError(f"{name} must be (T, V) or (B, L, V)")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride over V")
    V = t.shape[-1]
    if t.dim() == 2:
        return t.shape[0], V, (t.stride(0) if t.shape[0] > 1 else V)
    B, L, _ = t.shape
    stride = t.stride(1) if L > 1 else (t.stride(0) if B > 1 else V)
    if B > 1 and L > 0 and t.stride(0) != L * stride:
        raise ValueError(f"{name} must have evenly spaced rows")
    return B * L, V, stride


def _sup(suppress_ids: Sequence[int]):
    ids = [_int32(v, "suppress_ids") for v in suppress_ids]
    return ((C.c_int32 * len(ids))(*ids) if ids else None), len(ids)


def _int32(v, name: str) -> int:
    """v as the library takes it (ctypes would cut it to its low bits)."""
    v = int(v)
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{name}: {v} is out of range")
    return v


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, top: int = 0, suppress_ids: Sequence[int] = (),
                   out=None, stream=None):
    """Scores given tokens under logits (T, V) or (B, L, V), bf16 or fp32.

    Returns (logprob, entropy, lse, top_ids, top_logprob): float32 shaped like
    ``targets`` (int32, the logits' shape without V; an id outside [0, V) is
    no target and scores 0), and the ids (int32) and log probabilities of the
    ``top`` largest logits, shaped (..., top); the last two are None when top
    is 0.  ``out``: the same five, preallocated."""
    _need_cuda(logits, targets)
    T, V, stride = _rows(logits, "logits")
    dt, dev, idx, shape, top = _dtype_code(logits), logits.device, logits.get_device(), logits.shape[:-1], _int32(top, "top")
    if out is None:
        lp = _empty(shape, torch.float32, dev, stream)
        ent = _empty(shape, torch.float32, dev, stream)
        lse = _empty(shape, torch.float32, dev, stream)
        lp_at, ent_at, lse_at = lp.data_ptr(), ent.data_ptr(), lse.data_ptr()
        ids = _empty((*shape, top), torch.int32, dev, stream) if top > 0 else None
        tlp = _empty((*shape, top), torch.float32, dev, stream) if top > 0 else None
    else:
        lp, ent, lse, ids, tlp = out
        lp_at, ent_at, lse_at = [_at(t, name, T, _F32, idx, dev)
                                 for t, name in ((lp, "logprob"), (ent, "entropy"), (lse, "lse"))]
    sup, n_sup = _sup(suppress_ids)
    _check(_lib.dllm_token_logprobs(logits.data_ptr(), dt, T, V, stride, _at(targets, "targets", T, _I32, idx, dev), sup,
                                    n_sup, top, lp_at, ent_at, lse_at,
                                    _at_or_none(ids, "top_ids", T * top, _I32, idx, dev),
                                    _at_or_none(tlp, "top_logprob", T * top, _F32, idx, dev),
                                    _raw_stream(stream, idx)), "dllm_token_logprobs")
    return lp, ent, lse, ids, tlp


def token_logprobs_backward(logits: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor, entropy: torch.Tensor,
                            grad_logprob: Optional[torch.Tensor], grad_entropy: Optional[torch.Tensor] = None,
                            top_ids: Optional[torch.Tensor] = None, grad_top: Optional[torch.Tensor] = None,
                            suppress_ids: Sequence[int] = (), out: Optional[torch.Tensor] = None, stream=None):
    """The gradient of token_logprobs with respect to the logits, in their
    dtype: from the saved ``lse`` and ``entropy`` and the gradients of
    logprob, entropy and top_logprob (None: zero; ``grad_top`` comes with the
    ``top_ids`` it belongs to).  ``out`` may be ``logits`` itself."""
    _need_cuda(logits, targets)
    T, V, stride = _rows(logits, "logits")
    dt, dev, idx = _dtype_code(logits), logits.device, logits.get_device()
    top, ids_at, top_at = 0, None, None
    if grad_top is not None:
        if top_ids is None or not torch.is_tensor(grad_top) or grad_top.dim() < 1:
            raise ValueError("grad_top comes with the top_ids it belongs to")
        top = grad_top.shape[-1]
        top_at = _at(grad_top, "grad_top", T * top, _F32, idx, dev)
        ids_at = _at(top_ids, "top_ids", T * top, _I32, idx, dev)
    if out is None:
        out = _empty(logits.shape, logits.dtype, dev, stream)
    elif not torch.is_tensor(out) or out.dtype != logits.dtype or out.device != dev or out.shape != logits.shape:
        raise ValueError("out must be shaped and typed like logits, on the same device")
    _, _, out_stride = _rows(out, "out")
    sup, n_sup = _sup(suppress_ids)
    _check(_lib.dllm_token_logprobs_backward(logits.data_ptr(), dt, T, V, stride,
                                             _at(targets, "targets", T, _I32, idx, dev), sup, n_sup,
                                             _at(lse, "lse", T, _F32, idx, dev),
                                             _at(entropy, "entropy", T, _F32, idx, dev),
                                             _at_or_none(grad_logprob, "grad_logprob", T, _F32, idx, dev),
                                             _at_or_none(grad_entropy, "grad_entropy", T, _F32, idx, dev), top, ids_at,
                                             top_at, out.data_ptr(), out_stride, _raw_stream(stream, idx)),
           "dllm_token_logprobs_backward")
    return out


class _ScoreGrad(torch.autograd.Function):
    """The gradient as a step of a graph that is to be differentiated again: there
    is no second derivative, and leaving it out of a sum of losses would go unseen."""

    @staticmethod
    def forward(ctx, logits, targets, lse, ent, ids, suppress_ids, g_lp, g_ent, g_top):
        return _score_grad(logits, targets, lse, ent, ids, suppress_ids, g_lp, g_ent, g_top)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("the gradient of score_tokens cannot be differentiated again")


def _score_grad(logits, targets, lse, ent, ids, suppress_ids, g_lp, g_ent, g_top):
    # (gradients that reach here expanded from a scalar are not contiguous)
    g_lp, g_ent, g_top = [None if g is None else g.float().contiguous() for g in (g_lp, g_ent, g_top)]
    return token_logprobs_backward(logits, targets, lse, ent, g_lp, g_ent, ids if g_top is not None else None, g_top,
                                   suppress_ids=suppress_ids)


class _ScoreTokens(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, top, suppress_ids):
        lp, ent, lse, ids, tlp = token_logprobs(logits, targets, top=top, suppress_ids=suppress_ids)
        ctx.suppress_ids = suppress_ids
        ctx.save_for_backward(logits, targets, lse, ent, ids)
        if ids is not None:
            ctx.mark_non_differentiable(ids)
        return lp, ent, ids, tlp

    @staticmethod
    def backward(ctx, g_lp, g_ent, _g_ids, g_top):
        logits, targets, lse, ent, ids = ctx.saved_tensors
        grad = _ScoreGrad.apply if torch.is_grad_enabled() else _score_grad      # (enabled under create_graph)
        return grad(logits, targets, lse, ent, ids, ctx.suppress_ids, g_lp, g_ent, g_top), None, None, None


def score_tokens(logits: torch.Tensor, targets: torch.Tensor, top: int = 0, suppress_ids: Sequence[int] = ()):
    """token_logprobs for training: (logprob, entropy, top_ids, top_logprob),
    differentiable once with respect to ``logits`` through autograd."""
    return _ScoreTokens.apply(logits, targets, int(top), tuple(suppress_ids))
