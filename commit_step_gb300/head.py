"""Log probabilities of given tokens straight from the hidden states, and their
gradient with respect to hidden states and weight, without the logits in memory
(``dllm_lm_head_logprobs``, ``dllm_lm_head_logprobs_backward``)."""
from __future__ import annotations

import functools
import threading
from typing import Optional, Sequence

import torch

from . import DLLM_BF16, DLLM_F32, _F32, _I32, _check, _lib, _need_cuda
from .cache import _at, _at_or_none, _raw_stream
from .score import _rows, _sup


def _matrix(t, name: str, cols: int, device):
    """(rows, row stride) of a 2-D bf16 tensor of `cols` columns."""
    if not torch.is_tensor(t) or t.dtype != torch.bfloat16 or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D bfloat16 tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}; hidden is on {device}")
    (rows, width), (stride, unit) = t.shape, t.stride()
    if width != cols or (cols > 1 and unit != 1):
        raise ValueError(f"{name} must have {cols} columns at unit stride")
    return rows, (stride if rows > 1 else cols)


def _ends(hidden, weight, targets):
    """Shape and stride of hidden (T, d) or (B, L, d) and weight (V, d)."""
    try:                                     # (the usual case; a call's cost on the host is mostly these checks)
        h, w = hidden.shape, weight.shape
        if (len(h) == 2 and len(w) == 2 and h[1] == w[1] and hidden.dtype == weight.dtype == torch.bfloat16
                and hidden.get_device() == weight.get_device() >= 0):
            (hs, unit), (ws, w_unit) = hidden.stride(), weight.stride()
            if unit == 1 and w_unit == 1:
                return h[0], h[1], (hs if h[0] > 1 else h[1]), w[0], (ws if w[0] > 1 else h[1])
    except AttributeError:
        pass
    _need_cuda(hidden, weight, targets)
    if not torch.is_tensor(hidden) or hidden.dtype != torch.bfloat16 or hidden.dim() not in (2, 3):
        raise TypeError("hidden must be a (T, d) or (B, L, d) bfloat16 tensor")
    T, d, stride = _rows(hidden, "hidden")
    V, w_stride = _matrix(weight, "weight", d, hidden.device)
    return T, d, stride, V, w_stride


_KEPT = threading.local()
_KEEP = 32 << 20


def _workspace(ws, need: int, device, raw: int):
    """The caller's workspace, or one for a call on the current stream.  A call's
    launches pass their parts on through it, so it is kept for later calls of the
    same host thread on the same stream only, up to 32 MB (a larger one costs
    little beside the call that needs it), and a call that is captured gets memory
    of its graph's.  (Allocated anew for every call, 7 MB cost the host 7 of 30 us.)"""
    if ws is not None:
        if not torch.is_tensor(ws):
            raise TypeError("ws must be a tensor")
        if ws.device != device or not ws.is_contiguous():
            raise ValueError(f"ws must be a contiguous tensor on {device}")
        return ws
    if need > _KEEP or torch.cuda.is_current_stream_capturing():
        return torch.empty((need,), dtype=torch.uint8, device=device)
    try:
        kept = _KEPT.ws
    except AttributeError:
        kept = _KEPT.ws = {}
    key = (device.index, raw)
    ws = kept.get(key)
    if ws is None or ws.numel() < need:
        ws = kept[key] = torch.empty((need,), dtype=torch.uint8, device=device)
    return ws


_SIZES = {}


def _size(query, *shape):
    """What a size query answers on the current device."""
    key = (query, torch._C._cuda_getDevice(), shape)
    need = _SIZES.get(key)
    if need is None:
        if len(_SIZES) > 4096:                                                  # (ever new lengths)
            _SIZES.clear()
        need = _SIZES[key] = int(getattr(_lib, query)(*shape))
    return need


def lm_head_logprobs(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, suppress_ids: Sequence[int] = (),
                     out=None, ws: Optional[torch.Tensor] = None, stream=None):
    """Scores given tokens under the logits hidden @ weight^T, which are never
    stored: (logprob, entropy, lse), float32 shaped like ``targets``.

    hidden (T, d) or (B, L, d) and weight (V, d) bf16; ``targets`` int32, hidden's
    shape without d.  A row whose target lies outside [0, V) is not scored: it
    gets 0 for all three, and its hidden state may hold anything.  (Of more than 256
    rows it costs nothing; as many are one tile, which reads the weight whatever is
    scored.)  A hidden state with a NaN scores like logits of -inf: lse is -inf,
    logprob -ln of the number of ids.
    ``out``: the same three, preallocated.  ``ws``: a workspace of the caller's,
    not in use by another call; zeroed, it tells ``workspace_fault`` afterwards
    whether a wait ran out (``kernel_fault`` tells it of any call)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return lm_head_logprobs(hidden, weight, targets, suppress_ids, out, ws)
    T, d, stride, V, w_stride = _ends(hidden, weight, targets)
    dev, idx = hidden.device, hidden.get_device()
    if out is None:
        shape = hidden.shape[:-1]
        lp = torch.empty(shape, dtype=torch.float32, device=dev)
        ent = torch.empty(shape, dtype=torch.float32, device=dev)
        lse = torch.empty(shape, dtype=torch.float32, device=dev)
        at = lp.data_ptr(), ent.data_ptr(), lse.data_ptr()
    else:
        lp, ent, lse = out
        at = [_at(t, name, T, _F32, idx, dev) for t, name in ((lp, "logprob"), (ent, "entropy"), (lse, "lse"))]
    raw = _raw_stream(None, idx)
    ws = _workspace(ws, _size("dllm_lm_head_logprobs_workspace_size", T, V, d), dev, raw)
    sup, n_sup = _sup(suppress_ids)
    _check(_lib.dllm_lm_head_logprobs(hidden.data_ptr(), T, d, stride, weight.data_ptr(), V, w_stride,
                                      _at(targets, "targets", T, _I32, idx, dev), sup, n_sup, *at, ws.data_ptr(),
                                      ws.numel() * ws.element_size(), raw), "dllm_lm_head_logprobs")
    return lp, ent, lse


def lm_head_logprobs_backward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                              entropy: torch.Tensor, grad_logprob: Optional[torch.Tensor],
                              grad_entropy: Optional[torch.Tensor] = None, suppress_ids: Sequence[int] = (), out=None,
                              accumulate: bool = False, hidden_grad: bool = True, weight_grad: bool = True,
                              ws: Optional[torch.Tensor] = None, stream=None):
    """The gradient of lm_head_logprobs: (grad_hidden bf16 like hidden,
    grad_weight bf16 like weight), from the saved ``lse`` and ``entropy`` and the
    gradients of logprob and entropy (None: zero).  One that is not wanted
    (``hidden_grad``, ``weight_grad`` false) is None.  ``out``: the two,
    preallocated (grad_weight bf16 or float32, either None to be made here; a float32
    one is also made of a gradient of the logits held in more bits, for a product
    more); ``accumulate`` adds to out's grad_weight.  ``ws`` as in lm_head_logprobs."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return lm_head_logprobs_backward(hidden, weight, targets, lse, entropy, grad_logprob, grad_entropy, suppress_ids,
                                             out, accumulate, hidden_grad, weight_grad, ws)
    T, d, stride, V, w_stride = _ends(hidden, weight, targets)
    dev, idx = hidden.device, hidden.get_device()
    gh, gw = (None, None) if out is None else out
    if (gh is not None and not hidden_grad) or (gw is not None and not weight_grad):
        raise ValueError("out holds a gradient that is not wanted")
    if accumulate and gw is None:
        raise ValueError("accumulate adds to the grad_weight given in out")
    if hidden_grad and gh is None:
        gh = torch.empty(hidden.shape, dtype=torch.bfloat16, device=dev)
    if weight_grad and gw is None:
        gw = torch.empty((V, d), dtype=torch.bfloat16, device=dev)
    gh_stride, gw_stride, gw_dt = d, d, DLLM_BF16
    if gh is not None:
        if not torch.is_tensor(gh) or gh.dtype != torch.bfloat16 or gh.device != dev or gh.shape != hidden.shape:
            raise ValueError("grad_hidden must be shaped and typed like hidden, on the same device")
        _, _, gh_stride = _rows(gh, "grad_hidden")
    if gw is not None:
        if not torch.is_tensor(gw) or gw.dtype not in (torch.bfloat16, torch.float32) or gw.device != dev:
            raise ValueError("grad_weight must be a bfloat16 or float32 tensor on hidden's device")
        if gw.shape != (V, d) or (d > 1 and gw.stride(1) != 1):
            raise ValueError("grad_weight must be shaped like weight, with unit column stride")
        gw_stride = gw.stride(0) if V > 1 else d
        gw_dt = DLLM_F32 if gw.dtype == torch.float32 else DLLM_BF16
    raw = _raw_stream(None, idx)
    ws = _workspace(ws, _size("dllm_lm_head_logprobs_backward_workspace_size", T, V, d), dev, raw)
    sup, n_sup = _sup(suppress_ids)
    _check(_lib.dllm_lm_head_logprobs_backward(
        hidden.data_ptr(), T, d, stride, weight.data_ptr(), V, w_stride, _at(targets, "targets", T, _I32, idx, dev), sup,
        n_sup, _at(lse, "lse", T, _F32, idx, dev), _at(entropy, "entropy", T, _F32, idx, dev),
        _at_or_none(grad_logprob, "grad_logprob", T, _F32, idx, dev),
        _at_or_none(grad_entropy, "grad_entropy", T, _F32, idx, dev), None if gh is None else gh.data_ptr(), gh_stride,
        None if gw is None else gw.data_ptr(), gw_dt, gw_stride, 1 if accumulate else 0, ws.data_ptr(),
        ws.numel() * ws.element_size(), raw), "dllm_lm_head_logprobs_backward")
    return gh, gw


_STREAM = "commit_step_gb300.stream"


def _leaves(node):
    """The accumulators of the leaves that a step of a graph was made from.  One lives
    as long as any graph that holds it, and runs on the stream of the first."""
    return [f for f, _ in node.next_functions if f is not None and f.name().endswith("AccumulateGrad")]


def _mark(marks, index, *_):
    marks[_STREAM] = torch._C._cuda_getCurrentRawStream(index)


def _stamp(result):
    """Writes the leaves' accumulators' streams down: the current one where they seem
    new, and the one they run on once they have run (something else, a data-parallel
    wrapper say, may have made them and keep them)."""
    if result.requires_grad:
        for f in _leaves(result.grad_fn):
            marks = f.metadata
            if _STREAM not in marks:
                # (the hook holds the marks and not f, which would hold itself)
                mark = functools.partial(_mark, marks, result.get_device())
                mark()
                f.register_prehook(mark)


def _may_capture(node):
    """Refuses a captured gradient of a leaf whose accumulator a graph made on the
    default stream keeps: it would run there, which a capture may not touch."""
    if torch.cuda.is_current_stream_capturing() and any(f.metadata.get(_STREAM) == 0 for f in _leaves(node)):
        raise RuntimeError("this gradient is captured while a result computed from the same leaf on the default stream "
                           "lives: drop that result first, or compute it on another stream")


def _head_grad(hidden, weight, targets, lse, ent, suppress_ids, g_lp, g_ent, want):
    # (gradients that reach here expanded from a scalar are not contiguous)
    g_lp, g_ent = [None if g is None else g.float().contiguous() for g in (g_lp, g_ent)]
    return lm_head_logprobs_backward(hidden, weight, targets, lse, ent, g_lp, g_ent, suppress_ids=suppress_ids,
                                     hidden_grad=want[0], weight_grad=want[1])


class _HeadGrad(torch.autograd.Function):
    """The gradient as a step of a graph that is to be differentiated again: there
    is no second derivative, and leaving it out of a sum of losses would go unseen."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, lse, ent, suppress_ids, g_lp, g_ent, want):
        return _head_grad(hidden, weight, targets, lse, ent, suppress_ids, g_lp, g_ent, want)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the gradient of score_hidden cannot be differentiated again")


def _spaced(t):
    """Hidden states whose rows are evenly spaced and whole vectors: t, or a copy of it."""
    if t.dim() not in (2, 3) or t.numel() == 0:
        return t
    try:
        _, _, stride = _rows(t, "hidden")
    except ValueError:
        return t.contiguous()
    # (an expanded row, or one that begins between vectors)
    even = stride >= t.shape[-1] and (t.shape[-1] % 8 != 0 or (stride % 8 == 0 and t.data_ptr() % 16 == 0))
    return t if even else t.clone(memory_format=torch.contiguous_format)


class _ScoreHidden(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, targets, suppress_ids):
        ctx.set_materialize_grads(False)
        if torch.is_tensor(hidden) and hidden.is_cuda:
            hidden = _spaced(hidden)
        if torch.is_tensor(targets) and not targets.is_contiguous():
            targets = targets.contiguous()
        lp, ent, lse = lm_head_logprobs(hidden, weight, targets, suppress_ids=suppress_ids)
        ctx.suppress_ids = suppress_ids
        ctx.save_for_backward(hidden, weight, targets, lse, ent)
        return lp, ent

    @staticmethod
    def backward(ctx, g_lp, g_ent):
        hidden, weight, targets, lse, ent = ctx.saved_tensors
        want = ctx.needs_input_grad[:2]
        _may_capture(ctx)
        grad = _HeadGrad.apply if torch.is_grad_enabled() else _head_grad        # (enabled under create_graph)
        gh, gw = grad(hidden, weight, targets, lse, ent, ctx.suppress_ids, g_lp, g_ent, want)
        return gh, gw, None, None


def score_hidden(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, suppress_ids: Sequence[int] = ()):
    """lm_head_logprobs for training: (logprob, entropy), differentiable once with
    respect to ``hidden`` and ``weight`` through autograd.  Hidden states and targets
    of any strides (``hidden[:, :-1]``, ``tokens[:, 1:]``): what a call cannot read as it
    lies is copied.  A hidden state with a NaN keeps a loss finite (a logprob of -ln of
    the number of ids) and has no gradient: to see a run that diverges, look at the
    hidden states, or at lm_head_logprobs' lse (-inf there).  A backward pass that is
    captured into a CUDA graph is refused while a result lives that was computed from
    the same leaves on the default stream (warm up on another, backward pass included: a
    leaf's accumulator that something else made is known once it has run).  Workspaces are the
    binding's own: ``kernel_fault`` tells whether a wait of a call ran out."""
    logprob, entropy = _ScoreHidden.apply(hidden, weight, targets, tuple(suppress_ids))
    _stamp(logprob)
    return logprob, entropy
