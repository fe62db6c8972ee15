"""The scores of given tokens from hidden states, the embedding, and their
gradients, from the definitions in 64 bits (torch, on the inputs' device)."""
import math

import torch


def logits(hidden, weight, sup=()):
    z = hidden.double() @ weight.double().T
    z = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
    if len(sup):
        z[:, list(sup)] = -math.inf
    return z


def scores(hidden, weight, targets, sup=()):
    """(logprob, entropy, lse) of (T, d), (V, d), (T,)."""
    V = weight.shape[0]
    z = logits(hidden, weight, sup)
    live = torch.ones(V, dtype=torch.bool, device=z.device)
    live[list(sup)] = False
    lse = torch.logsumexp(z, 1)
    logp = z - lse[:, None]
    empty = torch.isneginf(lse)
    logp[empty] = torch.where(live, -math.log(int(live.sum())), -math.inf).to(logp)
    p = torch.exp(logp)
    entropy = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    t = targets.long()
    scored = (t >= 0) & (t < V)
    zero = torch.zeros_like(lse)
    logprob = logp.gather(1, t.clamp(0, V - 1)[:, None])[:, 0]
    return [torch.where(scored, x, zero) for x in (logprob, entropy, lse)]


def _taking_part(hidden, weight, targets, lse, g, gh, sup):
    """(rows that take part, g, gH) in 64 bits."""
    T, V = hidden.shape[0], weight.shape[0]
    t = targets.long()
    zero = torch.zeros(T, dtype=torch.float64, device=hidden.device)
    g = zero if g is None else g.double()
    gh = zero if gh is None else gh.double()
    for v in sup:
        g = torch.where(t == v, zero, g)
    return (t >= 0) & (t < V) & torch.isfinite(lse) & ((g != 0) | (gh != 0)), g, gh


def grads(hidden, weight, targets, lse, entropy, g, gh, sup=()):
    """dz (T, V), and the hidden states of the rows that take part; the gradients are dz @ weight and dz^T @ hidden."""
    T, V = hidden.shape[0], weight.shape[0]
    t = targets.long()
    zero = torch.zeros(T, dtype=torch.float64, device=hidden.device)
    rows, g, gh = _taking_part(hidden, weight, targets, lse, g, gh, sup)
    clean = torch.where(rows[:, None], hidden.double(), torch.zeros((), dtype=torch.float64, device=hidden.device))
    y = logits(clean, weight, sup) - torch.where(rows, lse.double(), zero)[:, None]
    p = torch.exp(y)
    y = torch.where(p > 0, y, torch.zeros_like(y))
    dz = -p * (g[:, None] + gh[:, None] * (y + entropy.double()[:, None]))
    dz[torch.arange(T, device=dz.device), t.clamp(0, V - 1)] += g
    return torch.where(rows[:, None], dz, torch.zeros_like(dz)), clean


def grad_parts(hidden, weight, targets, lse, entropy, g, gh, sup=()):
    """The magnitude of what the elements of dz are made of, p (|g| + |gH| (|z - lse + H| + 1)): a relative error of p, or an
    error of z, moves an element by that share of it, however small what is left of the element."""
    zero = torch.zeros(hidden.shape[0], dtype=torch.float64, device=hidden.device)
    _, clean = grads(hidden, weight, targets, lse, entropy, g, gh, sup)
    rows, g, gh = _taking_part(hidden, weight, targets, lse, g, gh, sup)
    y = logits(clean, weight, sup) - torch.where(rows, lse.double(), zero)[:, None]
    p = torch.exp(y)
    y = torch.where(p > 0, y, torch.zeros_like(y))
    size = p * (g.abs()[:, None] + gh.abs()[:, None] * ((y + entropy.double()[:, None]).abs() + 1))
    return torch.where(rows[:, None], size, torch.zeros_like(size))


def embedding_grad(tokens, grad, V, scale=1.0):
    d = grad.shape[-1]
    t = tokens.reshape(-1).long()
    ok = (t >= 0) & (t < V)
    out = torch.zeros((V, d), dtype=torch.float64, device=grad.device)
    out.index_add_(0, t[ok], grad.reshape(-1, d)[ok].double())
    return out * scale
