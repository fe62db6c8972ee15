"""The operators at the two ends of a model that is trained, as measured calls.

A masked diffusion language model embeds a canvas (mask tokens, or noise tokens,
among the placed ones) and ends in an LM head whose softmax scores the tokens of
the positions that were masked.  Embedding and head often share one weight.
Here are the scores of given tokens straight from the hidden states, with the
logits never stored, their gradient with respect to hidden states and weight,
the embedding of a canvas, and its gradient.

With ``own`` false ``run`` computes each operator in plain torch operations in
32 bits; with ``own`` true it calls ``commit_step_gb300``.
"""
import math

import torch

own = False


def listed():
    return [
        # One committed block of 32 scored for a client: the head's weight is what is read.
        {"name": "score-block", "op": "score", "T": 32, "V": 126464, "d": 4096, "scored": 1.0, "suppress": 1},
        # A short answer under a small model of an odd vocabulary: the smallest score.
        {"name": "score-odd", "op": "score", "T": 61, "V": 50257, "d": 768, "scored": 1.0, "suppress": 0},
        # The loss of a training batch, half of its positions masked and so scored.
        {"name": "score-train", "op": "score", "T": 8192, "V": 152064, "d": 3584, "scored": 0.5, "suppress": 1},
        # The gradient of the short answer, its entropy weighed as well.
        {"name": "grad-odd", "op": "grad", "T": 61, "V": 50257, "d": 768, "scored": 1.0, "suppress": 0, "entropy": True},
        # A policy gradient over one sequence, its completion scored.
        {"name": "grad-row", "op": "grad", "T": 1024, "V": 126464, "d": 4096, "scored": 0.5, "suppress": 1,
         "entropy": False},
        # A training batch with an entropy bonus, a little over half of the positions scored.
        {"name": "grad-train", "op": "grad", "T": 8192, "V": 126464, "d": 4096, "scored": 0.55, "suppress": 1,
         "entropy": True},
        # The canvas of one block, embedded before each forward of a decoder: the smallest call.
        {"name": "embed-block", "op": "embed", "B": 1, "L": 32, "V": 126464, "d": 4096, "dtype": "bf16", "masked": 0.6,
         "scaled": False},
        # A training batch of noised canvases of a model that scales its embedding.
        {"name": "embed-train", "op": "embed", "B": 16, "L": 4096, "V": 262144, "d": 2560, "dtype": "bf16",
         "masked": 0.0, "scaled": True},
        # The embedding's gradient for one short sequence in 32 bits.
        {"name": "embed-grad-odd", "op": "embed-grad", "B": 1, "L": 333, "V": 50257, "d": 768, "dtype": "f32",
         "masked": 0.5, "scaled": True},
        # A batch of blocks: most of the gradient's rows are zero.
        {"name": "embed-grad-blocks", "op": "embed-grad", "B": 64, "L": 32, "V": 152064, "d": 3584, "dtype": "bf16",
         "masked": 0.3, "scaled": False},
        # A training batch, half of it the mask token: one row sums half of all positions.
        {"name": "embed-grad-train", "op": "embed-grad", "B": 16, "L": 4096, "V": 126464, "d": 4096, "dtype": "bf16",
         "masked": 0.5, "scaled": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["score", "score", "grad", "grad", "embed", "embed-grad"])
    V, d = _log(rng, 300, 152064), 8 * _log(rng, 8, 512)
    if op in ("score", "grad"):
        T = _log(rng, 1, 8192)
        case = {"op": op, "T": T, "V": V, "d": d, "scored": rng.choice([0.02, 0.3, 0.5, 0.5, 1.0, 1.0]),
                "suppress": rng.choice([0, 1, 5])}
        while _rows(case) * V * d > 2.2e12:
            case["T"] = max(1, case["T"] // 2)
        if op == "grad":
            case["entropy"] = rng.random() < 0.5
        return case
    T = _log(rng, 1, 65536)
    B = rng.choice([b for b in (1, 1, 2, 3, 8, 16) if b <= T])
    case = {"op": op, "B": B, "L": max(1, T // B), "V": V, "d": d, "dtype": rng.choice(["bf16", "bf16", "f32"]),
            "masked": rng.choice([0.0, 0.1, 0.5, 0.9]), "scaled": rng.random() < 0.5}
    while work(case)["bytes"] > 1.5e9:
        case["d"] = 8 * (case["d"] // 16)
    return case


def _rows(case):
    """The positions that are scored."""
    return max(1, int(round(case["T"] * case["scored"])))


def _masked(case):
    return int(case["B"] * case["L"] * case["masked"])


def work(case):
    op, V, d = case["op"], case["V"], case["d"]
    if op in ("score", "grad"):
        T, n = case["T"], _rows(case)
        if op == "score":
            return {"bytes": 2 * d * (n + V) + 16 * T, "flops": 2 * n * V * d}
        # the weight and the scored hidden states in, the gradient of the weight and of every hidden state out
        return {"bytes": 2 * d * (n + V) + 2 * d * (T + V) + 20 * T, "flops": 6 * n * V * d}
    T, size = case["B"] * case["L"], 2 if case["dtype"] == "bf16" else 4
    if op == "embed":
        others = T - _masked(case)
        # ids are V u^2 with u uniform: the expected number of different ones, in 64 steps of V
        seen = 0.0
        for i in range(64):
            share = math.sqrt((i + 1) / 64) - math.sqrt(i / 64)
            seen += V / 64 * (1.0 - math.exp(-others * share * 64 / V))
        return {"bytes": int(size * d * (T + seen + (others < T)) + 4 * T), "flops": T * d}
    return {"bytes": size * d * (T + V) + 4 * T, "flops": T * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": dict(case)}
    return _prepare_head(case, g, s) if case["op"] in ("score", "grad") else _prepare_embed(case, g, s)


def _prepare_head(case, g, s):
    T, V, d = case["T"], case["V"], case["d"]
    # logits of a spread of 2.5, a trained model's peaks at most of the targets
    s["weight"] = torch.randn((V, d), device="cuda", generator=g, dtype=torch.bfloat16).mul_(2.5 / math.sqrt(d))
    h = torch.randn((T, d), device="cuda", generator=g)
    s["ids"] = [(7919 * (i + 1)) % V for i in range(case["suppress"])]
    s["sup"] = torch.tensor(s["ids"], dtype=torch.long, device="cuda")
    target = torch.randint(0, V, (T,), device="cuda", generator=g)
    target = torch.where((target[:, None] == s["sup"]).any(1), (target + 1) % V, target)
    pull = torch.rand((T, 1), device="cuda", generator=g).mul_(2.5) * (torch.rand((T, 1), device="cuda", generator=g) < 0.7)
    s["hidden"] = (h + pull * s["weight"][target].float()).to(torch.bfloat16)
    n = _rows(case)
    scored = torch.zeros((T,), dtype=torch.bool, device="cuda")
    scored[torch.randperm(T, device="cuda", generator=g)[:n]] = True
    s["targets"] = torch.where(scored, target, torch.full_like(target, -1)).to(torch.int32)
    s["n"] = n                                     # a loss divides by it
    if case["op"] == "grad":
        with torch.no_grad():
            s["logprob"], s["entropy"], s["lse"] = _plain_score(s)
        s["g_logprob"] = torch.randn((T,), device="cuda", generator=g)
        s["g_entropy"] = torch.randn((T,), device="cuda", generator=g).mul_(0.1) if case["entropy"] else None
    return s


def _prepare_embed(case, g, s):
    B, L, V, d = case["B"], case["L"], case["V"], case["d"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    mask_id = V - 1 - V // 300
    # some ids are far more frequent than others
    ids = torch.rand((B, L), device="cuda", generator=g, dtype=torch.float64).square_().mul_(V).long().clamp_(max=V - 1)
    covered = torch.randperm(B * L, device="cuda", generator=g)[:_masked(case)]
    ids.view(-1)[covered] = mask_id
    # the window of a longer canvas, as a decoder holds it
    canvas = torch.full((B, L + 17), mask_id, dtype=torch.int32, device="cuda")
    canvas[:, 9:9 + L] = ids.to(torch.int32)
    s["tokens"] = canvas[:, 9:9 + L]
    s["scale"] = math.sqrt(d) if case["scaled"] else 1.0
    if case["op"] == "embed":
        s["weight"] = torch.randn((V, d), device="cuda", generator=g, dtype=dt).mul_(0.02)
    else:
        s["grad"] = torch.randn((B, L, d), device="cuda", generator=g, dtype=dt).mul_(0.01)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    return (_own if own else _plain)(case["op"], case, s)


def _own(op, case, s):
    import commit_step_gb300 as cs

    if op == "score":
        return list(cs.lm_head_logprobs(s["hidden"], s["weight"], s["targets"], suppress_ids=s["ids"]))
    if op == "grad":
        return list(cs.lm_head_logprobs_backward(s["hidden"], s["weight"], s["targets"], s["lse"], s["entropy"],
                                                 s["g_logprob"], grad_entropy=s["g_entropy"], suppress_ids=s["ids"]))
    if op == "embed":
        return cs.embed_tokens(s["tokens"], s["weight"], scale=s["scale"])
    return cs.embed_tokens_backward(s["tokens"], s["grad"], case["V"], scale=s["scale"])


def _plain(op, case, s):
    if op == "score":
        return list(_plain_score(s))
    if op == "grad":
        return _plain_grad(s)
    if op == "embed":
        return (s["weight"][s["tokens"].long()].float() * s["scale"]).to(s["weight"].dtype)
    grad = s["grad"]
    # a row's sum over tens of thousands of positions: 64 bits where the result has 32
    wide = torch.float64 if grad.dtype == torch.float32 else torch.float32
    total = torch.zeros((case["V"], case["d"]), dtype=wide, device=grad.device)
    total.index_add_(0, s["tokens"].reshape(-1).long(), grad.reshape(-1, case["d"]).to(wide))
    return (total * s["scale"]).to(grad.dtype)


def _plain_logits(s):
    """The scored rows' positions, their logits and targets."""
    at = torch.argsort((s["targets"] < 0).to(torch.int32), stable=True)[:s["n"]]
    z = torch.matmul(s["hidden"][at].float(), s["weight"].float().T)
    return at, z.index_fill_(1, s["sup"], -math.inf), s["targets"][at].long()


def _plain_score(s):
    at, z, t = _plain_logits(s)
    m = z.amax(1, keepdim=True)
    zt = z.gather(1, t[:, None])[:, 0]
    y = z.sub_(m)
    e = torch.exp(y)
    Z = e.sum(1)
    entropy = torch.log(Z) - torch.where(e > 0, e * y, torch.zeros((), device=z.device)).sum(1) / Z
    lse = m[:, 0] + torch.log(Z)
    out = torch.zeros((3, s["targets"].shape[0]), device=z.device)
    out[:, at] = torch.stack([zt - lse, entropy, lse])
    return out[0], out[1], out[2]


def _plain_grad(s):
    at, z, t = _plain_logits(s)
    y = z.sub_(s["lse"][at][:, None])
    p = torch.exp(y)
    g = s["g_logprob"][at]
    bracket = g[:, None]
    if s["g_entropy"] is not None:
        y = torch.where(p > 0, y, torch.zeros((), device=z.device))
        bracket = bracket + s["g_entropy"][at][:, None] * (y + s["entropy"][at][:, None])
    dz = -(p * bracket)
    dz.scatter_add_(1, t[:, None], g[:, None])
    gh = torch.zeros(s["hidden"].shape, device=z.device)
    gh[at] = torch.matmul(dz, s["weight"].float())
    gw = torch.matmul(dz.T, s["hidden"][at].float())
    return [gh.to(torch.bfloat16), gw.to(torch.bfloat16)]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op in ("score", "grad") and work(case)["flops"] > 7e12:
        return None
    s = prepare(case, seed)
    with torch.no_grad():
        if op == "embed":
            flat = s["tokens"].reshape(-1).long()
            return (s["weight"].index_select(0, flat).double() * s["scale"]).view(*s["tokens"].shape, case["d"])
        if op == "embed-grad":
            return _exact_embed_grad(case, s)
        return _exact_head(case, s)


def _exact_embed_grad(case, s):
    """Sums over runs of the sorted tokens, by differences of running sums, some columns at a time."""
    V, d = case["V"], case["d"]
    flat = s["tokens"].reshape(-1)
    order = torch.argsort(flat.long(), stable=True)
    count = torch.bincount(flat.long(), minlength=V)
    end = torch.cumsum(count, 0)
    grad = s["grad"].reshape(-1, d)
    out = torch.empty((V, d), dtype=torch.float64, device="cuda")
    for a in range(0, d, 256):
        run_sum = torch.cumsum(grad[order, a:a + 256].double(), 0)
        run_sum = torch.cat([torch.zeros_like(run_sum[:1]), run_sum])
        out[:, a:a + 256] = (run_sum[end] - run_sum[end - count]) * s["scale"]
    return out


def _exact_head(case, s):
    T, V, d = case["T"], case["V"], case["d"]
    w, targets = s["weight"].double(), s["targets"].long()
    rows = torch.nonzero(targets >= 0)[:, 0]
    outs = [torch.zeros((T,), dtype=torch.float64, device="cuda") for _ in range(3)]
    gh = torch.zeros((T, d), dtype=torch.float64, device="cuda") if case["op"] == "grad" else None
    gw = torch.zeros((V, d), dtype=torch.float64, device="cuda") if case["op"] == "grad" else None
    for at in torch.split(rows, max(1, 2 ** 27 // V)):
        h, t = s["hidden"][at].double(), targets[at]
        z = h @ w.T
        z[:, s["sup"]] = -math.inf
        if case["op"] == "score":
            logp = torch.log_softmax(z, 1)
            outs[0][at] = logp.gather(1, t[:, None])[:, 0]
            outs[1][at] = -torch.nan_to_num(torch.exp(logp) * logp, nan=0.0).sum(1)
            outs[2][at] = torch.logsumexp(z, 1)
            continue
        # the saved log-sum-exp and entropy are inputs of the backward pass
        z -= s["lse"][at].double()[:, None]
        p = torch.exp(z)
        dz = torch.nn.functional.one_hot(t, V).double() - p
        dz *= s["g_logprob"][at].double()[:, None]
        if s["g_entropy"] is not None:
            inner = torch.nan_to_num(p * (z + s["entropy"][at].double()[:, None]), nan=0.0)
            dz -= s["g_entropy"][at].double()[:, None] * inner
        gh[at] = dz @ w
        gw += dz.T @ h
    return outs if case["op"] == "score" else [gh, gw]
