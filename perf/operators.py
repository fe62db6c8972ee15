"""The operators of cached block decoding and of token scoring, as measured calls.

A block-diffusion decoder keeps the finished blocks' keys and values in a paged
8-bit cache (e4m3 codes, one scale for each page and head), attends from the
current block over it, drops the tokens that attract the least attention when
the cache is full, and scores given tokens under the logits (with the gradient
of that score for training).

With ``own`` false ``run`` computes each operator in plain torch operations in
32 bits; with ``own`` true it calls ``commit_step_gb300``.
"""
import math

import torch

own = False

LOG2E = 1.4426950408889634


def listed():
    return [
        # One new token for each of a few sequences: the smallest append, where latency counts.
        {"name": "append-token", "op": "append", "B": 4, "L": 1, "H": 8, "D": 128, "ps": 64, "at": 1000},
        # Prompts written into the cache after their forward, lengths not a multiple of the page.
        {"name": "append-prompt", "op": "append", "B": 8, "L": 4093, "H": 8, "D": 128, "ps": 64, "at": 37},
        # One sequence, one token: the shortest attention call of a decoder (7 query heads share a key head).
        {"name": "attend-token", "op": "attend", "B": 1, "L": 1, "Hq": 28, "H": 4, "D": 128, "ps": 64, "lo": 1999,
         "hi": 1999, "mask": False, "weights": False},
        # A block of 32 of a model without shared heads, ragged sequences, small pages, some keys masked.
        {"name": "attend-block", "op": "attend", "B": 8, "L": 32, "Hq": 32, "H": 32, "D": 128, "ps": 16, "lo": 517,
         "hi": 4096, "mask": True, "weights": False},
        # A block of 32 with 7 query heads to a key head, over a full batch, with the weights that eviction reads.
        {"name": "attend-block-weights", "op": "attend", "B": 16, "L": 32, "Hq": 28, "H": 4, "D": 128, "ps": 64,
         "lo": 2000, "hi": 8192, "mask": False, "weights": True},
        # Single tokens over long caches: the bytes of the cache are what it costs.
        {"name": "attend-long", "op": "attend", "B": 4, "L": 1, "Hq": 32, "H": 8, "D": 128, "ps": 128, "lo": 60001,
         "hi": 131072, "mask": False, "weights": False},
        # One short sequence halved.
        {"name": "evict-one", "op": "evict", "B": 1, "H": 4, "D": 128, "ps": 64, "lo": 1000, "hi": 1000, "budget": 512,
         "first": 4, "last": 32},
        # A full batch of long sequences cut to a quarter, the first tokens and the latest blocks kept.
        {"name": "evict-batch", "op": "evict", "B": 16, "H": 8, "D": 128, "ps": 64, "lo": 9001, "hi": 16384,
         "budget": 4096, "first": 16, "last": 512},
        # The tokens of one committed block, scored with alternatives for a client.
        {"name": "score-block", "op": "score", "T": 32, "V": 126464, "dtype": "bf16", "top": 8, "suppress": 1},
        # A batch of rollouts scored.
        {"name": "score-batch", "op": "score", "T": 4096, "V": 152064, "dtype": "bf16", "top": 20, "suppress": 0},
        # Gradient of a policy loss on one batch row, fp32 logits of an odd vocabulary.
        {"name": "score-grad-f32", "op": "grad", "T": 61, "V": 50257, "dtype": "f32", "top": 5, "suppress": 1},
        # Gradient for a training batch: one read and one write of the logits.
        {"name": "score-grad-batch", "op": "grad", "T": 4096, "V": 126464, "dtype": "bf16", "top": 0, "suppress": 1},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "evict", "score", "grad"])
    D = rng.choice([64, 128, 128])
    ps = rng.choice([16, 32, 64, 128])
    if op == "append":
        return {"op": op, "B": _log(rng, 1, 32), "L": _log(rng, 1, 1024), "H": rng.choice([1, 2, 4, 8]), "D": D,
                "ps": ps, "at": rng.randrange(0, 3000)}
    if op == "attend":
        H, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 7, 8])
        hi = _log(rng, 1, 16384)
        return {"op": op, "B": _log(rng, 1, 16), "L": rng.choice([1, 1, 4, 8, 16, 32, 33, 64]), "Hq": H * group, "H": H,
                "D": D, "ps": ps, "lo": rng.randrange(0, hi + 1), "hi": hi, "mask": rng.random() < 0.3,
                "weights": rng.random() < 0.4}
    if op == "evict":
        hi = _log(rng, 40, 16384)
        budget = rng.randrange(16, hi)
        first = rng.randrange(0, min(16, budget))
        return {"op": op, "B": _log(rng, 1, 16), "H": rng.choice([1, 2, 4, 8]), "D": D, "ps": ps,
                "lo": rng.randrange(1, hi + 1), "hi": hi, "budget": budget, "first": first,
                "last": rng.randrange(0, min(64, budget - first) + 1)}
    return {"op": op, "T": _log(rng, 1, 2048), "V": _log(rng, 300, 152064), "dtype": rng.choice(["bf16", "f32"]),
            "top": rng.choice([0, 1, 5, 8, 20, 32]), "suppress": rng.choice([0, 1, 5])}


def _lens(case):
    """Ragged lengths from lo to hi (their order is drawn from the seed)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi - (hi - lo) * b // max(B - 1, 1) for b in range(B)]


def _cells(case):
    return sum(_lens(case)) * case["H"]


def work(case):
    op = case["op"]
    if op == "append":
        n = case["B"] * case["L"] * case["H"] * case["D"] * 2
        return {"bytes": n * 3, "flops": n * 2}
    if op == "attend":
        rows = case["B"] * case["L"] * case["Hq"]
        n = _cells(case)
        flops = 4 * n * case["L"] * (case["Hq"] // case["H"]) * case["D"]
        nbytes = 2 * n * case["D"] + rows * (4 * case["D"] + 4)
        if case["weights"]:
            nbytes += 4 * n
        return {"bytes": nbytes, "flops": flops}
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in _lens(case)) * case["H"]
        return {"bytes": 4 * _cells(case) + kept * (4 * case["D"] + 8), "flops": kept * 4 * case["D"]}
    n = case["T"] * case["V"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "score":
        return {"bytes": n * size + case["T"] * (16 + 8 * case["top"]), "flops": 6 * n}
    return {"bytes": 2 * n * size + case["T"] * (20 + 8 * case["top"]), "flops": 6 * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _cache(g, pages, case):
    """Page pools of e4m3 codes and scales, as a model's keys and values leave them: the range differs by page and head."""
    H, ps, D = case["H"], case["ps"], case["D"]
    codes, scales = [], []
    for _ in range(2):
        codes.append(torch.randn((pages, H, ps, D), device="cuda", generator=g, dtype=torch.bfloat16).mul_(120).clamp_(
            -448, 448).to(torch.float8_e4m3fn))
        scales.append(torch.pow(2.0, -torch.randint(6, 9, (pages, H), device="cuda", generator=g).float()))
    return {"k": codes[0], "v": codes[1], "k_scale": scales[0], "v_scale": scales[1]}


def _tables(g, B, width, pages, count=1):
    """`count` page tables (B, width) of distinct pages in random order; the pool's last page is in none of them."""
    order = torch.randperm(pages - 1, device="cuda", generator=g)[:count * B * width].to(torch.int32)
    return list(order.view(count, B, width).contiguous())


def _wrap(state):
    if own:
        import commit_step_gb300 as cs

        c = state["cache"]
        state["handle"] = cs.KVCache.from_tensors(c["k"], c["v"], c["k_scale"], c["v_scale"])
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if op in ("score", "grad"):
        return _prepare_score(case, g, s)
    B, H, D, ps = case["B"], case["H"], case["D"], case["ps"]
    if op == "append":
        width = -(-(case["at"] + case["L"]) // ps) + 1
        pages = B * width + 1
        s["cache"] = _cache(g, pages, case)
        s["table"], = _tables(g, B, width, pages)
        s["start"] = torch.randint(max(0, case["at"] - ps), case["at"] + 1, (B,), device="cuda", generator=g,
                                   dtype=torch.int32)
        # keys and values as they leave a projection: slices of one packed tensor, unit stride over D only
        kv = torch.randn((B, case["L"], 2, H, D), device="cuda", generator=g, dtype=torch.bfloat16)
        s["k_new"], s["v_new"] = kv[:, :, 0], kv[:, :, 1]
        return _wrap(s)
    lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    s["lens"] = lens[torch.randperm(B, device="cuda", generator=g)].contiguous()
    width = max(1, -(-case["hi"] // ps))
    if op == "attend":
        pages = B * width + 1
        s["cache"] = _cache(g, pages, case)
        s["table"], = _tables(g, B, width, pages)
        s["q"] = torch.randn((B, case["L"], case["Hq"], D), device="cuda", generator=g, dtype=torch.bfloat16)
        s["mask"] = None
        if case["mask"]:
            s["mask"] = (torch.rand((B, width * ps), device="cuda", generator=g) < 0.9).to(torch.uint8)
        s["weights"] = torch.zeros((B, H, width * ps), device="cuda") if case["weights"] else None
        return _wrap(s)
    dst = -(-case["budget"] // ps)
    pages = B * (width + dst) + 1
    s["cache"] = _cache(g, pages, case)
    order, = _tables(g, 1, B * (width + dst), pages)
    s["table"] = order[0, :B * width].view(B, width).contiguous()
    s["dst"] = order[0, B * width:].view(B, dst).contiguous()
    # accumulated weights: most tokens draw little, a few draw much; many are equal
    w = torch.rand((B, H, width * ps), device="cuda", generator=g)
    s["weights"] = torch.round(w ** 8 * 4096) / 64
    return _wrap(s)


def _prepare_score(case, g, s):
    T, V = case["T"], case["V"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    z = torch.randn((T, V), device="cuda", generator=g, dtype=dt).mul_(2.5)
    peak = torch.randint(0, V, (T, 4), device="cuda", generator=g)
    z.scatter_add_(1, peak, torch.rand((T, 4), device="cuda", generator=g).mul_(14).to(dt))
    s["logits"] = z
    s["targets"] = torch.where(torch.rand((T,), device="cuda", generator=g) < 0.6, peak[:, 0],
                               torch.randint(0, V, (T,), device="cuda", generator=g)).to(torch.int32)
    s["ids"] = [(7919 * (i + 1)) % V for i in range(case["suppress"])]
    s["sup"] = torch.tensor(s["ids"], dtype=torch.long, device="cuda")
    s["targets"] = torch.where((s["targets"][:, None] == s["sup"]).any(1), -1, s["targets"])  # positions not scored
    if case["op"] == "grad":
        with torch.no_grad():
            lp, ent, lse, top, _ = _plain_score(z, s["targets"], case["top"], s["sup"])
        s["lse"], s["entropy"] = lse, ent
        s["top_ids"] = top if case["top"] else None
        s["g_logprob"] = torch.randn((T,), device="cuda", generator=g)
        s["g_entropy"] = torch.randn((T,), device="cuda", generator=g).mul_(0.1)
        s["g_top"] = torch.randn((T, case["top"]), device="cuda", generator=g) if case["top"] else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    return (_own if own else _plain)(case["op"], case, s)


def _held(c):
    return {"k": c["k"], "v": c["v"], "k_scale": c["k_scale"], "v_scale": c["v_scale"]}


def _own(op, case, s):
    import commit_step_gb300 as cs

    if op == "append":
        cs.cache_append(s["handle"], s["k_new"], s["v_new"], s["table"], s["start"])
        return _held(s["cache"])
    if op == "attend":
        out, lse = cs.cache_attention(s["q"], s["handle"], s["table"], s["lens"], key_mask=s["mask"],
                                      weights=s["weights"], decay=0.0)
        return [out, lse] if s["weights"] is None else [out, lse, s["weights"]]
    if op == "evict":
        keep, lens, weights = cs.cache_evict(s["handle"], s["table"], s["lens"], s["weights"], case["budget"],
                                             s["dst"], keep_first=case["first"], keep_last=case["last"])
        return {"keep": keep, "lens": lens, "weights": weights, **_held(s["cache"])}
    if op == "score":
        r = cs.token_logprobs(s["logits"], s["targets"], top=case["top"], suppress_ids=s["ids"])
        return list(r if case["top"] else r[:3])
    return cs.token_logprobs_backward(s["logits"], s["targets"], s["lse"], s["entropy"], s["g_logprob"],
                                      grad_entropy=s["g_entropy"], top_ids=s["top_ids"], grad_top=s["g_top"],
                                      suppress_ids=s["ids"])


def _plain(op, case, s):
    if op == "append":
        _plain_append(s["cache"], "k", s["k_new"], s["table"], s["start"])
        _plain_append(s["cache"], "v", s["v_new"], s["table"], s["start"])
        return _held(s["cache"])
    if op == "attend":
        return _plain_attend(case, s)
    if op == "evict":
        return _plain_evict(case, s)
    if op == "score":
        r = _plain_score(s["logits"], s["targets"], case["top"], s["sup"])
        return list(r if case["top"] else r[:3])
    return _plain_grad(s)


def _power_scale(amax):
    """The smallest power of two 2^e, e >= -100, with amax / 2^e <= 448 (2^-100 for amax 0)."""
    m, e = torch.frexp(amax)                      # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(min=-100)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)                # the bits of 2^e


def _codes(x, scale):
    return torch.clamp(x / scale, -448.0, 448.0).to(torch.float8_e4m3fn)


def _plain_append(c, name, new, table, start):
    """Tokens new[b, j] go to positions start[b] + j, seen as a window of whole pages."""
    pool, scales = c[name], c[name + "_scale"]
    B, L, H, D = new.shape
    pages, _, ps, _ = pool.shape
    W = (L + ps - 1) // ps + 1                       # pages a window spans at most
    off = (start % ps).long()
    at = torch.arange(W * ps, device=new.device)[None, :] - off[:, None]         # (B, W ps): index into new
    fresh = (at >= 0) & (at < L)
    x = new.float().gather(1, at.clamp(0, L - 1)[:, :, None, None].expand(B, W * ps, H, D))
    x = torch.where(fresh[:, :, None, None], x, torch.zeros((), device=x.device))
    x = x.view(B, W, ps, H, D).transpose(2, 3)                                   # (B, W, H, ps, D)
    fresh = fresh.view(B, W, ps)
    scale = _power_scale(x.abs().amax((3, 4)))
    col = (start // ps).long()[:, None] + torch.arange(W, device=new.device)[None, :]
    page = table.long().gather(1, col.clamp(max=table.shape[1] - 1))
    page = torch.where(fresh.any(2), page, torch.full_like(page, pages - 1))     # untouched pages: the spare one
    old_codes = pool.view(torch.uint8)[page].view(torch.float8_e4m3fn)
    old_scale = scales[page]                                                     # (B, W, H)
    held = (at < 0).view(B, W, ps) & (page != pages - 1)[:, :, None]             # the tokens before the new ones
    begun = held.any(2)[:, :, None]
    scale = torch.where(begun, torch.maximum(scale, old_scale), scale)
    value = torch.where(held[:, :, None, :, None], old_codes.float() * old_scale[..., None, None], x)
    codes = _codes(value, scale[..., None, None]).view(torch.uint8)
    touched = (held | fresh)[:, :, None, :, None]
    codes = torch.where(touched, codes, old_codes.view(torch.uint8))
    spare = (page == pages - 1)[:, :, None]
    scale = torch.where(spare, old_scale, scale)
    pool.view(torch.uint8)[page.reshape(-1)] = codes.view(B * W, H, ps, D)
    scales[page.reshape(-1)] = scale.view(B * W, H)


def _values(c, name, table):
    """(B, H, width ps, D) fp32 of a table's pages."""
    pool, scales = c[name], c[name + "_scale"]
    t = table.long()
    x = pool.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * scales[t][..., None, None]
    B, W, H, ps, D = x.shape
    return x.transpose(1, 2).reshape(B, H, W * ps, D)


def _plain_attend(case, s):
    q, c, table, lens = s["q"], s["cache"], s["table"], s["lens"]
    B, L, Hq, D = q.shape
    H = case["H"]
    G = Hq // H
    k, v = _values(c, "k", table), _values(c, "v", table)
    n = k.shape[2]
    ok = torch.arange(n, device=q.device)[None, :] < lens[:, None]
    if s["mask"] is not None:
        ok = ok & (s["mask"] != 0)
    rows = q.float().view(B, L, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, L * G, D)
    x = torch.matmul(rows, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    x = torch.where(ok[:, None, None, :], x, torch.full((), -math.inf, device=x.device))
    m = x.amax(3, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    l = p.sum(3, keepdim=True)
    p = p / torch.where(l > 0, l, torch.ones_like(l))
    out = torch.matmul(p, torch.where(ok[:, None, :, None], v, torch.zeros((), device=v.device)))
    lse = (m + torch.log(l))[..., 0]
    out = out.view(B, H, L, G, D).permute(0, 2, 1, 3, 4).reshape(B, L, Hq, D).to(torch.bfloat16)
    lse = lse.view(B, H, L, G).permute(0, 2, 1, 3).reshape(B, L, Hq)
    if s["weights"] is None:
        return [out, lse]
    s["weights"].copy_(p.sum(2))
    return [out, lse, s["weights"]]


def _plain_evict(case, s):
    c, lens, w = s["cache"], s["lens"].long(), s["weights"]
    B, H, n = w.shape
    budget, first, last = case["budget"], case["first"], case["last"]
    at = torch.arange(n, device=w.device)
    here = at[None, :] < lens[:, None]
    always = here & ((at < first)[None, :] | (at[None, :] >= lens[:, None] - last))
    rank = torch.where(always[:, None], torch.full((), math.inf, device=w.device), w)
    rank = torch.where(here[:, None], rank, torch.full((), -math.inf, device=w.device))
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices[:, :, :budget]
    order = torch.sort(torch.where(order < lens[:, None, None], order, torch.full((), n, device=w.device)), dim=2).values
    if order.shape[2] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[2]), value=n)
    got = order < n
    keep = torch.where(got, order, torch.full((), -1, device=w.device)).to(torch.int32)
    weights = torch.zeros_like(w)
    m = min(budget, n)
    weights[:, :, :m] = torch.where(got, w.gather(2, order.clamp(max=n - 1)), torch.zeros((), device=w.device))[:, :, :m]
    pages, _, ps, D = c["k"].shape
    W = s["dst"].shape[1]
    src = torch.nn.functional.pad(order, (0, W * ps - budget), value=n).view(B, H, W, ps)
    got = src < n
    src = src.clamp(max=n - 1)
    page = s["table"].long()[torch.arange(B, device=w.device)[:, None, None, None], src // ps]
    head = torch.arange(H, device=w.device)[None, :, None, None].expand_as(src)
    used = got.any(3)                                                            # (B, H, W)
    to = s["dst"].long()[:, None, :].expand(B, H, W)
    _plain_move(c, "k", page, head, src % ps, got, to, used)
    _plain_move(c, "v", page, head, src % ps, got, to, used)
    return {"keep": keep, "lens": torch.clamp(lens, max=budget).to(torch.int32), "weights": weights, **_held(c)}


def _plain_move(c, name, page, head, slot, got, to, used):
    """The tokens (page, head, slot), each (B, H, W, ps), become the pages `to` (B, H, W) of the same pool."""
    pool, scales = c[name], c[name + "_scale"]
    x = pool.view(torch.uint8)[page, head, slot].view(torch.float8_e4m3fn).float()
    x = x * scales[page, head][..., None]
    x = torch.where(got[..., None], x, torch.zeros((), device=x.device))
    scale = _power_scale(x.abs().amax((3, 4)))
    old = pool.view(torch.uint8)[to, head[..., 0]]
    codes = _codes(x, scale[..., None, None]).view(torch.uint8)
    pool.view(torch.uint8)[to, head[..., 0]] = torch.where(got[..., None], codes, old)
    scales[to, head[..., 0]] = torch.where(used, scale, scales[to, head[..., 0]])


def _plain_score(logits, targets, top, sup):
    T, V = logits.shape
    z = logits.float()
    z = torch.where(torch.isnan(z), torch.full((), -math.inf, device=z.device), z)
    z = z.index_fill(1, sup, -math.inf)
    m = z.amax(1, keepdim=True)
    y = z - m
    e = torch.exp(y)
    Z = e.sum(1)
    ent = torch.log(Z) - torch.where(e > 0, e * y, torch.zeros((), device=z.device)).sum(1) / Z
    lse = m[:, 0] + torch.log(Z)
    t = targets.long()
    lp = torch.where(t >= 0, z.gather(1, t.clamp(min=0)[:, None])[:, 0] - lse, torch.zeros_like(lse))
    if not top:
        return lp, ent, lse, None, None
    bits = z.view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)                      # ordered as the values are
    key = key * 2 ** 20 + (2 ** 20 - 1 - torch.arange(V, device=z.device))[None, :]   # ties to the lower id
    ids = 2 ** 20 - 1 - (torch.topk(key, top, dim=1).values & (2 ** 20 - 1))
    return lp, ent, lse, ids.to(torch.int32), z.gather(1, ids) - lse[:, None]


def _plain_grad(s):
    z = s["logits"].float()
    z = z.index_fill(1, s["sup"], -math.inf)
    t = s["targets"].long()
    g = torch.where(t >= 0, s["g_logprob"], torch.zeros_like(s["g_logprob"]))
    y = z - s["lse"][:, None]
    p = torch.exp(y)
    total = g if s["g_top"] is None else g + s["g_top"].sum(1)
    bracket = total[:, None] + s["g_entropy"][:, None] * (torch.where(p > 0, y, torch.zeros((), device=z.device))
                                                          + s["entropy"][:, None])
    dz = -p * bracket
    dz.scatter_add_(1, t.clamp(min=0)[:, None], g[:, None])
    if s["g_top"] is not None:
        dz.scatter_add_(1, s["top_ids"].long(), s["g_top"])
    return dz.to(s["logits"].dtype)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _round_e4m3(x):
    """x rounded to e4m3 (ties to even), saturated at 448, in 64 bits."""
    a = x.abs().clamp(max=448.0)
    e = (torch.frexp(a.clamp(min=2.0 ** -20)).exponent - 1).clamp(min=-6).long()
    step = ((e - 3 + 1023) << 52).view(torch.float64)                           # the bits of 2^(e - 3)
    return torch.sign(x) * torch.clamp(torch.round(a / step) * step, max=448.0)


def _fit(amax):
    """2^e for the least e >= -100 with amax <= 448 2^e."""
    e = max(-100, math.ceil(math.log2(amax / 448.0))) if amax > 0 else -100
    while e > -100 and amax <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _fits(amax):
    return torch.tensor([_fit(a) for a in amax.flatten().tolist()], dtype=torch.float64,
                        device=amax.device).view(amax.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op == "append":
            return _exact_append(case, s)
        if op == "attend":
            return _exact_attend(case, s)
        if op == "evict":
            return _exact_evict(case, s)
        return _exact_score(case, s)


def _exact_append(case, s):
    c, out = s["cache"], {}
    L, ps = case["L"], case["ps"]
    if case["B"] * (L // ps + 2) > 3000:
        return None
    for name in ("k", "v"):
        pool, scales, new = c[name].double(), c[name + "_scale"].double(), s[name + "_new"].double()
        for b in range(case["B"]):
            start = int(s["start"][b])
            for col in range(start // ps, (start + L - 1) // ps + 1):
                page = int(s["table"][b, col])
                a, e = max(start, col * ps), min(start + L, (col + 1) * ps)
                x = new[b, a - start:e - start].transpose(0, 1)                  # (H, tokens, D)
                scale = _fits(x.abs().amax((1, 2)))
                held = a - col * ps
                if held:
                    scale = torch.maximum(scale, scales[page])
                    pool[page, :, :held] = _round_e4m3(pool[page, :, :held] * (scales[page] / scale)[:, None, None])
                pool[page, :, held:held + e - a] = _round_e4m3(x / scale[:, None, None])
                scales[page] = scale
        out[name], out[name + "_scale"] = pool, scales
    return out


def _exact_attend(case, s):
    B, L, Hq, D = s["q"].shape
    H, ps = case["H"], case["ps"]
    G = Hq // H
    if 4.0 * _cells(case) * L * G * D > 4e12:
        return None
    out = torch.zeros((B, L, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, L, Hq), -math.inf, dtype=torch.float64, device="cuda")
    weights = None if s["weights"] is None else torch.zeros_like(s["weights"], dtype=torch.float64)
    c = s["cache"]
    for b in range(B):
        n = int(s["lens"][b])
        at = torch.arange(n, device="cuda")
        if s["mask"] is not None:
            at = at[s["mask"][b, :n] != 0]
        if at.numel() == 0:
            continue
        page = s["table"][b].long()[at // ps]
        for h in range(H):
            k, v = [c[i].view(torch.uint8)[page, h, at % ps].view(torch.float8_e4m3fn).double()
                    * c[i + "_scale"][page, h].double()[:, None] for i in ("k", "v")]
            q = s["q"][b, :, h * G:(h + 1) * G].double().reshape(L * G, D)
            x = q @ k.T / math.sqrt(D)
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            out[b, :, h * G:(h + 1) * G] = (p @ v).view(L, G, D)
            lse[b, :, h * G:(h + 1) * G] = z.view(L, G)
            if weights is not None:
                weights[b, h, at] = p.sum(0)
    return [out, lse] if weights is None else [out, lse, weights]


def _exact_evict(case, s):
    B, H, n = s["weights"].shape
    ps, budget = case["ps"], case["budget"]
    c, lens = s["cache"], s["lens"].tolist()
    if B * H * (budget // ps + 1) > 12000:
        return None
    w = s["weights"].double().cpu()
    keep = torch.full((B, H, budget), -1, dtype=torch.int32)
    weights = torch.zeros((B, H, n), dtype=torch.float64)
    pools = {i: c[i].double() for i in ("k", "v")}
    scales = {i: c[i + "_scale"].double() for i in ("k", "v")}
    for b in range(B):
        m = lens[b]
        last = max(0, m - case["last"])
        for h in range(H):
            middle = [j for j in range(m) if case["first"] <= j < last]
            others = [j for j in range(m) if not case["first"] <= j < last]
            row = w[b, h].tolist()
            middle.sort(key=lambda j: (-row[j], j))
            ids = sorted(others + middle[:max(0, min(budget, m) - len(others))])
            keep[b, h, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
            at = torch.tensor(ids, device="cuda", dtype=torch.long)
            weights[b, h, :len(ids)] = w[b, h, ids]
            page = s["table"][b].long()[at // ps]
            for i in ("k", "v"):
                x = c[i].view(torch.uint8)[page, h, at % ps].view(torch.float8_e4m3fn).double()
                x = x * c[i + "_scale"][page, h].double()[:, None]
                for col in range(-(-len(ids) // ps)):
                    to = int(s["dst"][b, col])
                    y = x[col * ps:(col + 1) * ps]
                    scale = _fit(float(y.abs().max()))
                    pools[i][to, h, :y.shape[0]] = _round_e4m3(y / scale)
                    scales[i][to, h] = scale
    return {"keep": keep, "lens": torch.tensor([min(m, budget) for m in lens], dtype=torch.int32), "weights": weights,
            "k": pools["k"], "v": pools["v"], "k_scale": scales["k"], "v_scale": scales["v"]}


def _exact_score(case, s):
    T, V = s["logits"].shape
    rows = max(1, 2 ** 26 // V)
    parts = []
    for a in range(0, T, rows):
        z = s["logits"][a:a + rows].double()
        z[:, s["sup"]] = -math.inf
        lse = torch.logsumexp(z, 1)
        t = s["targets"][a:a + rows].long()
        y = z - lse[:, None]
        p = torch.exp(y)
        if case["op"] == "score":
            ent = -torch.nan_to_num(p * y, nan=0.0).sum(1)
            lp = torch.where(t >= 0, y.gather(1, t.clamp(min=0)[:, None])[:, 0], torch.zeros_like(lse))
            part = [lp, ent, lse]
            if case["top"]:
                order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["top"]]
                part += [order.to(torch.int32), y.gather(1, order)]
            parts.append(part)
            continue
        # the saved log-sum-exp and entropy are inputs of the backward pass
        lse, ent = s["lse"][a:a + rows].double(), s["entropy"][a:a + rows].double()
        y = z - lse[:, None]
        p = torch.exp(y)
        hot = torch.zeros_like(z)
        g = torch.where(t >= 0, s["g_logprob"][a:a + rows].double(), torch.zeros_like(lse))
        hot.scatter_add_(1, t.clamp(min=0)[:, None], g[:, None])
        if s["g_top"] is not None:
            hot.scatter_add_(1, s["top_ids"][a:a + rows].long(), s["g_top"][a:a + rows].double())
        d_ent = -torch.nan_to_num(p * (y + ent[:, None]), nan=0.0)
        parts.append([hot - p * hot.sum(1, keepdim=True) + s["g_entropy"][a:a + rows].double()[:, None] * d_ent])
    if case["op"] == "grad":
        return torch.cat([x[0] for x in parts]) if T * V * 8 < 2 ** 33 else None
    return [torch.cat([x[i] for x in parts]) for i in range(len(parts[0]))]
