"""Log probabilities of given tokens and their gradient on the GPU, against
64-bit formulas and against differences.

Tolerances (derived): log Z and the sums behind it are fp32 sums of up to V
terms, each off by 2^-21 of itself (exponent's rounding and the exponential),
added in chains of at most 2^9 and then by halves: 2^-15 of Z at the very
worst, so lse, log probabilities and the entropy are within 2^-15 + 2^-21
|value| (2^-12 for the entropy, whose terms carry the exponent as a factor of
up to 17).  The gradient's p = exp(z - lse) is off by 2^-20 (1 + |z - lse|) of
itself; each output is then rounded to its type (half a step).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def reference(z, targets, top, sup):
    """z: float64 (T, V) numpy."""
    T, V = z.shape
    z = np.where(np.isnan(z), -np.inf, z).copy()
    live = np.ones(V, dtype=bool)
    live[list(sup)] = False
    z[:, ~live] = -np.inf
    m = z.max(1)
    lse, ent, lp = np.empty(T), np.empty(T), np.zeros(T)
    logp = np.full((T, V), -np.inf)
    for t in range(T):
        if m[t] == np.inf:
            n = (z[t] == np.inf).sum()
            logp[t, z[t] == np.inf] = -math.log(n)
            lse[t], ent[t] = np.inf, math.log(n)
        elif m[t] == -np.inf:
            logp[t, live] = -math.log(live.sum())
            lse[t], ent[t] = -np.inf, math.log(live.sum())
        else:
            e = np.exp(z[t] - m[t])
            lse[t] = m[t] + math.log(e.sum())
            logp[t] = z[t] - m[t] - math.log(e.sum())
            p = e / e.sum()
            ent[t] = -(p[p > 0] * logp[t][p > 0]).sum()
        if 0 <= targets[t] < V:
            lp[t] = logp[t, targets[t]] if live[targets[t]] else -np.inf
    order = np.full((T, top), -1, dtype=np.int64)
    for t in range(T):
        ids = np.flatnonzero(live)
        order[t] = ids[np.lexsort((ids, -z[t, ids]))[:top]]
    return lp, ent, lse, order, np.take_along_axis(logp, order, 1) if top else None


def close(got, want, tol):
    g = got.double().cpu().numpy().reshape(want.shape)
    inf = ~np.isfinite(want)
    assert np.array_equal(g[inf], want[inf])
    err = np.abs(g[~inf] - want[~inf])
    lim = tol + 2.0 ** -21 * np.abs(want[~inf])
    assert (err <= lim).all(), (err.max(), tol)


def check(cs, z, targets, top=0, sup=()):
    """z: device (T, V)."""
    T, V = z.shape
    lp, ent, lse, ids, tlp = cs.token_logprobs(z, targets, top=top, suppress_ids=sup)
    want = reference(z.double().cpu().numpy(), targets.cpu().numpy(), top, sup)
    close(lp, want[0], 2.0 ** -15)
    close(ent, want[1], 2.0 ** -12)
    close(lse, want[2], 2.0 ** -15)
    if top:
        assert np.array_equal(ids.cpu().numpy(), want[3])
        close(tlp, want[4], 2.0 ** -15)
    else:
        assert ids is None and tlp is None


def logits(rng, T, V, dtype, scale=3.0):
    z = torch.from_numpy(rng.standard_normal((T, V)) * scale).to(dtype)
    for t in range(T):
        z[t, rng.integers(0, V)] += 9
    return z.cuda()


def some_targets(rng, T, V):
    t = rng.integers(0, V, T)
    t[::7] = -1
    return torch.from_numpy(t.astype(np.int32)).cuda()


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,top,n_sup", [(1, 1, 1, 0), (1, 2, 1, 1), (3, 7, 5, 2), (5, 33, 32, 1), (400, 300, 8, 5),
                                           (2, 8192, 20, 0), (64, 16385, 3, 64), (1, 50257, 0, 0), (31, 50257, 32, 5),
                                           (32, 126464, 8, 1), (310, 20001, 20, 1)])
def test_scores(cs, dtype, T, V, top, n_sup):
    rng = np.random.default_rng(T * V + top)
    sup = [int(v) for v in rng.permutation(V)[:n_sup]]
    check(cs, logits(rng, T, V, dtype), some_targets(rng, T, V), top, sup)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 5000, 70001])
def test_orders_that_defeat_a_running_threshold(cs, dtype, V):
    """Rows that ascend, descend, are all equal, hold few distinct values, or keep their best at either end."""
    rng = np.random.default_rng(V)
    z = torch.zeros((6, V), dtype=torch.float64)
    z[0] = torch.linspace(-8, 8, V)
    z[1] = torch.linspace(8, -8, V)
    z[2] = 1.5
    z[3] = torch.from_numpy(rng.integers(0, 3, V).astype(np.float64))
    z[4, -32:] = torch.arange(32) * 0.25
    z[5, :32] = -0.0
    z = z.to(dtype).cuda()
    check(cs, z, some_targets(rng, 6, V), 32, [0, V - 1, V // 2])


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [65, 33001])
def test_infinities_nan_and_extreme_values(cs, dtype, V):
    rng = np.random.default_rng(V + 1)
    z = logits(rng, 10, V, dtype)
    low = torch.finfo(dtype).min
    z[0] = -math.inf
    z[1] = math.nan
    z[2, 1::2] = math.nan
    z[3, 3:] = -math.inf
    z[4, 5], z[4, V - 1], z[4, 7] = math.inf, math.inf, math.nan
    z[5, 2:] = low                                       # a mask of the type's lowest value
    z[6] = low
    z[6, 9] = 0
    z[7] = -low                                          # the largest values, all equal
    z[8] = z[8] * 2.0 ** 60
    z[9, 0] = math.inf
    targets = torch.tensor([3, 4, 1, 40, 5, 30, 9, 2, 11, 0], dtype=torch.int32, device="cuda")
    check(cs, z, targets, 6, [0, 13])                    # (row 9's only +inf is suppressed)
    check(cs, z, targets.flip(0).contiguous(), 6, ())


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("offset,extra", [(0, 0), (1, 0), (3, 5), (8, 16), (5, 1)])
def test_unaligned_rows_and_strides(cs, dtype, offset, extra):
    rng = np.random.default_rng(offset * 10 + extra)
    T, V = 9, 4099
    wide = torch.full((T, V + offset + extra), math.nan, dtype=dtype, device="cuda")
    z = wide[:, offset:offset + V]
    z.copy_(logits(rng, T, V, dtype))
    targets = some_targets(rng, T, V)
    check(cs, z, targets, 10, [5, V - 1])
    check_grad(cs, z, targets, 4, [5, V - 1], rng)
    out = torch.full((T, V + 3), 5.0, dtype=dtype, device="cuda")
    check_grad(cs, z, targets, 4, [5, V - 1], rng, out=out[:, 2:2 + V])
    assert (out[:, :2] == 5).all() and (out[:, 2 + V:] == 5).all()


def test_batched_logits_shape(cs):
    rng = np.random.default_rng(0)
    z = logits(rng, 12, 1000, torch.bfloat16)
    t = some_targets(rng, 12, 1000)
    flat = cs.token_logprobs(z, t, top=3)
    batched = cs.token_logprobs(z.view(3, 4, 1000), t.view(3, 4), top=3)
    assert batched[0].shape == (3, 4) and batched[3].shape == (3, 4, 3)
    for a, b in zip(flat, batched):
        assert torch.equal(a.view(-1), b.reshape(-1))


def test_repeats_bit_for_bit(cs):
    rng = np.random.default_rng(2)
    z, t = logits(rng, 7, 90001, torch.bfloat16), some_targets(rng, 7, 90001)
    first = [x.clone() for x in cs.token_logprobs(z, t, top=20)]
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(first, cs.token_logprobs(z, t, top=20)))


# ---------------------------------------------------------------- gradient
def check_grad(cs, z, targets, top, sup, rng, out=None, in_place=False, parts=(True, True, True)):
    T, V = z.shape
    _, ent, lse, ids, _ = cs.token_logprobs(z, targets, top=top, suppress_ids=sup)
    g, ge = [torch.from_numpy(rng.standard_normal(T).astype(np.float32)).cuda() for _ in range(2)]
    gt = torch.from_numpy(rng.standard_normal((T, top)).astype(np.float32)).cuda() if top else None
    g, ge, gt = [x if on else None for x, on in zip((g, ge, gt), parts)]
    zd = z.double().cpu().numpy()
    if in_place:
        out = z
    dz = cs.token_logprobs_backward(z, targets, lse, ent, g, grad_entropy=ge, top_ids=ids, grad_top=gt,
                                    suppress_ids=sup, out=out)
    got = dz.double().cpu().numpy()
    # the formula in 64 bits, from the same saved lse and entropy
    ls, H = lse.double().cpu().numpy()[:, None], ent.double().cpu().numpy()[:, None]
    live = np.ones(V, dtype=bool)
    live[list(sup)] = False
    hot = np.zeros((T, V))
    t = targets.cpu().numpy()
    for r in range(T):
        if g is not None and 0 <= t[r] < V:
            hot[r, t[r]] += float(g[r])
        if gt is not None:
            np.add.at(hot[r], ids[r].cpu().numpy(), gt[r].double().cpu().numpy())
    hot[:, ~live] = 0
    e = np.zeros((T, 1)) if ge is None else ge.double().cpu().numpy()[:, None]
    total = hot.sum(1, keepdims=True)
    zd = np.where(np.isnan(zd), -np.inf, zd)
    with np.errstate(invalid="ignore"):
        y = zd - ls
        p = np.exp(y)
        inner = np.where(p > 0, total + e * (y + H), 0.0)
        want = hot - p * inner
        err_p = 2.0 ** -20 * (1 + np.abs(np.where(p > 0, y, 0)))
        size = np.abs(np.where(p > 0, p * (np.abs(hot).sum(1, keepdims=True) + np.abs(e) * (np.abs(y) + H)), 0.0))
    dead = ~np.isfinite(ls[:, 0])
    want[:, ~live] = 0
    want[dead] = 0
    size[dead] = 0
    half = torch.finfo(z.dtype).eps / 2
    tiny = 2.0 ** -126
    tol = half * np.abs(want) + (err_p + 2.0 ** -20) * size + 2.0 ** -22 * np.abs(hot) + tiny
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3], tol[bad][:3])
    return dz


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,top,n_sup", [(1, 1, 0, 0), (2, 2, 1, 1), (3, 7, 5, 2), (40, 300, 8, 5), (6, 16384, 0, 1),
                                           (5, 50257, 32, 64), (3, 126464, 4, 1)])
def test_gradient_formula(cs, dtype, T, V, top, n_sup):
    rng = np.random.default_rng(T + V)
    sup = [int(v) for v in rng.permutation(V)[:n_sup]]
    z, t = logits(rng, T, V, dtype), some_targets(rng, T, V)
    if n_sup:
        t[T - 1] = sup[0]                                # a suppressed target has no gradient
    apart = check_grad(cs, z, t, top, sup, np.random.default_rng(1))
    check_grad(cs, z, t, top, sup, rng, parts=(True, False, False))
    check_grad(cs, z, t, top, sup, rng, parts=(False, True, False))
    check_grad(cs, z, t, top, sup, rng, parts=(False, False, True))
    inplace = check_grad(cs, z, t, top, sup, np.random.default_rng(1), in_place=True)
    assert inplace.data_ptr() == z.data_ptr() and torch.equal(inplace, apart)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_gradient_of_rows_without_an_ordinary_softmax(cs, dtype):
    rng = np.random.default_rng(3)
    z = logits(rng, 6, 777, dtype)
    z[0] = -math.inf
    z[1] = math.nan
    z[2, 5] = math.inf
    z[3, 1::2] = math.nan
    z[4, 9:] = -math.inf
    z[5, 9:] = torch.finfo(dtype).min
    t = torch.tensor([1, 1, 5, 2, 3, 700], dtype=torch.int32, device="cuda")
    check_grad(cs, z, t, 4, [8], rng)


def test_repeated_named_ids_add_up(cs):
    """The target among the alternatives, an alternative given twice, ids out of range."""
    rng = np.random.default_rng(4)
    T, V = 3, 100
    z = logits(rng, T, V, torch.float32)
    t = torch.tensor([5, 5, -1], dtype=torch.int32, device="cuda")
    _, ent, lse, _, _ = cs.token_logprobs(z, t)
    ids = torch.tensor([[5, 7, 7, -1], [1, 2, 3, 100], [5, 5, 5, 5]], dtype=torch.int32, device="cuda")
    gt = torch.ones((T, 4), device="cuda")
    g = torch.ones(T, device="cuda")
    dz = cs.token_logprobs_backward(z, t, lse, ent, g, top_ids=ids, grad_top=gt).double()
    p = torch.softmax(z.double(), 1)
    hot = torch.zeros((T, V), dtype=torch.float64, device="cuda")
    hot[0, 5], hot[0, 7] = 2, 2
    hot[1, 5], hot[1, 1], hot[1, 2], hot[1, 3] = 1, 1, 1, 1
    hot[2, 5] = 4
    want = hot - p * hot.sum(1, keepdim=True)
    assert (dz - want).abs().max() < 4 * 2.0 ** -18


def test_gradient_against_differences(cs):
    """(f(z + h) - f(z - h)) / 2h of the scores themselves, fp32: off by h^2 / 6
    of the third derivative (at most 2 in sum of the parts) and by the scores'
    rounding over h."""
    rng = np.random.default_rng(5)
    T, V, top, h = 4, 50, 3, 2.0 ** -5
    z, t = logits(rng, T, V, torch.float32, scale=1.0), torch.tensor([3, 49, 0, 20], dtype=torch.int32, device="cuda")
    a, b, c = 0.7, -0.4, 0.3
    _, ent, lse, ids, _ = cs.token_logprobs(z, t, top=top)

    def value(x):
        lp, e, ls, _, _ = cs.token_logprobs(x, t)
        alt = x.gather(1, ids.long()) - ls[:, None]
        return (a * lp + b * e + c * alt.sum(1)).double()

    dz = cs.token_logprobs_backward(z, t, lse, ent, torch.full((T,), a, device="cuda"),
                                    grad_entropy=torch.full((T,), b, device="cuda"), top_ids=ids,
                                    grad_top=torch.full((T, top), c, device="cuda")).double()
    for v in range(V):
        up, down = z.clone(), z.clone()
        up[:, v] += h
        down[:, v] -= h
        diff = (value(up) - value(down)) / (2 * h)
        assert (diff - dz[:, v]).abs().max() < h * h / 6 * 8 + 2.0 ** -19 / h


def test_autograd(cs):
    rng = np.random.default_rng(6)
    z0, t = logits(rng, 8, 1000, torch.float32), some_targets(rng, 8, 1000)
    z = z0.clone().requires_grad_()
    lp, ent, ids, tlp = cs.score_tokens(z, t, top=2, suppress_ids=(7,))
    (lp.sum() - 0.1 * ent.mean() + (tlp * tlp).sum()).backward()
    y = z0.clone().double().requires_grad_()
    x = y.index_fill(1, torch.tensor([7], device="cuda"), -math.inf)
    logp = torch.log_softmax(x, 1)
    lp2 = torch.where(t >= 0, logp.gather(1, t.clamp(min=0).long()[:, None])[:, 0], 0.0)
    p = logp.exp()
    ent2 = -torch.where(p > 0, p * logp.clamp(min=-1e4), 0.0).sum(1)
    alt = logp.gather(1, ids.long())
    (lp2.sum() - 0.1 * ent2.mean() + (alt * alt).sum()).backward()
    assert (z.grad.double() - y.grad).abs().max() < 2.0 ** -15
    assert not ids.requires_grad


def test_score_in_a_graph_and_another_stream(cs):
    rng = np.random.default_rng(7)
    z, t = logits(rng, 16, 30000, torch.bfloat16), some_targets(rng, 16, 30000)
    want = cs.token_logprobs(z, t, top=4)
    out = [torch.empty_like(x) for x in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cs.token_logprobs(z, t, top=4, out=out)
        dz = cs.token_logprobs_backward(z, t, out[2], out[1], out[0])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert torch.equal(dz, cs.token_logprobs_backward(z, t, want[2], want[1], want[0]))
    with torch.cuda.stream(side):
        again = cs.token_logprobs(z, t, top=4)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, again))
