"""Scores of given tokens from hidden states, and their gradients, on the GPU
against 64-bit formulas.

Tolerances (derived).  A logit is a sum of d products, added in parts of at most
640 (1024 backward) one by one in 32 bits, truncated, and the parts rounded: off by
at most (640 + d / 640) 2^-23 sum |h w|, called e below (its largest over the ids).
lse and log probabilities move by at most 2 e, the entropy by at most e sum p |log p + H| <= 2 e (H + 1) <= 2 e (ln V + 1), beside
2^-15 + 2^-21 |value| (2^-12 for the entropy) of the sums of exponentials.

The gradient's dz is rounded to bf16 (2^-8 of itself at most) after the errors of z
(e) and of p (e, and 2^-18 for the exponent's roundings and the exponential), which
move it by that share of what it is made of (grad_parts: at a confident target what
is left of g - g p is far smaller); sums of n terms in 32 bits are off by n 2^-23 of
the sum of magnitudes at most; the result is rounded to its type.  So an element is
within (2^-8 + n 2^-23) sum |dz| |w| + (2 e + 2^-18) sum parts |w| + half a step.
That bound is wide for sums whose terms cancel, so the 2-norm of the whole error is
held too: two roundings of at most 2^-8, spread evenly, have a root mean square of
2^-8 / sqrt 3 each, sqrt(2 / 3) 2^-8 together (fp32 results: one), and 2^-8 is
asked for beside the second term's norm; of few rows a handful of elements decides,
which may all be off by the most: twice that.
"""
import ctypes
import math

import pytest
import torch

from head_reference import grad_parts, grads, scores

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def inputs(T, V, d, seed, scored=1.0, n_sup=0, spread=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn((V, d), device="cuda", generator=g) * spread / math.sqrt(d)).to(BF16)
    t = torch.randint(0, V, (T,), device="cuda", generator=g)
    h = torch.randn((T, d), device="cuda", generator=g) + torch.rand((T, 1), device="cuda", generator=g) * w[t].float()
    drop = torch.rand((T,), device="cuda", generator=g) >= scored
    t = torch.where(drop, torch.where(torch.rand((T,), device="cuda", generator=g) < 0.5, -1, V + 3), t).to(torch.int32)
    sup = torch.randperm(V, device="cuda", generator=g)[:n_sup].tolist()
    return h.to(BF16), w, t, sup


def logit_error(h, w, scored, part=640):
    """e, per row."""
    d = h.shape[1]
    terms = min(d, part) + d // part
    live = torch.where(scored[:, None], h.double(), torch.zeros((), dtype=torch.float64, device=h.device))
    return terms * 2.0 ** -23 * (live.abs() @ w.double().abs().T).amax(1)


def near(got, want, tol):
    got, want = got.double().reshape(want.shape), want.double()
    odd = ~torch.isfinite(want)
    assert torch.equal(got[odd], want[odd])
    err = (got[~odd] - want[~odd]).abs()
    lim = (tol + 2.0 ** -21 * want.abs())[~odd]
    assert bool((err <= lim).all()), (float(err.max()), float(lim.min()))


def check_scores(cs, h, w, t, sup, **kw):
    lp, ent, lse = cs.lm_head_logprobs(h, w, t, suppress_ids=sup, **kw)
    flat, tt, V = h.reshape(-1, h.shape[-1]), t.reshape(-1), w.shape[0]
    scored = (tt >= 0) & (tt < V)
    e = logit_error(flat, w, scored)
    clean = torch.where(scored[:, None], flat, torch.zeros((), dtype=flat.dtype, device=flat.device))
    want = scores(clean, w, tt, sup)
    near(lp, want[0], 2 * e + 2.0 ** -15)
    near(ent, want[1], 2 * e * (math.log(V) + 1) + 2.0 ** -12)
    near(lse, want[2], 2 * e + 2.0 ** -15)
    for x in (lp, ent, lse):
        assert x.shape == t.shape and not bool(x.reshape(-1)[~scored].any())
    return lp, ent, lse


def check_grad(got, dz, parts, by, e, old=None, dz_bits=8):
    """got against dz @ by (dz and its parts transposed for the weight's), dz rounded by 2^-dz_bits."""
    half = torch.finfo(got.dtype).eps / 2
    exact, by = dz @ by.double(), by.double().abs()
    want = exact if old is None else exact + old.double()
    slack = (2 * e + 2.0 ** -18) * (parts @ by)
    lim = (2.0 ** -dz_bits + dz.shape[1] * 2.0 ** -23) * (dz.abs() @ by) + slack + half * want.abs() + 1e-30
    err = (got.double() - want).abs()
    assert bool((err <= lim * (1 + half)).all()), float((err - lim).max())
    if exact.numel() >= 4096 and old is None:
        few = int((dz != 0).any(0).sum()) < 100 or int((dz != 0).any(1).sum()) < 100
        assert float(err.norm()) <= (2 if few else 1) * 2.0 ** -8 * float(want.norm()) + float(slack.norm())


def check_backward(cs, h, w, t, sup, with_entropy=True, with_logprob=True, seed=0, **kw):
    flat, tt = h.reshape(-1, h.shape[-1]), t.reshape(-1)
    T, V = flat.shape[0], w.shape[0]
    _, ent, lse = cs.lm_head_logprobs(h, w, t, suppress_ids=sup)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    gl = torch.randn(t.shape, device="cuda", generator=g) if with_logprob else None
    ge = torch.randn(t.shape, device="cuda", generator=g) * 0.2 if with_entropy else None
    gh, gw = cs.lm_head_logprobs_backward(h, w, t, lse, ent, gl, ge, suppress_ids=sup, **kw)
    what = (flat, w, tt, lse.reshape(-1), ent.reshape(-1), None if gl is None else gl.reshape(-1),
            None if ge is None else ge.reshape(-1), sup)
    (dz, clean), parts = grads(*what), grad_parts(*what)
    scored = (tt >= 0) & (tt < V)
    e = float(logit_error(flat, w, scored, 1024).max()) if T else 0.0
    if gh is not None:
        check_grad(gh.reshape(-1, h.shape[-1]), dz, parts, w, e)
        assert not bool(gh.reshape(-1, h.shape[-1])[~scored].any())
    if gw is not None and kw.get("accumulate") is None:
        check_grad(gw, dz.T, parts.T, clean, e)
    return gh, gw, dz, clean, parts


SIZES = [(1, 1, 8, 1.0, 0), (1, 2, 8, 1.0, 1), (3, 7, 16, 1.0, 2), (33, 300, 64, 0.5, 1), (61, 1000, 72, 1.0, 0),
         (128, 257, 200, 0.9, 5), (129, 513, 320, 1.0, 64), (65, 255, 1288, 1.0, 1), (300, 2049, 768, 0.3, 1),
         (64, 50257, 768, 1.0, 0), (700, 20001, 136, 0.6, 3), (1025, 1024, 512, 1.0, 0), (40, 126464, 256, 0.02, 1)]


@pytest.mark.parametrize("T,V,d,scored,n_sup", SIZES)
def test_scores(cs, T, V, d, scored, n_sup):
    check_scores(cs, *inputs(T, V, d, T + V, scored, n_sup))


@pytest.mark.parametrize("T,V,d,scored,n_sup", SIZES)
def test_gradients(cs, T, V, d, scored, n_sup):
    h, w, t, sup = inputs(T, V, d, T + V + 1, scored, n_sup)
    check_backward(cs, h, w, t, sup)
    check_backward(cs, h, w, t, sup, with_entropy=False)


def test_several_bands_and_pieces(cs):
    """More rows than one pass over the vocabulary takes, and a dz of several pieces, the last a short one."""
    h, w, t, sup = inputs(9000, 33000, 64, 5, 0.9, 1)
    check_scores(cs, h, w, t, sup)
    check_backward(cs, h, w, t, sup)


def test_few_scored_rows_of_many(cs):
    """Splits of the second product follow the scored rows, pieces all rows."""
    h, w, t, sup = inputs(70000, 9000, 64, 6, 0.004, 1)
    check_scores(cs, h, w, t, sup)
    check_backward(cs, h, w, t, sup)


def test_no_row_is_scored(cs):
    h, w, t, _ = inputs(70, 500, 64, 7, 0.0)
    h.fill_(math.nan)
    lp, ent, lse = cs.lm_head_logprobs(h, w, t)
    assert not bool(lp.any() or ent.any() or lse.any())
    one = torch.ones(70, device="cuda")
    gh, gw = cs.lm_head_logprobs_backward(h, w, t, lse, ent, one, one)
    assert not bool(gh.any() or gw.any())
    old = torch.randn_like(w)
    kept = old.clone()
    _, same = cs.lm_head_logprobs_backward(h, w, t, lse, ent, one, one, out=(None, old), accumulate=True)
    assert same is old and torch.equal(old, kept)


@pytest.mark.parametrize("T", [70, 300, 9000])
@pytest.mark.parametrize("dtype", [BF16, torch.float32], ids=["bf16", "f32"])
def test_no_row_takes_part(cs, T, dtype):
    """Every row scored and none with a gradient: the weight's is zero in either type, and adding leaves what is there."""
    h, w, t, _ = inputs(T, 500, 64, 77)
    _, ent, lse = cs.lm_head_logprobs(h, w, t)
    none = torch.zeros(T, device="cuda")
    wide = torch.full((500, 72), 7.0, dtype=dtype, device="cuda")
    gh, gw = cs.lm_head_logprobs_backward(h, w, t, lse, ent, none, none, out=(None, wide[:, :64]), accumulate=True)
    assert not bool(gh.any()) and bool((wide == 7).all())
    cs.lm_head_logprobs_backward(h, w, t, lse, ent, none, out=(None, wide[:, :64]))
    assert not bool(wide[:, :64].any()) and bool((wide[:, 64:] == 7).all())


def test_no_rows(cs):
    h, w, _, _ = inputs(4, 100, 64, 8)
    h, t, f = h[:0], torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    assert [x.numel() for x in cs.lm_head_logprobs(h, w, t)] == [0, 0, 0]
    for dtype in (BF16, torch.float32):
        wide = torch.full((100, 72), 7.0, dtype=dtype, device="cuda")
        gh, gw = cs.lm_head_logprobs_backward(h, w, t, f, f, f, out=(None, wide[:, :64]))
        assert gh.shape == (0, 64) and not bool(wide[:, :64].any()) and bool((wide[:, 64:] == 7).all())


def test_nan_and_infinities_where_no_row_is_scored(cs):
    """Rows without a target, without a gradient or with a lost log-sum-exp are in no result."""
    h, w, t, sup = inputs(200, 777, 128, 9, 0.5, 1)
    dead = t < 0
    h[dead] = math.nan
    h[t > 776] = math.inf
    check_scores(cs, h, w, t, sup)
    _, ent, lse = cs.lm_head_logprobs(h, w, t, suppress_ids=sup)
    live = torch.nonzero((t >= 0) & (t < 777))[:, 0]
    gl, ge = torch.ones(200, device="cuda"), torch.zeros(200, device="cuda")
    gl[live[3]] = 0.0
    h[live[3]] = math.nan
    lse[live[5]] = math.inf
    h[live[5]] = -math.inf
    gh, gw = cs.lm_head_logprobs_backward(h, w, t, lse, ent, gl, ge, suppress_ids=sup)
    assert bool(torch.isfinite(gh).all()) and bool(torch.isfinite(gw).all())
    assert not bool(gh[live[3]].any()) and not bool(gh[live[5]].any())
    (dz, clean), parts = grads(h, w, t, lse, ent, gl, ge, sup), grad_parts(h, w, t, lse, ent, gl, ge, sup)
    e = float(logit_error(clean, w, torch.ones_like(dead), 1024).max())
    check_grad(gh, dz, parts, w, e)
    check_grad(gw, dz.T, parts.T, clean, e)


def test_rows_without_mass_and_with_infinite_logits(cs):
    """NaN and infinite products read as dllm_token_logprobs reads such logits."""
    V, d = 300, 64
    h = torch.zeros((6, d), device="cuda")
    h[:, 0] = 1.0
    h[1, 0] = math.nan                                   # every product NaN
    h[3, 0] = 0.0                                        # every product 0
    h[4, 0] = 2.0 ** 120                                 # products beyond any bound but finite differences
    h[5, 0] = -2.0 ** 100
    w = torch.zeros((V, d), device="cuda")
    w[:, 0] = torch.linspace(-3, 3, V, device="cuda")
    h, w = h.to(BF16), w.to(BF16)
    t = torch.tensor([5, 5, 299, 7, 299, 0], dtype=torch.int32, device="cuda")
    lp, ent, lse = cs.lm_head_logprobs(h, w, t, suppress_ids=[17])
    want = scores(h, w, t, [17])
    e = torch.full((6,), 2.0 ** -12, device="cuda", dtype=torch.float64)
    near(lp, want[0], e)
    near(ent, want[1], 10 * e)
    near(lse, want[2], e)
    assert float(lse[1]) == -math.inf and abs(float(lp[1]) + math.log(299)) < 1e-5
    w[40, 0], w[41, 0] = math.inf, math.inf              # two ids share all the mass
    lp, ent, lse = cs.lm_head_logprobs(h[:1], w, torch.tensor([41], dtype=torch.int32, device="cuda"))
    assert float(lse[0]) == math.inf and abs(float(lp[0]) + math.log(2)) < 1e-5 and abs(float(ent[0]) - math.log(2)) < 1e-5


@pytest.mark.parametrize("T", [5, 200])
@pytest.mark.parametrize("far", [-2.0 ** 62, -2.0 ** 66, -2.0 ** 67, math.nan])
def test_an_id_without_mass_under_a_large_entropy_gradient(cs, T, far):
    """An id whose logit is far below the others' (-2^122 .. -2^127, or NaN) has no gradient, however large the entropy's:
    bit for bit what suppressing it gives."""
    h, w, t, _ = inputs(T, 300, 64, 80 + T)
    h[:, 0], w[:, 0] = 2.0 ** 60, 0.0
    w[17, 0] = far
    t[t == 17] = 3
    _, ent, lse = cs.lm_head_logprobs(h, w, t)
    assert bool((lse.abs() < 100).all())
    gl, ge = torch.randn(T, device="cuda"), torch.randn(T, device="cuda") * 1e4
    finite = not math.isnan(far)                         # (times 0 a NaN would reach grad_hidden)
    got = cs.lm_head_logprobs_backward(h, w, t, lse, ent, gl, ge, hidden_grad=finite)
    want = cs.lm_head_logprobs_backward(h, w, t, lse, ent, gl, ge, suppress_ids=[17], hidden_grad=finite)
    assert bool(torch.isfinite(got[1]).all()) and torch.equal(got[1], want[1])
    assert not finite or (bool(torch.isfinite(got[0]).all()) and torch.equal(got[0], want[0]))


def test_suppressed_target(cs):
    h, w, t, _ = inputs(9, 333, 64, 10)
    t[4] = 11
    lp, ent, lse = check_scores(cs, h, w, t, [11, 12])
    assert float(lp[4]) == -math.inf
    one = torch.ones(9, device="cuda")
    gh, gw = cs.lm_head_logprobs_backward(h, w, t, lse, ent, one, suppress_ids=[11, 12])
    assert not bool(gh[4].any()) and bool(gh[3].any()) and not bool(gw[11].any() or gw[12].any())
    check_backward(cs, h, w, t, [11, 12])


def test_one_wanted_gradient(cs):
    h, w, t, sup = inputs(150, 700, 96, 11, 0.7, 1)
    both = check_backward(cs, h, w, t, sup)
    only_h = check_backward(cs, h, w, t, sup, weight_grad=False)
    only_w = check_backward(cs, h, w, t, sup, hidden_grad=False)
    assert only_h[1] is None and only_w[0] is None
    assert torch.equal(only_h[0], both[0]) and torch.equal(only_w[1], both[1])


@pytest.mark.parametrize("dtype", [BF16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_given_outputs(cs, dtype, accumulate):
    """Rows of wider tensors, and adding to what is there (rows no token moves among it)."""
    T, V, d = 130, 600, 136
    h, w, t, sup = inputs(T, V, d, 12, 0.8, 2)
    gw_all = torch.randn((V, d + 24), device="cuda").to(dtype)
    gh_all = torch.randn((T, d + 8), device="cuda").to(BF16)
    old = gw_all.clone()
    before = gh_all.clone()
    gh, gw, dz, clean, parts = check_backward(cs, h, w, t, sup, out=(gh_all[:, :d], gw_all[:, :d]),
                                          **({"accumulate": True} if accumulate else {}))
    assert gw.data_ptr() == gw_all.data_ptr() and torch.equal(gw_all[:, d:], old[:, d:])
    assert torch.equal(gh_all[:, d:], before[:, d:])
    e = float(logit_error(h, w, (t >= 0) & (t < V), 1024).max())
    check_grad(gw, dz.T, parts.T, clean, e, old[:, :d] if accumulate else None)


@pytest.mark.parametrize("dtype", [BF16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,d", [(40, 9001, 520), (700, 30011, 264), (300, 2000, 64)])
def test_adding_over_many_tiles(cs, dtype, T, V, d):
    """Micro-batches added to one gradient: each call adds its own, rounded once."""
    h, w, t, sup = inputs(T, V, d, V, 0.9, 1)
    gw = torch.randn((V, d), device="cuda").to(dtype) * 0.1
    e = float(logit_error(h, w, (t >= 0) & (t < V), 1024).max())
    for seed in range(2):
        old = gw.clone()
        gh, got, dz, clean, parts = check_backward(cs, h, w, t, sup, seed=seed, out=(None, gw), accumulate=True)
        assert got is gw
        check_grad(gw, dz.T, parts.T, clean, e, old)


@pytest.mark.parametrize("T,V,d,scored", [(1, 300, 64, 1.0), (7, 5000, 136, 1.0), (64, 3001, 256, 0.5), (65, 1000, 520, 1.0),
                                          (128, 40000, 72, 0.9)])
def test_few_rows_keep_what_bf16_cuts_off(cs, T, V, d, scored):
    """dz in two parts: 2^-16 of an element is lost, so a gradient in 32 bits is that exact, and one in bf16 is off by its
    own rounding (2^-8 / sqrt 3 in the root mean square, 0.6 of 2^-8 asked for)."""
    h, w, t, sup = inputs(T, V, d, 90 + T, scored, 1)
    wide = torch.empty((V, d), device="cuda")
    gh, gw, dz, clean, parts = check_backward(cs, h, w, t, sup, out=(None, wide))
    e = float(logit_error(h, w, (t >= 0) & (t < V), 1024).max())
    check_grad(wide, dz.T, parts.T, clean, e, dz_bits=16)
    check_grad(gh, dz, parts, w, e, dz_bits=16)
    narrow = check_backward(cs, h, w, t, sup)[1]
    want = dz.T @ clean
    slack = (2 * e + 2.0 ** -18) * (parts.T @ clean.abs())
    if want.numel() >= 4096:
        assert float((narrow.double() - want).norm()) <= 0.6 * 2.0 ** -8 * float(want.norm()) + float(slack.norm())


@pytest.mark.parametrize("T,V,d,scored", [(129, 300, 64, 0.02), (300, 3001, 256, 0.03), (8192, 5000, 136, 0.002),
                                          (200, 1000, 520, 0.55), (20000, 9000, 64, 0.005)])
def test_few_scored_rows_of_many_keep_what_bf16_cuts_off(cs, T, V, d, scored):
    """The parts of dz go by the rows that take part, not by the rows given."""
    h, w, t, sup = inputs(T, V, d, 95 + T, scored, 1)
    n = int(((t >= 0) & (t < V)).sum())
    assert 0 < n <= 128
    wide = torch.empty((V, d), device="cuda")
    gh, gw, dz, clean, parts = check_backward(cs, h, w, t, sup, out=(None, wide))
    e = float(logit_error(h, w, (t >= 0) & (t < V), 1024).max())
    check_grad(wide, dz.T, parts.T, clean, e, dz_bits=16)
    check_grad(gh, dz, parts, w, e, dz_bits=16)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,V,d,scored", [(129, 200, 64, 1.0), (257, 513, 72, 1.0), (300, 3000, 520, 0.6), (1025, 2049, 264, 1.0),
                                          (700, 30011, 136, 0.9), (9000, 33000, 64, 0.9), (8192, 700, 128, 0.7)])
def test_a_weight_gradient_in_32_bits_keeps_what_bf16_cuts_off(cs, T, V, d, scored, accumulate):
    """dz in two parts for it, however many rows take part."""
    h, w, t, sup = inputs(T, V, d, 97 + T, scored, 1)
    wide = torch.randn((V, d), device="cuda") * 0.1
    old = wide.clone() if accumulate else None
    gh, gw, dz, clean, parts = check_backward(cs, h, w, t, sup, out=(None, wide), **({"accumulate": True} if accumulate else {}))
    assert int((dz != 0).any(1).sum()) > 128
    e = float(logit_error(h, w, (t >= 0) & (t < V), 1024).max())
    check_grad(wide, dz.T, parts.T, clean, e, old, dz_bits=16)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [BF16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,d", [(8200, 300, 72), (17000, 600, 136)])
def test_weight_gradients_in_several_parts(cs, T, V, d, dtype, accumulate):
    """More rows than one accumulator takes, stored and added to in either type."""
    h, w, t, sup = inputs(T, V, d, 99 + T, 1.0, 1)
    gw = (torch.randn((V, d), device="cuda") * 0.1).to(dtype)
    old = gw.clone() if accumulate else None
    _, _, dz, clean, parts = check_backward(cs, h, w, t, sup, out=(None, gw), **({"accumulate": True} if accumulate else {}))
    e = float(logit_error(h, w, (t >= 0) & (t < V), 1024).max())
    check_grad(gw, dz.T, parts.T, clean, e, old, dz_bits=8 if dtype is BF16 else 16)


@pytest.mark.parametrize("T", [1 << 15, 1 << 21])
def test_long_sums_of_one_sign_do_not_drift(cs, T):
    """A weight's gradient of many rows, every term of a sum of one sign.  The tensor core cuts off what 32 bits do not hold,
    product by product at worst, so a part of 8192 products is off by 8192 2^-23 of itself at most; the parts of dz's two
    are added rounded (2 T / 8192 2^-24).  In 32 bits an element of dz is off by 2^-16 of itself at most (rounded to bf16 it
    would be by 2^-8, and where all terms are nearly one value, 1 - p near 1, all of them the same way)."""
    V, d = 64, 64
    g = torch.Generator(device="cuda").manual_seed(T)
    h = (torch.rand((T, d), device="cuda", generator=g) + 0.5).to(BF16)
    w = (torch.randn((V, d), device="cuda", generator=g) * 0.1).to(BF16)
    t = torch.zeros(T, dtype=torch.int32, device="cuda")
    one = torch.ones(T, device="cuda")
    _, ent, lse = cs.lm_head_logprobs(h, w, t)
    got = torch.empty((V, d), device="cuda")
    cs.lm_head_logprobs_backward(h, w, t, lse, ent, one, hidden_grad=False, out=(None, got))
    dz, clean = grads(h, w, t, lse, ent, one, None)
    assert bool((dz[:, 0] >= 0).all()) and bool((dz[:, 1:] <= 0).all())
    want = dz.T @ clean
    e = float(logit_error(h, w, torch.ones_like(t, dtype=torch.bool), 1024).max())
    lim = 8192 * 2.0 ** -23 + T / 4096 * 2.0 ** -24 + 2.0 ** -16
    part = grad_parts(h, w, t, lse, ent, one, None, [])
    slack = (2 * e + 2.0 ** -18) * (part.T @ clean)
    assert bool(((got.double() - want).abs() <= lim * want.abs() + slack).all()), float(((got - want) / want).abs().max())


def test_strided_inputs_and_batches(cs):
    h, w, t, sup = inputs(150, 700, 96, 13, 0.7, 1)
    hw = torch.full((150, 200), math.nan, dtype=BF16, device="cuda")
    ww = torch.full((700, 104), math.nan, dtype=BF16, device="cuda")
    hw[:, :96], ww[:, :96] = h, w
    a = check_scores(cs, h.view(3, 50, 96), w, t.view(3, 50), sup)
    b = cs.lm_head_logprobs(hw[:, :96], ww[:, :96], t, suppress_ids=sup)
    assert all(torch.equal(x.reshape(-1), y) for x, y in zip(a, b))
    g = torch.ones(150, device="cuda")
    c = cs.lm_head_logprobs_backward(h, w, t, b[2], b[1], g, suppress_ids=sup)
    e = cs.lm_head_logprobs_backward(hw[:, :96], ww[:, :96], t, b[2], b[1], g, suppress_ids=sup)
    assert torch.equal(c[0], e[0]) and torch.equal(c[1], e[1])


def far(x, step):
    """x in rows of `step` elements."""
    wide = torch.empty((x.shape[0] * step,), dtype=x.dtype, device=x.device).as_strided(x.shape, (step, 1))
    return wide.copy_(x)


@pytest.mark.parametrize("T", [300, 200])
def test_offsets_past_32_bits(cs, T):
    h, w, t, sup = inputs(T, 1000, 64, 60 + T, 0.8, 2)
    h, w = far(h, 1 << 24), far(w, 1 << 22)
    check_scores(cs, h, w, t, sup)
    check_backward(cs, h, w, t, sup, out=(far(h, 1 << 24), far(w.float(), 1 << 22)))
    check_backward(cs, h, w, t, sup, out=(far(h, 1 << 24), far(w, 1 << 22)))


def test_results_repeat_and_do_not_depend_on_the_workspace(cs):
    h, w, t, sup = inputs(900, 30000, 256, 14, 0.5, 1)
    g = torch.randn(900, device="cuda")
    runs = []
    for fill in (0, 255):
        need = cs.lib_handle().dllm_lm_head_logprobs_workspace_size(900, 30000, 256)
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        s = cs.lm_head_logprobs(h, w, t, suppress_ids=sup, ws=ws)
        need = cs.lib_handle().dllm_lm_head_logprobs_backward_workspace_size(900, 30000, 256)
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        runs.append([*s, *cs.lm_head_logprobs_backward(h, w, t, s[2], s[1], g, g, suppress_ids=sup, ws=ws)])
        if fill == 0:
            assert cs.workspace_fault(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("T,V,d,scored", [(61, 1000, 72, 1.0), (300, 3000, 64, 0.5)])
def test_workspaces_at_any_16_bytes(cs, T, V, d, scored):
    """A workspace of just the size asked for, wherever it begins: the same results, and nothing behind it is touched."""
    h, w, t, sup = inputs(T, V, d, 70 + T, scored, 1)
    g = torch.randn(T, device="cuda")
    want = [*cs.lm_head_logprobs(h, w, t, suppress_ids=sup)]
    want += cs.lm_head_logprobs_backward(h, w, t, want[2], want[1], g, g, suppress_ids=sup)
    sizes = [int(getattr(cs.lib_handle(), f"dllm_lm_head_logprobs_{x}workspace_size")(T, V, d)) for x in ("", "backward_")]
    for shift in (16, 32, 48, 128, 240, 256):
        pools = [torch.zeros(shift + need + 64, dtype=torch.uint8, device="cuda") for need in sizes]
        ws = [pool[shift:shift + need] for pool, need in zip(pools, sizes)]
        assert all(x.data_ptr() % 256 == shift % 256 for x in ws)
        got = [*cs.lm_head_logprobs(h, w, t, suppress_ids=sup, ws=ws[0])]
        got += cs.lm_head_logprobs_backward(h, w, t, got[2], got[1], g, g, suppress_ids=sup, ws=ws[1])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(cs.workspace_fault(x) == 0 for x in ws)
        assert not any(bool(pool[:shift].any() or pool[shift + need:].any()) for pool, need in zip(pools, sizes))


def test_the_devices_fault_word(cs):
    """It is read and cleared, and calls whose waits end leave it alone.  (The code that a kernel would leave is written by
    the test.)"""
    lib, code, word = cs.lib_handle(), ctypes.c_int32(2), ctypes.c_void_p()
    assert lib.dllm_fault_word(ctypes.byref(word)) == 0
    assert cs.kernel_fault() == 0
    lib.cudaMemcpy.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]     # (its runtime's)
    assert lib.cudaMemcpy(word, ctypes.byref(code), 4, 1) == 0
    h, w, t, sup = inputs(300, 3000, 64, 18, 0.5, 1)
    ha, wa = h.clone().requires_grad_(), w.clone().requires_grad_()
    cs.score_hidden(ha, wa, t)[0].sum().backward()
    cs.embed_tokens_backward(t, h, 3000)
    assert cs.kernel_fault() == 2 and cs.kernel_fault() == 0
    cs.score_hidden(ha, wa, t)[0].sum().backward()
    cs.embed_tokens_backward(t, h, 3000, stream=torch.cuda.Stream())
    assert cs.kernel_fault() == 0


def test_autograd(cs):
    h, w, t, sup = inputs(77, 900, 128, 15, 0.6, 1)
    ha, wa = h.view(7, 11, 128).clone().requires_grad_(), w.clone().requires_grad_()
    lp, ent = cs.score_hidden(ha, wa, t.view(7, 11), suppress_ids=sup)
    (lp.sum() * -0.5 + 0.1 * ent.sum()).backward()
    l0, e0, s0 = cs.lm_head_logprobs(h, w, t, suppress_ids=sup)
    one = torch.ones(77, device="cuda")
    gh, gw = cs.lm_head_logprobs_backward(h, w, t, s0, e0, -0.5 * one, 0.1 * one, suppress_ids=sup)
    assert torch.equal(lp.reshape(-1), l0) and torch.equal(ent.reshape(-1), e0)
    assert torch.equal(ha.grad.reshape(77, 128), gh) and torch.equal(wa.grad, gw)
    lp, _ = cs.score_hidden(h.requires_grad_(), w, t, suppress_ids=sup)      # one output, one input
    lp.mean().backward()
    assert h.grad is not None and w.grad is None
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        lp, _ = cs.score_hidden(ha, wa, t.view(7, 11))
        g, = torch.autograd.grad(lp.sum(), ha, create_graph=True)
        g.float().sum().backward()


@pytest.mark.parametrize("B,L", [(3, 21), (5, 1), (1, 40), (2, 300)])
def test_autograd_of_windows(cs, B, L):
    """Shifted scoring: hidden states without their last position, targets without their first; and other strides."""
    h, w, t, sup = inputs(B * (L + 1), 700, 64, 90 + L, 0.8, 1)
    h, t = h.view(B, L + 1, 64), t.view(B, L + 1)
    wide = torch.zeros((B, L + 1, 68), dtype=BF16, device="cuda")
    wide[..., 4:] = h
    want = None
    for x, y in ((h[:, :-1].contiguous(), t[:, 1:].contiguous()), (h[:, :-1], t[:, 1:]), (wide[:, :-1, 4:], t[:, 1:]),
                 (h[:, :-1].transpose(0, 1).contiguous().transpose(0, 1), t[:, 1:].T.contiguous().T),
                 (h[:, :-1].transpose(1, 2).contiguous().transpose(1, 2), t[:, 1:])):
        x, v = x.detach().requires_grad_(), w.clone().requires_grad_()
        lp, ent = cs.score_hidden(x, v, y, suppress_ids=sup)
        (torch.nan_to_num(lp, neginf=0.0).sum() + 0.1 * ent.sum()).backward()
        got = lp, ent, x.grad, v.grad
        assert lp.shape == y.shape and x.grad.shape == x.shape
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    row = h[:1, :1].clone().requires_grad_()
    lp, _ = cs.score_hidden(row.expand(B, L, 64), w, t[:, 1:])
    lp.sum().backward()
    each = h[:1, :1].expand(B, L, 64).contiguous().requires_grad_()
    cs.score_hidden(each, w, t[:, 1:])[0].sum().backward()
    assert torch.equal(row.grad, each.grad.sum((0, 1), keepdim=True))


def test_matches_the_scores_of_stored_logits(cs):
    """The same model through logits in memory: one softmax, one loss."""
    h, w, t, sup = inputs(64, 4000, 256, 16, 1.0, 1)
    z = h.float() @ w.float().T
    want = cs.token_logprobs(z, t, suppress_ids=sup)
    got = cs.lm_head_logprobs(h, w, t, suppress_ids=sup)
    for a, b in zip(got, want[:3]):
        assert float((a - b).abs().max()) < 1e-3
    e = float(logit_error(h, w, torch.ones_like(t, dtype=torch.bool)).max())
    assert float((got[0] - want[0]).abs().max()) <= 4 * e + 2.0 ** -14


def test_confident_rows_of_long_sums(cs):
    """Log probabilities near 0, -ln(1 + sum over the others of exp(z_v - z_t)): off by the differences' errors, 2 e, times
    themselves, and 2^-20 of the exponentials."""
    T, V, d = 8, 300, 4096
    g = torch.Generator(device="cuda").manual_seed(21)
    w = (torch.randn((V, d), device="cuda", generator=g) * 2.5 / math.sqrt(d)).to(BF16)
    t = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    h = (torch.randn((T, d), device="cuda", generator=g) + 2.5 * w[t.long()].float()).to(BF16)
    lp = cs.lm_head_logprobs(h, w, t)[0]
    want = scores(h, w, t)[0]
    e = logit_error(h, w, torch.ones_like(t, dtype=torch.bool))
    assert float(want.max()) > -0.05
    assert bool(((lp.double() - want).abs() <= (2 * e + 2.0 ** -20) * want.abs() + 2.0 ** -23).all())


def test_two_threads_on_one_stream(cs):
    import threading

    jobs = []
    for i in range(2):
        h, w, t, sup = inputs(200 + 77 * i, 3000 + 999 * i, 128, 30 + i, 0.6, 1)
        g = torch.randn(t.shape, device="cuda")
        first = [*cs.lm_head_logprobs(h, w, t, suppress_ids=sup)]
        first += cs.lm_head_logprobs_backward(h, w, t, first[2], first[1], g, g, suppress_ids=sup)
        jobs.append((h, w, t, sup, g, first))
    torch.cuda.synchronize()
    bad = []

    def work(h, w, t, sup, g, first):
        for _ in range(30):
            got = [*cs.lm_head_logprobs(h, w, t, suppress_ids=sup)]
            got += cs.lm_head_logprobs_backward(h, w, t, got[2], got[1], g, g, suppress_ids=sup)
            if not all(torch.equal(a, b) for a, b in zip(got, first)):
                bad.append(t.shape)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not bad


def test_two_graphs_at_once(cs):
    """Graphs hold memory of their own: replayed on two streams together, neither meets the other's workspace."""
    cases, graphs, outs = [], [], []
    for i in range(2):
        h, w, t, sup = inputs(150 + i, 20000, 256, 40 + i, 0.7, 0)
        g = torch.randn(t.shape, device="cuda")
        want = [*cs.lm_head_logprobs(h, w, t)]
        want += cs.lm_head_logprobs_backward(h, w, t, want[2], want[1], g)
        cases.append((h, w, t, g, want))
    torch.cuda.synchronize()
    for h, w, t, g, _ in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = [*cs.lm_head_logprobs(h, w, t)]
            got += cs.lm_head_logprobs_backward(h, w, t, got[2], got[1], g)
        graphs.append(graph)
        outs.append(got)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for got, (_, _, _, _, want) in zip(outs, cases):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_of_other_sizes_in_between(cs):
    """A kept workspace serves calls of any size and kind in turn."""
    h, w, t, sup = inputs(64, 2000, 64, 50, 1.0, 1)
    big = inputs(300, 9000, 512, 51, 0.5, 1)
    first = cs.lm_head_logprobs(h, w, t, suppress_ids=sup)
    for _ in range(3):
        cs.lm_head_logprobs(*big[:3], suppress_ids=big[3])
        cs.embed_tokens_backward(t, h, 2000)
        again = cs.lm_head_logprobs(h, w, t, suppress_ids=sup)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_the_binding_refuses(cs):
    h, w, t, _ = inputs(8, 100, 64, 60)
    f = torch.zeros(8, device="cuda")
    for bad in (lambda: cs.lm_head_logprobs(h.float(), w, t), lambda: cs.lm_head_logprobs(h, w.half(), t),
                lambda: cs.lm_head_logprobs(h[None, None], w, t), lambda: cs.score_hidden(h, w[0], t),
                lambda: cs.lm_head_logprobs(h, w, t, ws="no")):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: cs.lm_head_logprobs(h, w[:, :32], t), lambda: cs.lm_head_logprobs(h, w, t.long()),
                lambda: cs.lm_head_logprobs(h, w, t[:7]), lambda: cs.lm_head_logprobs(h.T, w, t),
                lambda: cs.lm_head_logprobs(h, w, t, suppress_ids=[1 << 33]),
                lambda: cs.lm_head_logprobs(h, w, t, ws=torch.zeros(8, dtype=torch.uint8)),
                lambda: cs.lm_head_logprobs_backward(h, w, t, f, f, f, accumulate=True),
                lambda: cs.lm_head_logprobs_backward(h, w, t, f, f, f, out=(h.clone(), None), hidden_grad=False),
                lambda: cs.lm_head_logprobs_backward(h, w, t, f, f, f, out=(None, w.half())),
                lambda: cs.lm_head_logprobs_backward(h, w, t, f, f, f, out=(None, w[:50].clone())),
                lambda: cs.lm_head_logprobs_backward(h, w, t, f[:4], f, f)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cs.lm_head_logprobs(h, w, t, suppress_ids=[100]),
                lambda: cs.lm_head_logprobs(h, w, t, ws=torch.zeros(256, dtype=torch.uint8, device="cuda")),
                lambda: cs.lm_head_logprobs(h[:, :60].contiguous(), w[:, :60].contiguous(), t),
                lambda: cs.lm_head_logprobs_backward(h, w, t, f, f, f, out=(h, None)),
                lambda: cs.lm_head_logprobs_backward(h, w, t, f, f, f, out=(None, w))):
        with pytest.raises(cs.DllmError):
            bad()


def test_side_stream_and_graph(cs):
    h, w, t, sup = inputs(300, 5000, 192, 17, 0.5, 1)
    g = torch.randn(300, device="cuda")
    want = [*cs.lm_head_logprobs(h, w, t, suppress_ids=sup)]
    want += cs.lm_head_logprobs_backward(h, w, t, want[2], want[1], g, suppress_ids=sup)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [*cs.lm_head_logprobs(h, w, t, suppress_ids=sup, stream=side)]
    got += cs.lm_head_logprobs_backward(h, w, t, got[2], got[1], g, suppress_ids=sup, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = [*cs.lm_head_logprobs(h, w, t, suppress_ids=sup)]
        cap += cs.lm_head_logprobs_backward(h, w, t, cap[2], cap[1], g, suppress_ids=sup)
    t.copy_(t.roll(7))                                   # other rows are scored in the replay
    h.copy_(h.roll(3, 0))
    graph.replay()
    torch.cuda.synchronize()
    want = [*cs.lm_head_logprobs(h, w, t, suppress_ids=sup)]
    want += cs.lm_head_logprobs_backward(h, w, t, want[2], want[1], g, suppress_ids=sup)
    assert all(torch.equal(a, b) for a, b in zip(cap, want))
