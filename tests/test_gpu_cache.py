"""The paged 8-bit cache on the GPU against plain 64-bit implementations.

Tolerances of the attention (derived, not fitted).  A query's scores: fp32
sums of head_dim products, and a query whose elements below 2^-9 of its
largest are rounded at 2^-18 of that, are off by at most e = 2^-16 a with a =
scale max|q| sum|k| (twice 2^-17, one for each cause).  lse then is off by e
plus the rounding of its parts, 2^-19 (1 + |lse|); a probability by the factor
exp(2 e); the output by its own rounding to bf16 (2^-8 of the value) and by
the probabilities' rounding to no fewer than 11 bits (2^-11) and the scores'
error, each of sum p |v|.  A token's weight is a sum of probabilities.
Codes, scales, kept positions and lengths are compared exactly.
"""
import math
import threading

import numpy as np
import pytest
import torch

from cache_reference import Pool, random_pool, same_values

pytestmark = pytest.mark.gpu


def device_cache(cs, arrays):
    k, v, ks, vs = arrays
    return cs.KVCache.from_tensors(*[torch.from_numpy(np.array(a)).cuda() for a in (k, v, ks, vs)])


def assert_pool(cache, pool, pages=None):
    for name in ("k", "v"):
        got = getattr(cache, name).view(torch.uint8).cpu().numpy()
        scale = getattr(cache, name + "_scale").cpu().numpy().astype(np.float64)
        sel = slice(None) if pages is None else pages
        assert np.array_equal(scale[sel], pool.scale[name][sel]), name
        assert same_values(got[sel], pool.codes[name][sel]), name


def tables(rng, pages, B, width):
    return rng.permutation(pages)[:B * width].reshape(B, width).astype(np.int32)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("ps,dim,H,L", [(16, 64, 1, 1), (16, 128, 3, 33), (64, 128, 2, 130), (128, 64, 2, 300),
                                        (32, 64, 1, 31), (128, 128, 1, 129)])
def test_append(cs, ps, dim, H, L):
    rng = np.random.default_rng(ps + L)
    B = 5
    width = (L + 3 * ps) // ps + 2
    arrays = random_pool(rng, B * width + 2, H, ps, dim)
    cache, pool = device_cache(cs, arrays), Pool(*arrays)
    table = tables(rng, B * width + 2, B, width)
    start = np.array([0, 1, ps - 1, ps, 2 * ps + 3], dtype=np.int32)
    x = torch.from_numpy(rng.standard_normal((B, L, 2, H, dim))).to(torch.bfloat16)
    x[1] *= 64                       # scales grow past the old ones
    x[2] *= 2.0 ** -20               # and stay below them
    x[3, :, :, 0, : dim // 2] = 0
    xd = x.cuda()
    cs.cache_append(cache, xd[:, :, 0], xd[:, :, 1], dev(table), dev(start))
    xn = x.double().numpy()
    pool.append(xn[:, :, 0], xn[:, :, 1], table, start)
    assert_pool(cache, pool)


def test_append_counts_holes_and_edges(cs):
    rng = np.random.default_rng(5)
    ps, dim, H, L, B = 16, 128, 2, 40, 6
    width = 4
    arrays = random_pool(rng, B * width + 1, H, ps, dim)
    cache, pool = device_cache(cs, arrays), Pool(*arrays)
    table = tables(rng, B * width + 1, B, width)
    table[1, 1] = -1                 # entries that name no page
    table[2, 0] = B * width + 1
    table[3, 2] = 2 ** 31 - 1
    start = np.array([30, 5, 0, 20, -7, 2 ** 31 - 20], dtype=np.int32)   # past the table's end, below 0, far off
    count = np.array([40, 33, 0, 500, 20, -3], dtype=np.int32)
    x = torch.from_numpy(rng.standard_normal((B, L, H, dim))).to(torch.bfloat16)
    y = torch.from_numpy(rng.standard_normal((B, L, H, dim))).to(torch.bfloat16)
    x[0, 3, 0, 5], x[0, 4, 1, 7] = math.inf, -math.inf
    y[1, 2, 0, 0] = math.nan
    cs.cache_append(cache, x.cuda(), y.cuda(), dev(table), dev(start), dev(count))
    pool.append(x.double().numpy(), y.double().numpy(), table, start, count)
    assert_pool(cache, pool)


def test_append_extremes_of_the_scale(cs):
    """All-zero pages, subnormal and the largest bf16 values, magnitudes next to 448 2^e."""
    ps, dim = 16, 64
    rng = np.random.default_rng(2)
    arrays = random_pool(rng, 8, 1, ps, dim)
    cache, pool = device_cache(cs, arrays), Pool(*arrays)
    table = np.arange(8, dtype=np.int32)[None]
    x = torch.zeros((1, 8 * ps, 1, dim), dtype=torch.bfloat16)
    x[0, ps] = 2.0 ** -133
    x[0, 2 * ps] = 3.3895e38
    x[0, 3 * ps, 0, 0] = 448.0
    x[0, 4 * ps, 0, 0] = 450.0
    x[0, 5 * ps, 0, 0] = 446.0
    x[0, 6 * ps, 0, 0] = math.inf
    x[0, 7 * ps:] = math.nan
    cs.cache_append(cache, x.cuda(), (-x).cuda(), dev(table), dev(np.zeros(1, dtype=np.int32)))
    pool.append(x.double().numpy(), (-x).double().numpy(), table, np.zeros(1, dtype=np.int32))
    assert_pool(cache, pool)


def test_append_in_steps_equals_one_append_when_the_first_is_largest(cs):
    """Tokens added one at a time behind a page's largest token leave what one call leaves."""
    rng = np.random.default_rng(9)
    ps, dim, H, L = 64, 128, 2, 50
    x = torch.from_numpy(rng.standard_normal((1, L, H, dim))).to(torch.bfloat16).cuda()
    x[:, 0] = 8.0
    table = dev(np.zeros((1, 1), dtype=np.int32))
    one, steps = cs.KVCache(1, ps, H, dim), cs.KVCache(1, ps, H, dim)
    cs.cache_append(one, x, x, table, dev(np.zeros(1, dtype=np.int32)))
    for j in range(L):
        cs.cache_append(steps, x[:, j:j + 1], x[:, j:j + 1], table, dev(np.full(1, j, dtype=np.int32)))
    for a, b in ((one.k, steps.k), (one.v, steps.v)):
        assert torch.equal(a.view(torch.uint8)[:, :, :L], b.view(torch.uint8)[:, :, :L])
    assert torch.equal(one.k_scale, steps.k_scale) and torch.equal(one.v_scale, steps.v_scale)


# --------------------------------------------------------------- attention
def check_attention(cs, arrays, q, table, lens, scale=None, mask=None, weights=True, decay=0.5, stream=None):
    cache, pool = device_cache(cs, arrays), Pool(*arrays)
    B, L, Hq, D = q.shape
    s = 1.0 / math.sqrt(D) if scale is None else scale
    want, lse_want, w_want, spread, size = pool.attend(q.double().cpu().numpy(), table, lens, s, mask)
    cap = table.shape[1] * pool.ps
    w0 = np.random.default_rng(1).random((B, pool.heads, cap)).astype(np.float32)
    w = dev(w0) if weights else None
    out, lse = cs.cache_attention(q, cache, dev(table), dev(lens), scale=scale,
                                  key_mask=None if mask is None else dev(mask), weights=w, decay=decay, stream=stream)
    torch.cuda.synchronize()
    got, lse_got = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isnan(lse_got), np.isnan(lse_want))
    empty = np.isneginf(lse_want)
    assert np.array_equal(np.isneginf(lse_got), empty) and not got[empty].any()
    e = 2.0 ** -16 * size
    with np.errstate(invalid="ignore"):
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + np.expm1(2 * e)[..., None]) * spread + 1e-37
        bad = np.abs(got - want) > tol
        assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])
        bad = np.abs(lse_got - lse_want) > e + 2.0 ** -19 * (1 + np.abs(lse_want))
        bad &= np.isfinite(lse_want)
        assert not bad.any(), (np.argwhere(bad)[:3], lse_got[bad][:3], lse_want[bad][:3])
    if weights:
        total = (0.0 if decay == 0 else decay) * w0.astype(np.float64) + w_want
        fine = np.isfinite(lse_want)
        rel = np.expm1(2 * (e[fine].max() + 2.0 ** -19 * (1 + np.abs(lse_want[fine]).max()))) if fine.any() else 0.0
        err = np.abs(w.double().cpu().numpy() - total)
        assert (err <= rel * w_want + 2.0 ** -20 * total + 1e-37).all(), err.max()
    return out, lse


def queries(rng, B, L, Hq, D):
    return torch.from_numpy(rng.standard_normal((B, L, Hq, D))).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("ps,H,G,L", [(16, 1, 1, 1), (64, 2, 7, 1), (32, 2, 4, 5), (16, 3, 1, 32), (64, 1, 8, 16),
                                      (128, 2, 7, 32), (64, 1, 1, 130), (32, 1, 3, 17), (128, 1, 12, 33)])
def test_attention(cs, dim, ps, H, G, L):
    rng = np.random.default_rng(dim + ps + H * G + L)
    lens = np.array([0, 1, ps - 1, ps + 1, 127, 128, 129, 300], dtype=np.int32)
    B, width = len(lens), -(-300 // ps)
    arrays = random_pool(rng, B * width + 3, H, ps, dim)
    check_attention(cs, arrays, queries(rng, B, L, H * G, dim), tables(rng, B * width + 3, B, width), lens)


@pytest.mark.parametrize("L,G", [(1, 1), (1, 8), (32, 4)])
def test_attention_long_and_split(cs, L, G):
    """Few rows over long sequences (work split along the keys), very different lengths."""
    rng = np.random.default_rng(L + G)
    ps, H, dim = 64, 2, 128
    lens = np.array([5000, 17, 2049], dtype=np.int32)
    width = -(-5000 // ps)
    arrays = random_pool(rng, 3 * width, H, ps, dim)
    check_attention(cs, arrays, queries(rng, 3, L, H * G, dim), tables(rng, 3 * width, 3, width), lens, decay=0.0)


def test_attention_many_sequences(cs):
    """More sequences than SMs, most of them short or empty."""
    rng = np.random.default_rng(77)
    ps, H, dim, B, width = 16, 1, 64, 400, 6
    lens = rng.integers(0, width * ps + 1, B).astype(np.int32)
    lens[::5] = 0
    arrays = random_pool(rng, B * width, H, ps, dim)
    check_attention(cs, arrays, queries(rng, B, 2, 2, dim), tables(rng, B * width, B, width), lens)


@pytest.mark.parametrize("dim,L", [(64, 12), (128, 12), (64, 25), (128, 25)])
def test_attention_many_items_a_cta(cs, dim, L):
    """48 and 100 rows of ragged sequences, several to a CTA, cut anywhere."""
    rng = np.random.default_rng(dim + L)
    ps, H, G, B, width = 32, 2, 4, 110, 16
    lens = rng.integers(0, width * ps + 1, B).astype(np.int32)
    arrays = random_pool(rng, B * width, H, ps, dim)
    mask = (rng.random((B, width * ps)) < 0.9).astype(np.uint8)
    mask[::7] = 0
    check_attention(cs, arrays, queries(rng, B, L, H * G, dim), tables(rng, B * width, B, width), lens, mask=mask)


@pytest.mark.parametrize("L", [1, 40])
def test_attention_mask_holes_and_garbage(cs, L):
    """Masked tokens, slots past the length and pages that do not exist hold NaN
    codes and NaN scales; masks leave some sequences nothing."""
    rng = np.random.default_rng(11 + L)
    ps, H, G, dim, B, width = 16, 2, 4, 128, 6, 20
    arrays = random_pool(rng, B * width, H, ps, dim)
    table = tables(rng, B * width, B, width)
    lens = np.array([200, 320, 33, 150, 1, 2 ** 31 - 1], dtype=np.int32)   # the last is clamped to the table
    mask = (rng.random((B, width * ps)) < 0.7).astype(np.uint8) * 3
    mask[2] = 0
    mask[4, 0] = 0
    mask[1, :256] = 0                                                       # two whole tiles without a visible key
    table[3, 2], table[3, 5], table[0, 0] = -1, B * width, -(2 ** 31)
    for name in (0, 1):
        for b in range(B):
            for j in range(width * ps):
                p = table[b, j // ps]
                if 0 <= p < B * width and (j >= lens[b] or not mask[b, j]):
                    arrays[name][p, :, j % ps] = 0x7F if j % 2 else 0xFF
    arrays[2][table[1, 0]], arrays[3][table[1, 1]] = np.nan, np.nan         # wholly masked pages
    check_attention(cs, arrays, queries(rng, B, L, H * G, dim), table, lens, mask=mask)


@pytest.mark.parametrize("L", [4, 20])
def test_attention_very_negative_scores_behind_masked_tiles(cs, L):
    """Tiles without a visible key, then scores far below zero: a first reference
    near -180 meets an accumulator that holds products of nothing."""
    rng = np.random.default_rng(5 + L)
    ps, H, G, dim, B, width = 16, 2, 4, 128, 64, 32
    arrays = list(random_pool(rng, B * width, H, ps, dim, spread=1))
    arrays[0] = arrays[0] & 0x7F                                            # keys above zero, queries below
    q = -(queries(rng, B, L, H * G, dim).abs() + 12)
    mask = np.ones((B, width * ps), dtype=np.uint8)
    mask[:, :256] = 0
    lens = np.full(B, width * ps, dtype=np.int32)
    check_attention(cs, arrays, q, tables(rng, B * width, B, width), lens, mask=mask)


def test_attention_nan_and_inf_queries_stay_in_their_row(cs):
    rng = np.random.default_rng(3)
    ps, H, G, dim, B, width = 64, 1, 4, 128, 2, 4
    arrays = random_pool(rng, B * width, H, ps, dim)
    q = queries(rng, B, 8, H * G, dim)
    q[0, 3, 1, 7] = math.nan
    q[1, 2, 0, 0] = math.inf
    q[1, 5, 3, 9] = -math.inf
    q[1, 6, 2] = 0
    q[0, 0, 0] = 1e-30
    check_attention(cs, arrays, q, tables(rng, B * width, B, width), np.array([200, 256], dtype=np.int32))


def test_attention_sharp_and_growing_scores(cs):
    """Scores that grow along the sequence (the maximum moves in every tile), one
    key that takes almost all the mass, and large scales."""
    rng = np.random.default_rng(4)
    ps, H, dim, width = 32, 2, 128, 20
    n = width * ps
    arrays = [np.array(a) for a in random_pool(rng, width, H, ps, dim)]
    table = np.arange(width, dtype=np.int32)[None]
    arrays[2][:] = (2.0 ** (np.arange(width) // 3 - 8))[:, None]
    arrays[3][:] = (2.0 ** (-(np.arange(width) % 7)))[:, None]
    q = queries(rng, 1, 9, H * 2, dim)
    check_attention(cs, arrays, q, table, np.array([n], dtype=np.int32))
    check_attention(cs, arrays, q, table, np.array([n], dtype=np.int32), scale=2.0)
    arrays[0][0, 0, 3] = 0x7E                                               # one key along the first query
    check_attention(cs, arrays, q.abs(), table, np.array([n - 5], dtype=np.int32))


def test_attention_general_scales(cs):
    """Scales that are not powers of two, and span many."""
    rng = np.random.default_rng(8)
    ps, H, dim, B, width = 16, 2, 64, 2, 16
    k, v, _, _ = random_pool(rng, B * width, H, ps, dim)
    ks = (0.001 + 0.01 * rng.random((B * width, H))).astype(np.float32)
    vs = np.exp2(rng.uniform(-12, 6, (B * width, H))).astype(np.float32)
    check_attention(cs, (k, v, ks, vs), queries(rng, B, 6, H * 2, dim), tables(rng, B * width, B, width),
                    np.array([250, 100], dtype=np.int32))


def page_that_draws(rng, heads, G, L, ps, dim, width, drawn):
    """(q, arrays, table, lens) of one sequence whose queries put nearly all mass on the
    pages `drawn`: keys along the queries' common signs there, against them elsewhere."""
    sign = np.where(rng.random((heads, dim)) < 0.5, -1.0, 1.0)
    q = sign.repeat(G, 0)[None, None] * (0.5 + rng.random((1, L, heads * G, dim)))
    k, v, ks, vs = [np.array(a) for a in random_pool(rng, width, heads, ps, dim)]
    side = np.where(np.isin(np.arange(width), drawn), 1.0, -1.0)[:, None, None, None] * sign[None, :, None]
    x = side * (1.0 + rng.random((width, heads, ps, dim)))
    k[:] = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    ks[:] = 1.0
    table = np.arange(width, dtype=np.int32)[None]
    return torch.from_numpy(q).to(torch.bfloat16).cuda(), [k, v, ks, vs], table, np.array([width * ps - 3], np.int32)


@pytest.mark.parametrize("dim,L,G", [(64, 1, 1), (128, 8, 4), (128, 16, 4), (64, 25, 4), (128, 40, 4)])
@pytest.mark.parametrize("drawn", [[0], [13], [5, 6]])
@pytest.mark.parametrize("ratio", [2.0 ** 12, 2.0 ** 18, 2.0 ** 26, 1.7 * 2.0 ** 45])
def test_attention_of_a_page_of_small_values(cs, dim, L, G, drawn, ratio):
    """All mass lies on pages whose value scale is `ratio` times smaller than that of
    pages before, behind and between them, which the queries see and do not attend
    to: the result is as exact as without those.  (Mass elsewhere: about e^-67.)"""
    rng = np.random.default_rng(dim + L + drawn[0])
    q, arrays, table, lens = page_that_draws(rng, 2, G, L, 32, dim, 14, drawn)
    arrays[3][:] = 2.0 ** -8
    arrays[3][drawn] = 2.0 ** -8 / ratio
    check_attention(cs, arrays, q, table, lens, scale=0.5 * 45 / dim)


@pytest.mark.parametrize("L,G", [(1, 1), (8, 4), (25, 4)])
@pytest.mark.parametrize("small", [2.0 ** -100, 2.0 ** -70, 2.0 ** -45, 2.0 ** -30])
def test_attention_drawn_by_values_of_nothing(cs, L, G, small):
    """Pages of zero values (scale 2^-100), and of next to none, that draw a part of the
    mass, most of it or nearly all: it counts in the sums."""
    rng = np.random.default_rng(L + G)
    ps, dim, width = 16, 128, 30
    for scale in (2.0 ** -9, 2.0 ** -6, 2.0 ** -4):
        q, arrays, table, lens = page_that_draws(rng, 2, G, L, ps, dim, width, [3, 4, 20, 29])
        arrays[3][:] = 2.0 ** 5
        arrays[3][[3, 4, 20, 29]] = small
        if small == 2.0 ** -100:
            arrays[1][[3, 4, 20, 29]] = 0
        check_attention(cs, arrays, q, table, lens, scale=scale)


@pytest.mark.parametrize("L,G", [(1, 1), (8, 4), (25, 4)])
def test_attention_of_pages_without_values(cs, L, G):
    """What appends of zeros, of infinities and of NaN leave: the least scale, with codes
    of 0, 448 and NaN.  Such a page draws its share; NaN stays, all else counts as 0."""
    rng = np.random.default_rng(L)
    ps, dim, H, width = 16, 64, 2, 20
    arrays = [np.array(a) for a in random_pool(rng, width, H, ps, dim)]
    least = [0, 7, 8, 9, 15]
    arrays[3][least] = 2.0 ** -100
    arrays[1][least] = 0
    arrays[1][8, :, 3, 5:9] = 0x7E
    arrays[1][9, 1, 4, 17], arrays[1][15, 0, 0, 63] = 0x7F, 0xFF
    q = queries(rng, 1, L, H * G, dim)
    table = np.arange(width, dtype=np.int32)[None]
    check_attention(cs, arrays, q, table, np.array([width * ps - 5], np.int32))
    check_attention(cs, arrays, q, table[:, :1].copy(), np.array([ps], np.int32))


@pytest.mark.parametrize("scale_v", [2.0 ** -99, 2.0 ** -60, 1.3 * 2.0 ** -40, 2.0 ** 40, 1.9 * 2.0 ** 90, 2.0 ** 117])
@pytest.mark.parametrize("L,G", [(1, 1), (8, 4), (25, 4)])
def test_attention_of_values_of_any_size(cs, L, G, scale_v):
    """One scale on all pages, over the range that appends make."""
    rng = np.random.default_rng(L)
    ps, dim, H, width = 16, 64, 2, 30
    arrays = list(random_pool(rng, width, H, ps, dim))
    arrays[3] = np.full_like(arrays[3], scale_v)
    q = queries(rng, 1, L, H * G, dim)
    check_attention(cs, arrays, q, np.arange(width, dtype=np.int32)[None], np.array([width * ps - 5], np.int32))


def test_attention_strided_queries_and_stream(cs):
    rng = np.random.default_rng(6)
    ps, H, G, dim, B, width, L = 64, 2, 2, 128, 3, 4, 12
    arrays = random_pool(rng, B * width, H, ps, dim)
    packed = torch.from_numpy(rng.standard_normal((B, L, H * G + 3, dim))).to(torch.bfloat16).cuda()
    q = packed[:, :, 1:1 + H * G]
    table, lens = tables(rng, B * width, B, width), np.array([7, 129, 256], dtype=np.int32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check_attention(cs, arrays, q, table, lens, stream=side)
    t = packed.transpose(0, 1)[:, :, :H * G]                                # (L, B, heads): other outer order
    check_attention(cs, arrays, t.transpose(0, 1), table, lens)


def test_attention_repeats_bit_for_bit(cs):
    """No result depends on the order in which CTAs run."""
    rng = np.random.default_rng(21)
    ps, H, dim, B, width = 64, 4, 128, 3, 40
    cache = device_cache(cs, random_pool(rng, B * width, H, ps, dim))
    table, lens = dev(tables(rng, B * width, B, width)), dev(np.array([2500, 700, 64], dtype=np.int32))
    q = queries(rng, B, 20, H * 3, dim)
    first = None
    for _ in range(5):
        w = torch.zeros((B, H, width * ps), device="cuda")
        out, lse = cs.cache_attention(q, cache, table, lens, weights=w)
        got = [t.clone() for t in (out.view(torch.int16), lse, w)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.parametrize("L", [1, 20, 70])
def test_attention_over_its_own_queries(cs, L):
    """The output in the queries' place, and next to them."""
    rng = np.random.default_rng(L)
    ps, H, dim, B, width = 16, 2, 128, 9, 40
    cache = device_cache(cs, random_pool(rng, B * width, H, ps, dim))
    table, lens = dev(tables(rng, B * width, B, width)), dev(rng.integers(0, width * ps + 1, B).astype(np.int32))
    q = queries(rng, B, L, H * 3, dim)
    want, lse = cs.cache_attention(q, cache, table, lens)
    both = torch.zeros((2, *q.shape), dtype=torch.bfloat16, device="cuda")
    for at in (0, 1):
        both[at] = q
        cs.cache_attention(both[at], cache, table, lens, out=(both[1 - at], torch.empty_like(lse)),
                           weights=torch.zeros((B, H, width * ps), device="cuda"))
        assert torch.equal(both[1 - at].view(torch.int16), want.view(torch.int16))
        assert torch.equal(both[at].view(torch.int16), q.view(torch.int16))
    out, _ = cs.cache_attention(q, cache, table, lens, out=(q, torch.empty_like(lse)))
    assert out is q and torch.equal(q.view(torch.int16), want.view(torch.int16))


def test_attention_in_a_graph(cs):
    rng = np.random.default_rng(22)
    ps, H, dim, B, width = 64, 2, 128, 2, 6
    arrays = random_pool(rng, B * width, H, ps, dim)
    cache = device_cache(cs, arrays)
    table, lens = dev(tables(rng, B * width, B, width)), dev(np.array([300, 100], dtype=np.int32))
    q = queries(rng, B, 16, H * 2, dim)
    want = [t.clone() for t in cs.cache_attention(q, cache, table, lens)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(t) for t in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cs.cache_attention(q, cache, table, lens, out=out, ws=ws)
    for t in out:
        t.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(out[1], want[1])


def test_attention_in_a_graph_on_a_stream_that_goes_on(cs):
    """Warmed up, captured and followed by larger calls on one stream, with no
    workspace given: replays touch no memory that was given to someone else."""
    rng = np.random.default_rng(23)
    ps, H, dim, B, width = 64, 2, 128, 2, 40
    cache = device_cache(cs, random_pool(rng, B * width, H, ps, dim))
    table, lens = dev(tables(rng, B * width, B, width)), dev(np.array([2500, 900], dtype=np.int32))
    q, more = queries(rng, B, 4, H * 2, dim), queries(rng, B, 60, H * 2, dim)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in cs.cache_attention(q, cache, table, lens)]
        want_more = [t.clone() for t in cs.cache_attention(more, cache, table, lens)]
        cs.cache_attention(q, cache, table, lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = cs.cache_attention(q, cache, table, lens)
    with torch.cuda.stream(side):
        got_more = cs.cache_attention(more, cache, table, lens)
        side.synchronize()
        others = [torch.full((n << 10,), 5, dtype=torch.uint8, device="cuda") for n in (64, 256, 1024, 4096, 16384, 32768)]
        graph.replay()
        side.synchronize()
        assert all(bool((t == 5).all()) for t in others)
    assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])
    assert torch.equal(got_more[0].view(torch.int16), want_more[0].view(torch.int16))
    assert torch.equal(got_more[1], want_more[1])


def test_attention_from_two_threads_on_one_stream(cs):
    """Calls whose items are cut among CTAs, enqueued between one another."""
    rng = np.random.default_rng(24)
    ps, H, dim, B, width = 64, 2, 128, 2, 40
    cache = device_cache(cs, random_pool(rng, B * width, H, ps, dim))
    table, lens = dev(tables(rng, B * width, B, width)), dev(np.array([2500, 900], dtype=np.int32))
    qs = [queries(rng, B, 4, H * 2, dim) for _ in range(2)]
    want = [cs.cache_attention(q, cache, table, lens)[0].view(torch.int16) for q in qs]
    same = [[], []]

    def work(i):
        for _ in range(300):
            same[i].append(torch.equal(cs.cache_attention(qs[i], cache, table, lens)[0].view(torch.int16), want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert [len(x) for x in same] == [300, 300] and all(map(all, same))


def test_pages_past_4_gib(cs):
    """A pool of more than 2^32 bytes: append, attention and eviction in its last pages."""
    rng = np.random.default_rng(12)
    ps, H, dim = 64, 8, 128
    pages = (1 << 32) // (ps * H * dim) + 16
    big = cs.KVCache(pages, ps, H, dim)
    small = cs.KVCache(16, ps, H, dim)
    x = torch.from_numpy(rng.standard_normal((1, 200, H, dim))).to(torch.bfloat16).cuda()
    q = queries(rng, 1, 3, 2 * H, dim)
    lens, start = dev(np.array([200], dtype=np.int32)), dev(np.zeros(1, dtype=np.int32))
    got = []
    for cache, base in ((small, 0), (big, pages - 16)):
        table = dev(np.arange(base, base + 4, dtype=np.int32)[None])
        dst = dev(np.arange(base + 4, base + 6, dtype=np.int32)[None])
        cs.cache_append(cache, x, x * 2, table, start)
        w = torch.zeros((1, H, 4 * ps), device="cuda")
        out, lse = cs.cache_attention(q, cache, table, lens, weights=w)
        keep, n, w2 = cs.cache_evict(cache, table, lens, w, 100, dst, keep_first=3, keep_last=10)
        out2, lse2 = cs.cache_attention(q, cache, dst, n)
        got.append([t.float() for t in (out, lse, w, keep, w2, out2, lse2)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_empty_calls(cs):
    cache = cs.KVCache(4, 16, 2, 64)
    none = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    out, lse = cs.cache_attention(torch.zeros((0, 4, 4, 64), dtype=torch.bfloat16, device="cuda"), cache, none, z)
    assert out.shape == (0, 4, 4, 64) and lse.shape == (0, 4, 4)
    table = torch.zeros((1, 3), dtype=torch.int32, device="cuda")
    n = torch.ones(1, dtype=torch.int32, device="cuda")
    kv = torch.zeros((1, 0, 2, 64), dtype=torch.bfloat16, device="cuda")
    cs.cache_append(cache, kv, kv, table, n)
    out, lse = cs.cache_attention(torch.zeros((1, 0, 4, 64), dtype=torch.bfloat16, device="cuda"), cache, table, n)
    assert out.numel() == 0


# ------------------------------------------------------------------- evict
@pytest.mark.parametrize("ps,dim,H,cap,budget,first,last", [
    (16, 64, 1, 48, 1, 0, 0), (16, 128, 2, 320, 100, 4, 16), (64, 128, 3, 1024, 512, 0, 64), (32, 64, 2, 5000, 999, 10, 0),
    (128, 128, 1, 640, 129, 65, 64), (16, 64, 2, 64, 64, 30, 34)])
def test_evict(cs, ps, dim, H, cap, budget, first, last):
    rng = np.random.default_rng(cap + budget)
    B, width, dst_width = 4, -(-cap // ps), -(-budget // ps) + 1
    cap = width * ps
    lens = np.array([cap, 0, min(budget, cap), min(cap, budget + 1)], dtype=np.int32)
    pages = B * (width + dst_width)
    arrays = random_pool(rng, pages, H, ps, dim, spread=5)
    order = rng.permutation(pages).astype(np.int32)
    table, dst = order[:B * width].reshape(B, width), order[B * width:].reshape(B, dst_width)
    w = np.round(rng.random((B, H, cap)) ** 6 * 40).astype(np.float32) / 8      # many ties
    w[0, 0, : cap // 2] = 0.25
    w[3, -1, ::3] = np.nan
    w[3, 0, 1::7], w[3, 0, 2::9] = np.inf, -np.inf
    w[0, -1, 5::11] = -0.0
    cache, pool = device_cache(cs, arrays), Pool(*arrays)
    keep, n, moved = cs.cache_evict(cache, dev(table), dev(lens), dev(w), budget, dev(dst), keep_first=first,
                                    keep_last=last)
    keep_w, n_w, moved_w = pool.evict(table, lens, w, budget, first, last, dst)
    assert np.array_equal(keep.cpu().numpy(), keep_w)
    assert np.array_equal(n.cpu().numpy(), n_w)
    assert np.array_equal(moved.cpu().numpy(), moved_w, equal_nan=True)
    assert_pool(cache, pool)


def test_evict_bad_pages_and_nan_codes(cs):
    rng = np.random.default_rng(31)
    ps, dim, H, B, width, dst_width, budget = 16, 64, 2, 2, 6, 3, 40
    pages = B * (width + dst_width)
    arrays = random_pool(rng, pages, H, ps, dim)
    order = rng.permutation(pages).astype(np.int32)
    table, dst = order[:B * width].reshape(B, width).copy(), order[B * width:].reshape(B, dst_width).copy()
    arrays[0][table[0, 1], :, 3] = 0x7F
    table[0, 2], table[1, 0], dst[1, 1] = -1, pages, 2 ** 31 - 1
    lens = np.array([90, 1000], dtype=np.int32)
    w = rng.random((B, H, width * ps)).astype(np.float32)
    cache, pool = device_cache(cs, arrays), Pool(*arrays)
    keep, n, moved = cs.cache_evict(cache, dev(table), dev(lens), dev(w), budget, dev(dst), keep_first=20)
    keep_w, n_w, moved_w = pool.evict(table, lens, w, budget, 20, 0, dst)
    assert np.array_equal(keep.cpu().numpy(), keep_w) and np.array_equal(n.cpu().numpy(), n_w)
    assert np.array_equal(moved.cpu().numpy(), moved_w)
    assert_pool(cache, pool)


def test_evict_updates_the_lengths_in_place(cs):
    """Every head selects by the lengths from before the call, however early another
    one's block is done."""
    rng = np.random.default_rng(41)
    ps, dim, H, B, width, budget = 16, 64, 32, 24, 20, 60
    dst_width = -(-budget // ps)
    pages = B * (width + dst_width)
    arrays = random_pool(rng, pages, H, ps, dim)
    order = rng.permutation(pages).astype(np.int32)
    table, dst = order[:B * width].reshape(B, width), order[B * width:].reshape(B, dst_width)
    lens = rng.integers(0, width * ps + 1, B).astype(np.int32)
    w = rng.random((B, H, width * ps)).astype(np.float32)
    pool = Pool(*arrays)
    keep_w, n_w, moved_w = pool.evict(table, lens, w, budget, 4, 8, dst)
    cache, n = device_cache(cs, arrays), dev(lens)
    out = (torch.empty((B, H, budget), dtype=torch.int32, device="cuda"), n, torch.empty_like(dev(w)))
    keep, n_out, moved = cs.cache_evict(cache, dev(table), n, dev(w), budget, dev(dst), keep_first=4, keep_last=8,
                                        out=out)
    assert n_out is n and np.array_equal(n.cpu().numpy(), n_w)
    assert np.array_equal(keep.cpu().numpy(), keep_w)
    assert np.array_equal(moved.cpu().numpy(), moved_w)
    assert_pool(cache, pool)


def test_evict_weights_next_to_the_moved_ones(cs):
    rng = np.random.default_rng(42)
    ps, dim, H, width, budget = 16, 64, 2, 5, 30
    arrays = random_pool(rng, 8, H, ps, dim)
    table, dst, lens = np.arange(5, dtype=np.int32)[None], np.array([[5, 6]], dtype=np.int32), np.array([77], dtype=np.int32)
    w = rng.random((1, H, width * ps)).astype(np.float32)
    for first in (0, 1):
        cache, pool = device_cache(cs, arrays), Pool(*arrays)
        both = torch.zeros((2, 1, H, width * ps), device="cuda")
        both[first] = dev(w)
        out = (torch.empty((1, H, budget), dtype=torch.int32, device="cuda"), dev(lens), both[1 - first])
        keep, n, moved = cs.cache_evict(cache, dev(table), dev(lens), both[first], budget, dev(dst), out=out)
        keep_w, n_w, moved_w = pool.evict(table, lens, w, budget, 0, 0, dst)
        assert np.array_equal(keep.cpu().numpy(), keep_w) and np.array_equal(n.cpu().numpy(), n_w)
        assert np.array_equal(moved.cpu().numpy(), moved_w) and np.array_equal(both[first].cpu().numpy(), w)
