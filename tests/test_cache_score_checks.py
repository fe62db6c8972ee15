"""The cache and scoring entry points refuse bad arguments on the host, before
anything is launched (no device is needed), and the 64-bit references of the
GPU tests agree with independent statements.  CPU only."""
import ctypes as C

import numpy as np
import pytest
import torch

from cache_reference import VALUES, Pool, encode, fit_scale, random_pool
from test_binding_checks import cs

FAKE = 1 << 20          # never dereferenced: every call fails its checks
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def cache(**kw):
    from commit_step_gb300.cache import _CacheStruct

    f = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=8, page_size=64, heads=4, head_dim=128)
    f.update(kw)
    return C.byref(_CacheStruct(*[f[n] for n, _ in _CacheStruct._fields_]))


I3 = C.c_int64 * 3
GOOD = I3(1024, 512, 128)
BAD_CACHES = [(dict(k=None), INVALID), (dict(v_scale=None), INVALID), (dict(k=FAKE + 8), INVALID),
              (dict(num_pages=0), INVALID), (dict(heads=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
              (dict(page_size=24), UNSUPPORTED), (dict(page_size=0), UNSUPPORTED), (dict(num_pages=1 << 40), INVALID),
              (dict(heads=1 << 20), UNSUPPORTED)]


def append(c, k=FAKE, v=FAKE, ks=GOOD, vs=GOOD, B=2, L=4, table=FAKE, width=4, start=FAKE, count=None):
    return cs.lib_handle().dllm_cache_append(c, k, v, ks, vs, B, L, table, width, start, count, None)


def attend(c, q=FAKE, s=GOOD, B=2, L=4, Hq=8, table=FAKE, width=4, lens=FAKE, mask=None, ms=0, scale=1.0, out=FAKE,
           lse=FAKE, w=None, decay=1.0, ws=FAKE, wsb=1 << 40):
    return cs.lib_handle().dllm_cache_attention(c, q, s, B, L, Hq, table, width, lens, mask, ms, scale, out, lse, w,
                                                decay, ws, wsb, None)


def evict(c, table=FAKE, width=4, lens=FAKE, B=2, w=FAKE, budget=100, first=4, last=8, dst=FAKE, dw=2, keep=FAKE,
          lo=FAKE, wo=FAKE + 4096):
    return cs.lib_handle().dllm_cache_evict(c, table, width, lens, B, w, budget, first, last, dst, dw, keep, lo, wo,
                                            None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(kw, status):
    for call in (append, attend, evict):
        assert call(cache(**kw)) == status
    assert append(None) == INVALID and attend(None) == INVALID and evict(None) == INVALID


def test_append_refusals():
    for kw in (dict(k=None), dict(start=None), dict(table=None), dict(B=-1), dict(L=-1), dict(width=0), dict(ks=None),
               dict(ks=I3(-8, 8, 8)), dict(ks=I3(1 << 62, 8, 8)), dict(start=FAKE + 2)):
        assert append(cache(), **kw) == INVALID, kw
    for kw in (dict(k=FAKE + 2), dict(vs=I3(1024, 512, 100)), dict(width=1 << 26), dict(B=40000), dict(B=1 << 50)):
        assert append(cache(), **kw) == UNSUPPORTED, kw
    assert append(cache(), B=0) == 0 and append(cache(), L=0) == 0


def test_attention_refusals():
    inf = float("inf")
    for kw in (dict(q=None), dict(lens=None), dict(out=None), dict(lse=None), dict(Hq=6), dict(Hq=0), dict(L=-1),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=inf), dict(scale=float("nan")), dict(decay=-0.5),
               dict(decay=1.5), dict(decay=float("nan")), dict(mask=FAKE, ms=255), dict(s=None), dict(w=FAKE + 1),
               dict(L=1 << 61), dict(ws=FAKE + 8)):
        assert attend(cache(), **kw) == INVALID, kw
    for kw in (dict(q=FAKE + 2), dict(out=FAKE + 2), dict(s=I3(1024, 512, 4))):
        assert attend(cache(), **kw) == UNSUPPORTED, kw
    assert attend(cache(), ws=None) == WORKSPACE and attend(cache(), wsb=0) == WORKSPACE
    assert attend(cache(), B=0) == 0 and attend(cache(), L=0) == 0


def test_evict_refusals():
    for kw in (dict(lens=None), dict(w=None), dict(keep=None), dict(lo=None), dict(wo=None), dict(dst=None),
               dict(budget=0), dict(first=-1), dict(last=-1), dict(first=60, last=60), dict(budget=129), dict(dw=0),
               dict(wo=FAKE), dict(keep=FAKE + 1)):
        assert evict(cache(), **kw) == INVALID, kw
    assert evict(cache(), B=40000) == UNSUPPORTED
    assert evict(cache(), B=0) == 0


def score(dt=1, T=4, V=100, stride=100, z=FAKE, t=FAKE, sup=(), top=0, lp=FAKE, ent=FAKE, lse=FAKE, ids=FAKE,
          tlp=FAKE):
    arr = (C.c_int32 * max(1, len(sup)))(*sup)
    return cs.lib_handle().dllm_token_logprobs(z, dt, T, V, stride, t, arr, len(sup), top, lp, ent, lse, ids, tlp, None)


def grad(dt=1, T=4, V=100, stride=100, z=FAKE, t=FAKE, sup=(), top=0, lse=FAKE, ent=FAKE, g=FAKE, ge=None, ids=FAKE,
         gt=FAKE, out=FAKE, os=100):
    arr = (C.c_int32 * max(1, len(sup)))(*sup)
    return cs.lib_handle().dllm_token_logprobs_backward(z, dt, T, V, stride, t, arr, len(sup), lse, ent, g, ge, top,
                                                        ids, gt, out, os, None)


def test_score_refusals():
    for call in (score, grad):
        for kw in (dict(dt=2), dict(T=-1), dict(V=0), dict(stride=99), dict(z=None), dict(t=None), dict(top=-1),
                   dict(sup=(100,)), dict(sup=(-1,)), dict(V=2, stride=2, sup=(0, 1)), dict(V=20, stride=20, top=21),
                   dict(V=20, sup=(3, 3), top=20), dict(lse=None), dict(T=1 << 61), dict(z=FAKE + 1),
                   dict(top=3, ids=None), dict(V=1 << 31, stride=1 << 31)):
            assert call(**kw) == INVALID, (call, kw)
        for kw in (dict(top=33), dict(sup=tuple(range(65)))):
            assert call(**kw) == UNSUPPORTED, (call, kw)
        assert call(T=0) == 0
    assert score(lp=None) == INVALID and grad(out=None) == INVALID and grad(os=99) == INVALID
    assert grad(top=2, gt=None) == INVALID and grad(ge=FAKE + 2) == INVALID


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    z = torch.zeros((2, 8))
    with pytest.raises(ValueError):
        cs.token_logprobs(z, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        cs.KVCache(4, 16, 1, 64, device="cpu")
    from commit_step_gb300.cache import _strided
    from commit_step_gb300.score import _rows

    t = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    assert list(_strided(t, "q", (2, 3, 4, 64), t.device)) == [768, 256, 64]
    assert list(_strided(t[:1, :, :1], "q", (1, 3, 1, 64), t.device)) == [0, 256, 0]
    for bad in (t.float(), t[0], t.transpose(2, 3)):
        with pytest.raises((TypeError, ValueError)):
            _strided(bad, "q", tuple(t.shape), t.device)
    assert _rows(torch.zeros((3, 4, 5)), "logits") == (12, 5, 5)
    assert _rows(torch.zeros((3, 9))[:, 2:7], "logits") == (3, 5, 9)
    for bad in (torch.zeros(5), torch.zeros((5, 3)).t(), torch.zeros((3, 4, 5))[:, :2], [1]):
        with pytest.raises(ValueError):
            _rows(bad, "logits")


# ------------------------------------------------------- the references
def test_reference_codes_are_torch_codes():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * np.exp2(rng.uniform(-12, 9, 20000)), VALUES[~np.isnan(VALUES)],
                        (VALUES[:126] + VALUES[1:127]) / 2])
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(encode(x.astype(np.float32)), want)
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(every), np.isnan(VALUES)) and np.nanmax(np.abs(every - VALUES)) == 0


def test_reference_scale():
    assert fit_scale(np.array([448.0])) == 1.0 and fit_scale(np.array([448.1])) == 2.0
    assert fit_scale(np.array([224.0])) == 0.5 and fit_scale(np.array([0.0, np.inf])) == 2.0 ** -100


def test_reference_attention_is_softmax():
    rng = np.random.default_rng(1)
    arrays = random_pool(rng, 6, 2, 16, 64)
    pool = Pool(*arrays)
    table = np.array([[4, 1, -1], [0, 5, 2]], dtype=np.int32)
    q = rng.standard_normal((2, 3, 4, 64))
    out, lse, w, _, _ = pool.attend(q, table, np.array([40, 20]), 0.125)
    k = torch.from_numpy(VALUES[arrays[0]] * arrays[2][:, :, None, None])
    v = torch.from_numpy(VALUES[arrays[1]] * arrays[3][:, :, None, None])
    for b, pages, n in ((0, [4, 1], 32), (1, [0, 5], 20)):
        kk = torch.cat([k[p] for p in pages], 1)[:, :n].repeat_interleave(2, 0)
        vv = torch.cat([v[p] for p in pages], 1)[:, :n].repeat_interleave(2, 0)
        x = torch.einsum("lhd,hnd->hln", torch.from_numpy(q[b]), kk) * 0.125
        p = torch.softmax(x, -1)
        assert np.allclose(out[b], torch.einsum("hln,hnd->lhd", p, vv).numpy(), rtol=1e-12, atol=1e-14)
        assert np.allclose(lse[b], torch.logsumexp(x, -1).T.numpy())
        assert np.allclose(w[b, :, :n], p.sum(1).view(2, 2, n).sum(1).numpy())
