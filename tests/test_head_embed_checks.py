"""The head's and the embedding's entry points refuse bad arguments on the host,
before anything is launched (no device is needed), and the 64-bit references of
the GPU tests agree with independent statements.  CPU only."""
import ctypes as C
import math

import pytest
import torch

from head_reference import embedding_grad, grads, scores
from test_binding_checks import cs

FAKE = 1 << 20          # never dereferenced: every call fails its checks
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def ids(sup):
    return (C.c_int32 * max(1, len(sup)))(*sup), len(sup)


def score(h=FAKE, T=4, d=64, hs=64, w=FAKE, V=100, wst=64, t=FAKE, sup=(), lp=FAKE, ent=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 50):
    return cs.lib_handle().dllm_lm_head_logprobs(h, T, d, hs, w, V, wst, t, *ids(sup), lp, ent, lse, ws, wsb, None)


def grad(h=FAKE, T=4, d=64, hs=64, w=FAKE, V=100, wst=64, t=FAKE, sup=(), lse=FAKE, ent=FAKE, g=FAKE, ge=None, gh=FAKE,
         ghs=64, gw=FAKE, dt=1, gws=64, acc=0, ws=FAKE, wsb=1 << 50):
    return cs.lib_handle().dllm_lm_head_logprobs_backward(h, T, d, hs, w, V, wst, t, *ids(sup), lse, ent, g, ge, gh, ghs,
                                                          gw, dt, gws, acc, ws, wsb, None)


def test_head_refusals():
    for call in (score, grad):
        for kw in (dict(h=None), dict(w=None), dict(t=None), dict(T=-1), dict(V=0), dict(V=1 << 31), dict(d=0), dict(hs=63),
                   dict(wst=63), dict(sup=(100,)), dict(sup=(-1,)), dict(V=2, sup=(0, 1)), dict(t=FAKE + 2), dict(lse=None),
                   dict(ent=None), dict(ent=FAKE + 1), dict(T=1 << 60, hs=1 << 20, d=64), dict(ws=FAKE + 8)):
            assert call(**kw) == INVALID, (call, kw)
        for kw in (dict(d=60), dict(h=FAKE + 2), dict(w=FAKE + 8), dict(hs=68), dict(wst=100), dict(sup=tuple(range(65))),
                   dict(T=(1 << 24) + 1), dict(d=1 << 21, hs=1 << 21, wst=1 << 21, gws=1 << 21, ghs=1 << 21)):
            if call is score:
                kw = {k: v for k, v in kw.items() if k not in ("gws", "ghs")}
            assert call(**kw) == UNSUPPORTED, (call, kw)
        assert call(ws=None) == WORKSPACE and call(wsb=256) == WORKSPACE
    assert score(T=0) == 0 and score(lp=None) == INVALID
    for kw in (dict(dt=2), dict(ghs=63), dict(gws=63), dict(ge=FAKE + 2)):
        assert grad(**kw) == INVALID, kw
    for kw in (dict(gh=FAKE + 2), dict(gw=FAKE + 8), dict(ghs=68), dict(gws=100)):
        assert grad(**kw) == UNSUPPORTED, kw
    assert grad(gh=None, gw=None) == 0 and grad(T=0, gw=None) == 0 and grad(T=0, acc=1) == 0


def test_the_fault_word_needs_a_device():
    assert cs.lib_handle().dllm_fault_word(None) == INVALID
    if not torch.cuda.is_available():
        with pytest.raises(cs.DllmError):
            cs.kernel_fault()


def embed(t=FAKE, B=2, L=8, ts=8, w=FAKE, dt=1, V=100, d=64, wst=64, scale=1.0, out=FAKE):
    return cs.lib_handle().dllm_embed_tokens(t, B, L, ts, w, dt, V, d, wst, scale, out, None)


def embed_grad(t=FAKE, B=2, L=8, ts=8, w=FAKE, dt=1, V=100, d=64, wst=64, scale=1.0, out=FAKE, odt=1, acc=0, ws=FAKE,
               wsb=1 << 50):
    return cs.lib_handle().dllm_embed_tokens_backward(t, B, L, ts, w, dt, V, d, scale, out, odt, wst, acc, ws, wsb, None)


def test_embed_refusals():
    for call in (embed, embed_grad):
        for kw in (dict(t=None), dict(B=-1), dict(L=-1), dict(ts=7), dict(w=None), dict(dt=2), dict(V=0), dict(V=1 << 31),
                   dict(d=0), dict(wst=63), dict(scale=math.inf), dict(scale=math.nan), dict(out=None), dict(t=FAKE + 1),
                   dict(B=1 << 40, L=1 << 40, ts=1 << 40)):
            assert call(**kw) == INVALID, (call, kw)
        for kw in (dict(w=FAKE + 4), dict(out=FAKE + 8), dict(d=60), dict(wst=66), dict(dt=0, d=62, wst=64),
                   dict(B=1 << 16, L=1 << 15, ts=1 << 15)):
            assert call(**kw) == UNSUPPORTED, (call, kw)
        assert call(dt=0, d=62) == UNSUPPORTED
    assert embed(B=0) == 0 and embed(L=0) == 0
    assert embed_grad(odt=2) == INVALID and embed_grad(ws=None) == WORKSPACE and embed_grad(wsb=16) == WORKSPACE
    assert embed_grad(ws=FAKE + 8) == INVALID and embed_grad(dt=0, d=60) == UNSUPPORTED


FAR = [FAKE << k for k in range(1, 12)]                  # apart by more than the small calls below touch


def test_overlapping_outputs_are_refused():
    """(Only refused calls: the addresses are made up.)"""
    h, w, t, lp, ent, lse, ws, g, gh, gw = FAR[:10]
    good = dict(h=h, w=w, t=t, lp=lp, ent=ent, lse=lse, ws=ws)
    for kw in (dict(lp=h), dict(ent=w + 99 * 128 + 124), dict(lse=t + 12), dict(lp=ent + 12), dict(ws=h - 16), dict(lse=ws + 64)):
        assert score(**{**good, **kw}) == INVALID, kw
    good = dict(h=h, w=w, t=t, ent=ent, lse=lse, ws=ws, g=g, gh=gh, gw=gw)
    for kw in (dict(gh=h), dict(gw=w), dict(gh=gw + 99 * 128), dict(gw=h - 16), dict(ge=gw), dict(gw=lse), dict(ws=gw - 16),
               dict(gw=t - 256, dt=0)):
        assert grad(**{**good, **kw}) == INVALID, kw
    assert embed(t=t, w=w, out=w + 128) == INVALID and embed(t=t, w=w, out=t - 16) == INVALID
    good = dict(t=t, w=g, out=gw, ws=ws)
    for kw in (dict(out=g), dict(out=t - 16), dict(ws=g), dict(ws=gw + 99 * 128)):
        assert embed_grad(**{**good, **kw}) == INVALID, kw


def test_the_binding_refuses_host_tensors():
    h, w, t = torch.zeros((2, 8), dtype=torch.bfloat16), torch.zeros((5, 8), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(2)
    for call in (lambda: cs.lm_head_logprobs(h, w, t), lambda: cs.lm_head_logprobs_backward(h, w, t, f, f, f),
                 lambda: cs.embed_tokens(t, w), lambda: cs.embed_tokens_backward(t, h, 5), lambda: cs.score_hidden(h, w, t),
                 lambda: cs.embed_canvas(t, w)):
        with pytest.raises(ValueError):
            call()


def test_reference_scores_and_gradients_against_differences():
    """The formulas that the GPU is held to, against autograd of a plain softmax and against differences."""
    g = torch.Generator().manual_seed(1)
    T, V, d, sup = 6, 11, 5, [4]
    h, w = torch.randn((T, d), generator=g, dtype=torch.float64), torch.randn((V, d), generator=g, dtype=torch.float64)
    t = torch.tensor([0, 10, -1, 4, 3, 11])
    a, b = torch.randn(T, generator=g, dtype=torch.float64), torch.randn(T, generator=g, dtype=torch.float64)

    def loss(h, w):
        lp, ent, _ = scores(h, w, t, sup)
        keep = torch.tensor([1.0, 1.0, 0.0, 0.0, 1.0, 0.0], dtype=torch.float64)      # (a suppressed target has no gradient)
        return float((a * torch.nan_to_num(lp, neginf=0.0) * keep).sum() + (b * ent).sum())

    lp, ent, lse = scores(h, w, t, sup)
    p = torch.softmax(torch.cat([(h @ w.T)[:, :4], (h @ w.T)[:, 5:]], 1), 1)
    rows = torch.tensor([0, 1, 3, 4])
    assert torch.allclose(ent[rows], -(p * p.log()).sum(1)[rows]) and torch.allclose(lp[0], p[0, 0].log())
    assert float(lp[3]) == -math.inf and float(lp[2]) == 0 and float(lse[5]) == 0
    dz, clean = grads(h, w, t, lse, ent, a, b, sup)
    gh, gw = dz @ w, dz.T @ clean
    assert float(gw[4].abs().max()) == 0 and float(gh[2].abs().max()) == 0
    step = 1e-6
    for x, want in ((h, gh), (w, gw)):
        for i in range(x.shape[0]):
            for j in range(d):
                old = float(x[i, j])
                x[i, j] = old + step
                up = loss(h, w)
                x[i, j] = old - step
                down = loss(h, w)
                x[i, j] = old
                assert abs((up - down) / (2 * step) - float(want[i, j])) < 1e-7


def test_reference_embedding_gradient():
    t = torch.tensor([[2, 0, 2], [-1, 4, 5]])
    g = torch.arange(24.0).view(2, 3, 4)
    out = embedding_grad(t, g, 5, 2.0)
    assert torch.equal(out[2], 2 * (g[0, 0] + g[0, 2]).double()) and torch.equal(out[4], 2 * g[1, 1].double())
    assert not bool(out[1].any() or out[3].any()) and torch.equal(out[0], 2 * g[0, 1].double())


def test_a_captured_gradient_beside_a_living_graph_of_the_default_stream(monkeypatch):
    """On the CPU, with the two questions about streams answered by the test."""
    from commit_step_gb300 import head

    class Twice(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, y, n):
            return x * y.sum()

        @staticmethod
        def backward(ctx, g):
            head._may_capture(ctx)
            return g, None, None

    stream, capturing = [0], [False]
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: stream[0], raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])

    def graph(x, y, on):
        stream[0] = on
        out = Twice.apply(x, y, 3)
        head._stamp(out)
        return out.sum()

    w, v = torch.ones(4, requires_grad=True), torch.ones(2)
    head._stamp(Twice.apply(v, v, 3))                        # nothing to differentiate
    kept = graph(w, v, 0)
    kept.backward()
    capturing[0] = True
    captured = graph(w, v, 7)
    with pytest.raises(RuntimeError, match="default stream"):
        captured.backward()
    graph(w * 2, v, 7).backward()                            # not made from the leaf itself
    del kept, captured
    graph(w, v, 7).backward()
    capturing[0] = False
    warm = graph(w, v, 5)                                    # first made on a stream that may join a capture
    kept = graph(w, v, 0)
    capturing[0] = True
    graph(w, v, 7).backward()
    assert float(w.grad[0]) > 0 and warm is not None and kept is not None


def test_accumulators_that_something_else_made(monkeypatch):
    """Where an accumulator runs is known once it has run, whatever stream it was first scored on.  As above."""
    import gc
    import weakref

    from commit_step_gb300 import head

    class Twice(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return x * 2

        @staticmethod
        def backward(ctx, g):
            head._may_capture(ctx)
            return g * 2

    stream, capturing = [0], [False]
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: stream[0], raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])

    def step(w, on, accumulates_on):
        stream[0] = on
        out = Twice.apply(w)
        head._stamp(out)
        stream[0] = accumulates_on                           # (what the engine would make current)
        out.sum().backward()

    for made_on, scored_on in ((7, 0), (0, 7)):
        w = torch.ones(4, requires_grad=True)
        keeps = w.expand_as(w)                               # the accumulator, made elsewhere and kept
        capturing[0] = False
        step(w, scored_on, made_on)
        capturing[0] = True
        if made_on == 0:
            with pytest.raises(RuntimeError, match="default stream"):
                step(w, 9, made_on)
        else:
            step(w, 9, made_on)
        marks = keeps.grad_fn.next_functions[0][0].metadata
        assert marks[head._STREAM] == made_on
        gone = weakref.ref(w)
        del w, keeps, marks
        gc.collect()
        assert gone() is None                                # nothing holds the accumulator

