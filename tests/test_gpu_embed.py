"""The embedding of a canvas and its gradient on the GPU, against 64-bit sums.

Tolerances (derived): the forward pass is one product in 32 bits, rounded once:
compared bit for bit with the same in torch.  A gradient row is a sum of n terms
in 32 bits: at most n 2^-24 of the sum of their magnitudes (2^-23 with the
product by the scale and an addition), then rounded to its type (half a step).
"""
import math

import pytest
import torch

from head_reference import embedding_grad

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


def canvas(B, L, V, seed, masked=0.0, outside=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = (torch.rand((B, L), device="cuda", generator=g) ** 2 * V).long().clamp_(max=V - 1)
    t = torch.where(torch.rand((B, L), device="cuda", generator=g) < masked, V // 2, t)
    odd = torch.tensor([-1, V, 2 ** 31 - 1, -2 ** 31], device="cuda")[torch.randint(0, 4, (B, L), device="cuda", generator=g)]
    t = torch.where(torch.rand((B, L), device="cuda", generator=g) < outside, odd, t)
    wide = torch.full((B, L + 13), -7, dtype=torch.int32, device="cuda")
    wide[:, 5:5 + L] = t.to(torch.int32)
    return wide[:, 5:5 + L]


def check(got, tokens, grad, V, scale, old=None):
    want = embedding_grad(tokens, grad, V, scale)
    size = embedding_grad(tokens, grad.abs(), V, abs(scale))
    count = embedding_grad(tokens, torch.ones_like(grad[..., :1]), V)
    if old is not None:
        want, size = want + old.double(), size + old.double().abs()
    lim = (count + 1) * 2.0 ** -23 * size + torch.finfo(got.dtype).eps / 2 * want.abs() * (1 + 2.0 ** -7)
    err = (got.double() - want).abs()
    assert bool((err <= lim).all()), float((err - lim).max())


@TYPES
@pytest.mark.parametrize("B,L,V,d", [(1, 1, 1, 8), (1, 32, 1000, 4096), (3, 17, 50, 72), (2, 333, 5000, 264), (4, 1025, 300, 16)])
def test_embedding(cs, dtype, B, L, V, d):
    w = torch.randn((V, d), device="cuda").to(dtype)
    t = canvas(B, L, V, B + L, 0.3, 0.1)
    ok = (t >= 0) & (t < V)
    rows = w[torch.where(ok, t, torch.zeros_like(t)).long()]
    for scale in (1.0, math.sqrt(d), -0.37):
        want = (rows.float() * torch.tensor(scale, dtype=F32, device="cuda")).to(dtype)
        want = torch.where(ok[..., None], want, torch.zeros_like(want))
        got = cs.embed_tokens(t, w, scale=scale)
        assert got.shape == (B, L, d) and torch.equal(got, want)
    wide = torch.full((V, d + 16), math.nan, dtype=dtype, device="cuda")
    wide[:, :d] = w
    out = torch.empty((B, L, d), dtype=dtype, device="cuda")
    assert cs.embed_tokens(t, wide[:, :d], out=out) is out and torch.equal(out, torch.where(ok[..., None], rows, torch.zeros_like(rows)))
    assert torch.equal(cs.embed_tokens(t[0].contiguous(), w), out[0])


def test_embedding_keeps_nan_and_infinities(cs):
    w = torch.randn((4, 16), device="cuda").to(BF16)
    w[1, 3], w[2, 4], w[2, 5] = math.nan, math.inf, -math.inf
    got = cs.embed_tokens(torch.tensor([2, 1, 0, 9], dtype=torch.int32, device="cuda"), w, scale=2.0)
    assert torch.isnan(got[1, 3]) and got[0, 4] == math.inf and got[0, 5] == -math.inf and not bool(got[3].any())


SIZES = [(1, 1, 1, 8, 0.0), (1, 2, 3, 8, 0.0), (1, 64, 7, 16, 0.0), (1, 65, 5000, 72, 0.5), (2, 64, 4, 24, 1.0),
         (3, 333, 1000, 264, 0.5), (1, 2047, 1023, 40, 0.1), (1, 2049, 1024, 40, 0.9), (4, 1025, 70000, 16, 0.4),
         (2, 9000, 1 << 20, 8, 0.6), (1, 3000, (1 << 21) + 77, 8, 0.1), (3, 40, 9, 40000, 0.5), (16, 4096, 300, 520, 0.5), (1, 70001, 126464, 32, 0.99)]


@TYPES
@pytest.mark.parametrize("B,L,V,d,masked", SIZES)
def test_gradient(cs, dtype, B, L, V, d, masked):
    t = canvas(B, L, V, B + L + V, masked, 0.05)
    grad = torch.randn((B, L, d), device="cuda").to(dtype)
    for scale in (1.0, 2.3):
        check(cs.embed_tokens_backward(t, grad, V, scale=scale), t, grad, V, float(torch.tensor(scale, dtype=F32)))


@TYPES
@pytest.mark.parametrize("out_dtype", [BF16, F32], ids=["to-bf16", "to-f32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_given_output(cs, dtype, out_dtype, accumulate):
    B, L, V, d = 2, 500, 700, 136
    t = canvas(B, L, V, 3, 0.5, 0.1)
    grad = torch.randn((B, L, d), device="cuda").to(dtype)
    wide = torch.randn((V, d + 24), device="cuda").to(out_dtype)
    old = wide.clone()
    got = cs.embed_tokens_backward(t, grad, V, scale=0.5, out=wide[:, :d], accumulate=accumulate)
    assert got.data_ptr() == wide.data_ptr() and torch.equal(wide[:, d:], old[:, d:])
    check(got, t, grad, V, 0.5, old[:, :d] if accumulate else None)
    if accumulate:
        named = torch.zeros(V, dtype=torch.bool, device="cuda")
        named[t[(t >= 0) & (t < V)].long()] = True
        assert torch.equal(got[~named], old[:, :d][~named])


@pytest.mark.parametrize("kind", ["one", "outside", "distinct", "two", "sorted", "falling"])
def test_orders_of_tokens(cs, kind):
    T, V, d = 5000, 6000, 24
    i = torch.arange(T, device="cuda")
    t = {"one": torch.full_like(i, 17), "outside": torch.full_like(i, -1), "distinct": torch.randperm(V, device="cuda")[:T],
         "two": i % 2 * 5999, "sorted": i // 70, "falling": (T - i) // 64}[kind].to(torch.int32)
    grad = torch.randn((T, d), device="cuda").to(BF16)
    got = cs.embed_tokens_backward(t, grad, V)
    check(got, t, grad, V, 1.0)
    assert torch.equal(got, cs.embed_tokens_backward(t, grad, V))


def test_offsets_past_32_bits(cs):
    """Rows of a weight and of its gradient, then tokens of a canvas, whose elements lie past 2^31."""
    V, d, step = 1000, 64, 1 << 22
    t = canvas(2, 700, V, 60, 0.1, 0.1)
    t[0, :2] = torch.tensor([V - 1, V - 2], device="cuda")
    w = torch.empty((V * step,), dtype=BF16, device="cuda").as_strided((V, d), (step, 1)).copy_(torch.randn((V, d)))
    ok = (t >= 0) & (t < V)
    want = torch.where(ok[..., None], w[torch.where(ok, t, torch.zeros_like(t)).long()], torch.zeros((), dtype=BF16, device="cuda"))
    assert torch.equal(cs.embed_tokens(t, w), want)
    g = torch.randn((2, 700, d), device="cuda").to(BF16)
    check(cs.embed_tokens_backward(t, g, V, out=w), t, g, V, 1.0)
    del w
    B, L, V, d = 2, 270000, 50, 4096                       # 2.2e9 elements
    t = torch.randint(0, V, (B, L), dtype=torch.int32, device="cuda")
    w = torch.randn((V, d), device="cuda").to(BF16)
    x = cs.embed_tokens(t, w)
    for b in range(B):
        for l in range(0, L, 45000):
            assert torch.equal(x[b, l:l + 45000], w[t[b, l:l + 45000].long()])
    value = torch.arange(B * L, device="cuda") % 7         # (whole numbers: every order gives the same sum)
    x.copy_(value.view(B, L, 1))
    out = cs.embed_tokens_backward(t, x, V, out=torch.empty((V, d), device="cuda"))
    want = torch.bincount(t.view(-1).long(), weights=value.double(), minlength=V)
    assert torch.equal(out.double(), want[:, None].expand(V, d))


def test_no_tokens(cs):
    t, g = torch.empty((3, 0), dtype=torch.int32, device="cuda"), torch.empty((3, 0, 16), dtype=BF16, device="cuda")
    assert cs.embed_tokens(t, torch.randn((5, 16), device="cuda").to(BF16)).shape == (3, 0, 16)
    out = torch.ones((5, 16), dtype=BF16, device="cuda")
    assert bool((cs.embed_tokens_backward(t, g, 5, out=out, accumulate=True) == 1).all())
    assert not bool(cs.embed_tokens_backward(t, g, 5, out=out).any())


def test_nan_reaches_its_own_row_only(cs):
    t = torch.tensor([3, 5, 3, -1, 9], dtype=torch.int32, device="cuda")
    g = torch.ones((5, 16), dtype=BF16, device="cuda")
    g[2, 1], g[3] = math.nan, math.nan
    got = cs.embed_tokens_backward(t, g, 12)
    assert torch.isnan(got[3, 1]) and int(torch.isnan(got).sum()) == 1 and float(got[3, 0]) == 2.0


def test_autograd_of_canvases_of_any_strides(cs):
    w = torch.randn((50, 16), device="cuda").to(torch.bfloat16).requires_grad_()
    t = torch.randint(-1, 51, (6, 9), dtype=torch.int32, device="cuda")
    for view in (t.T, t[:, ::2], t[:1].expand(5, 9), t[:, :1].expand(6, 4), t[2:, 3:], t.T[4], t[0, :1], t[:0]):
        got = cs.embed_canvas(view, w)
        want = cs.embed_tokens(view.contiguous(), w.detach())
        assert torch.equal(got, want)
        g = torch.randn_like(got)
        grad, = torch.autograd.grad(got, w, g)
        assert torch.equal(grad, cs.embed_tokens_backward(view.contiguous(), g, 50))


def test_autograd_and_tied_weight(cs):
    """Embedding and head share a weight: one gradient, the embedding's added to the head's."""
    V, d, B, L = 500, 128, 2, 40
    w = (torch.randn((V, d), device="cuda") / math.sqrt(d)).to(BF16).requires_grad_()
    t = canvas(B, L, V, 8, 0.5)
    target = torch.where(t == V // 2, torch.randint(0, V, (B, L), dtype=torch.int32, device="cuda"), -1).contiguous()
    x = cs.embed_canvas(t, w, scale=math.sqrt(d))
    lp, _ = cs.score_hidden(x, w, target)
    (-lp.sum() / B).backward()
    # the same by hand
    wd = w.detach()
    xd = cs.embed_tokens(t, wd, scale=math.sqrt(d))
    _, ent, lse = cs.lm_head_logprobs(xd, wd, target)
    gx, gw = cs.lm_head_logprobs_backward(xd, wd, target, lse, ent, torch.full((B, L), -1.0 / B, device="cuda"),
                                          out=(None, torch.empty((V, d), device="cuda")))
    cs.embed_tokens_backward(t, gx, V, scale=math.sqrt(d), out=gw, accumulate=True)
    both = gw.double()
    # the engine adds two bf16 gradients: two roundings and the sum's
    a = cs.lm_head_logprobs_backward(xd, wd, target, lse, ent, torch.full((B, L), -1.0 / B, device="cuda"))[1]
    b = cs.embed_tokens_backward(t, gx, V, scale=math.sqrt(d))
    lim = 2.0 ** -8 * (a.double().abs() + b.double().abs() + w.grad.double().abs()) * (1 + 2.0 ** -7) + 1e-6
    assert bool(((w.grad.double() - both).abs() <= lim).all())
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        g, = torch.autograd.grad(cs.embed_canvas(t, w).float().square().sum(), w, create_graph=True)
        g.float().sum().backward()


def test_the_fault_word_and_the_workspaces_contents(cs):
    t = canvas(3, 700, 900, 5, 0.5)
    grad = torch.randn((3, 700, 64), device="cuda").to(BF16)
    need = cs.lib_handle().dllm_embed_tokens_backward_workspace_size(2100, 900, 64)
    got = []
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got.append(cs.embed_tokens_backward(t, grad, 900, ws=ws))
        if fill == 0:
            assert cs.workspace_fault(ws) == 0
    assert torch.equal(got[0], got[1])


def test_two_threads_on_one_stream(cs):
    import threading

    jobs = []
    for i in range(2):
        t = canvas(2, 900 + 400 * i, 5000, 10 + i, 0.5)
        g = torch.randn((*t.shape, 128), device="cuda").to(BF16)
        jobs.append((t, g, cs.embed_tokens_backward(t, g, 5000)))
    torch.cuda.synchronize()
    bad = []

    def work(t, g, want):
        for _ in range(40):
            if not torch.equal(cs.embed_tokens_backward(t, g, 5000), want):
                bad.append(t.shape)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not bad


def test_outputs_written_before_are_complete(cs):
    """The zero rows run ahead of the sums: what a kernel just before the call writes into the output is replaced."""
    V, d = 30000, 512
    t = canvas(1, 100, V, 9, 0.3)
    g = torch.randn((1, 100, d), device="cuda").to(BF16)
    want = cs.embed_tokens_backward(t, g, V)
    out = torch.empty_like(want)
    for _ in range(20):
        out.fill_(3.0)
        cs.embed_tokens_backward(t, g, V, out=out)
        assert torch.equal(out, want)


def test_the_binding_refuses(cs):
    w = torch.zeros((10, 16), dtype=BF16, device="cuda")
    t = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    g = torch.zeros((2, 4, 16), dtype=BF16, device="cuda")
    for bad in (lambda: cs.embed_tokens(t.long(), w), lambda: cs.embed_tokens(t, w.half()), lambda: cs.embed_tokens(t[None], w),
                lambda: cs.embed_tokens_backward(t, g.half(), 10), lambda: cs.embed_tokens_backward(t, g, 10, out=g.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: cs.embed_tokens(t.T, w), lambda: cs.embed_tokens(t, w.T), lambda: cs.embed_tokens(t.cpu(), w),
                lambda: cs.embed_tokens(t, w, out=g[:1]), lambda: cs.embed_tokens_backward(t, g[:1], 10),
                lambda: cs.embed_tokens_backward(t, g, 0), lambda: cs.embed_tokens_backward(t, g, 1 << 31),
                lambda: cs.embed_tokens_backward(t, g, 10, accumulate=True),
                lambda: cs.embed_tokens_backward(t, g, 10, out=w[:9].clone()),
                lambda: cs.embed_tokens_backward(t, g.transpose(0, 1), 10)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cs.embed_tokens(t, w[:, :4].contiguous()), lambda: cs.embed_tokens(t, w, scale=math.inf),
                lambda: cs.embed_tokens_backward(t, g, 10, ws=torch.zeros(16, dtype=torch.uint8, device="cuda")),
                lambda: cs.embed_tokens_backward(t, g, 8, out=g.view(8, 16))):
        with pytest.raises(cs.DllmError):
            bad()


def test_side_stream_and_graph(cs):
    t = canvas(3, 700, 900, 4, 0.5)
    grad = torch.randn((3, 700, 64), device="cuda").to(BF16)
    want = cs.embed_tokens_backward(t, grad, 900)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cs.embed_tokens_backward(t, grad, 900, stream=side)
    emb = cs.embed_tokens(t, want, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(emb, want[t.long()])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = cs.embed_tokens_backward(t, grad, 900)
        emb = cs.embed_tokens(t, cap, scale=3.0)
    t.copy_(t.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap, cs.embed_tokens_backward(t, grad, 900))
    assert torch.equal(emb, cs.embed_tokens(t, cap, scale=3.0))
