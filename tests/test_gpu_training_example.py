"""The training example: it runs, and its gradients are those of the same model in 64-bit torch operations."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("masked_training_step",
                                                  os.path.join(ROOT, "examples", "masked_training_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients(cs):
    m = example()
    model = m.TinyMaskedModel(seed=4)
    tokens = torch.randint(0, model.vocab - 1, (4, 64), dtype=torch.int32, generator=torch.Generator().manual_seed(5)).cuda()
    value = m.loss(model, tokens, torch.Generator().manual_seed(6), entropy_bonus=0.05)
    value.backward()
    w, mix, dense = [p.detach().double().requires_grad_() for p in model.parameters()]
    canvas, targets, weight = m.noised(tokens, model.mask_id, torch.Generator().manual_seed(6))
    x = w[canvas.long()] * math.sqrt(model.d)
    y = x + torch.einsum("lm,bmd->bld", mix, x)
    z = (y + torch.tanh(y @ dense)) @ w.T
    z = z.index_fill(2, torch.tensor([model.mask_id], device="cuda"), -math.inf)
    logp = torch.log_softmax(z, -1)
    on = (targets >= 0).double()
    lp = logp.gather(2, targets.clamp(min=0).long()[..., None])[..., 0] * on
    p = logp.exp()
    ent = -(p * torch.where(p > 0, logp, torch.zeros_like(logp))).sum(-1) * on
    want = (-(weight.double() * lp).sum() - 0.05 * ent.sum()) / tokens.numel()
    want.backward()
    # Activations and gradients pass through a dozen roundings to bf16, each 2^-8 of a value at most and of the same
    # spread: together about sqrt(12 / 3) 2^-8 of the norm, held to twice that.
    assert abs(value.item() - want.item()) <= 2.0 ** -6 * abs(want.item())
    for got, ref in zip(model.parameters(), (w, mix, dense)):
        assert float((got.grad.double() - ref.grad).norm()) <= 4 * 2.0 ** -8 * float(ref.grad.norm())


def test_a_captured_step(cs):
    """Forward and backward as one graph: what it replays is what the eager step computes."""
    m = example()
    model = m.TinyMaskedModel(seed=7)
    tokens = torch.randint(0, model.vocab - 1, (4, 64), dtype=torch.int32, generator=torch.Generator().manual_seed(8)).cuda()
    canvas, targets, weight = m.noised(tokens, model.mask_id, torch.Generator().manual_seed(9))

    def step():
        lp, ent = cs.score_hidden(model.hidden(canvas), model.weight, targets, suppress_ids=(model.mask_id,))
        value = (-(weight * lp).sum() - 0.01 * ent.sum()) / tokens.numel()
        return value.detach(), torch.autograd.grad(value, model.parameters())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        value, grads = step()
    for seed in (10, 11):
        c, t, w = m.noised(tokens, model.mask_id, torch.Generator().manual_seed(seed))
        canvas.copy_(c), targets.copy_(t), weight.copy_(w)
        graph.replay()
        torch.cuda.synchronize()
        got = [value.clone(), *[g.clone() for g in grads]]
        want_value, want = step()
        # (torch's own products may add in another order inside a graph)
        assert abs(got[0].item() - want_value.item()) <= 2.0 ** -8 * abs(want_value.item())
        for a, b in zip(got[1:], want):
            assert float((a.double() - b.double()).norm()) <= 2.0 ** -7 * float(b.double().norm())


def test_a_captured_step_beside_a_living_result(cs):
    """The leaves' accumulators of a result made on the default stream run there: a captured gradient is refused while
    it lives, and made when it is gone."""
    w = torch.randn((50, 16), device="cuda").to(torch.bfloat16).requires_grad_()
    t = torch.randint(0, 50, (2, 9), dtype=torch.int32, device="cuda")
    x = torch.randn((2, 9, 16), device="cuda").to(torch.bfloat16)
    for value in (lambda: cs.score_hidden(x, w, t)[0].sum(), lambda: cs.embed_canvas(t, w).float().square().sum()):
        want, = torch.autograd.grad(value(), w)
        kept = value()
        with pytest.raises(RuntimeError, match="default stream"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                torch.autograd.grad(value(), w)
        del kept
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got, = torch.autograd.grad(value(), w)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("made_on_side", [True, False])
def test_a_captured_step_of_leaves_whose_accumulators_something_else_keeps(cs, made_on_side):
    """As a data-parallel wrapper keeps them.  Made on a side stream, a step on the default stream before the capture does no
    harm; made on the default stream, a warm-up on a side stream does not hide it."""
    w = torch.randn((50, 16), device="cuda").to(torch.bfloat16).requires_grad_()
    t = torch.randint(0, 50, (2, 9), dtype=torch.int32, device="cuda")
    x = torch.randn((2, 9, 16), device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    default = torch.cuda.current_stream()

    def step():
        w.grad = None
        cs.score_hidden(x, w, t)[0].sum().backward()
        return w.grad

    with torch.cuda.stream(side if made_on_side else default):
        keeps = w.expand_as(w)
    with torch.cuda.stream(default if made_on_side else side):
        want = step().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if not made_on_side:
        with pytest.raises(RuntimeError, match="default stream"):
            with torch.cuda.graph(graph):
                step()
        return
    with torch.cuda.graph(graph):
        got = step()
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and keeps is not None


def test_it_runs(cs):
    example().main()
