"""The cached decoding example: runs, and with its attention replaced by one
computed in torch from the cache's values it places the same tokens."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("cached_block_decode",
                                                  os.path.join(ROOT, "examples", "cached_block_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def torch_attention(q, cache, table, lens, weights=None, decay=1.0):
    """cache_attention in fp64 torch operations (every page of the table exists)."""
    B, L, Hq, D = q.shape
    t = table.long()
    H, ps = cache.heads, cache.page_size

    def values(codes, scale):
        x = codes.view(torch.uint8)[t].view(torch.float8_e4m3fn).double() * scale[t].double()[..., None, None]
        return x.transpose(1, 2).reshape(B, H, -1, D).repeat_interleave(Hq // H, 1)

    k, v = values(cache.k, cache.k_scale), values(cache.v, cache.v_scale)
    here = torch.arange(k.shape[2], device=q.device)[None] < lens[:, None]
    x = q.double().transpose(1, 2) @ k.transpose(2, 3) / math.sqrt(D)
    x = x.masked_fill(~here[:, None, None], -math.inf)
    p = torch.softmax(x, -1)
    if weights is not None:
        weights.mul_(decay).add_(p.view(B, H, -1, p.shape[-1]).sum(2).float())
    return (p @ v).transpose(1, 2).to(torch.bfloat16), torch.logsumexp(x, -1).transpose(1, 2).float()


def test_the_models_embedding(cs):
    """The canvas is embedded by ``embed_tokens``: the rows of the table, an id outside it zeros."""
    model = example().TinyBlockModel(seed=2)
    tokens = torch.randint(0, model.vocab, (3, 16), dtype=torch.int32).cuda()
    x, q, k, v = model.project(tokens)
    assert torch.equal(x, model.embed[tokens.long()])
    tokens[1, 5] = -1
    assert not bool(model.project(tokens)[0][1, 5].any())


def test_example_runs_and_matches_a_plain_attention(cs):
    m = example()
    torch.manual_seed(1)
    model = m.TinyBlockModel(seed=3)
    prompt = torch.randint(0, model.vocab - 1, (3, 37), dtype=torch.int32).cuda()
    tokens, logits, lens = m.decode(model, prompt)
    again, logits_plain, lens_plain = m.decode(model, prompt, attention=torch_attention)
    assert tokens.shape == (3, 64) and not (tokens == model.mask_id).any()
    assert torch.equal(lens, lens_plain) and int(lens.max()) < 37 + 64      # something was evicted
    # bf16 activations: a rounding of the attention's output can move a near tie, nothing more
    assert (tokens == again).float().mean() > 0.9
    adv = torch.tensor([1.0, 0.5, -1.0], device="cuda")
    loss, logprob, top_ids, top_logprob, grad = m.score(model, tokens, logits, adv)
    z = logits.detach().double().clone().requires_grad_()
    masked = z.index_fill(2, torch.tensor([model.mask_id], device="cuda"), -math.inf)
    logp = torch.log_softmax(masked, -1)
    lp = logp.gather(2, tokens.long()[..., None])[..., 0]
    ent = -(logp.exp() * logp.clamp(min=-1e4)).sum(-1)
    want = -(adv[:, None].double() * lp).mean() - 0.01 * ent.mean()
    want.backward()
    assert abs(loss.double() - want.detach()) < 1e-4
    assert (logprob.double() - lp.detach()).abs().max() < 2.0 ** -12
    # the gradient in bf16: half a step of each value and of the largest's fp32 error
    err = (grad.double() - z.grad).abs()
    assert (err <= 2.0 ** -8 * z.grad.abs() + 2.0 ** -20).all()
