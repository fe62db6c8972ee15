"""Block decoding over the paged 8-bit cache, and a policy-gradient score of the result.

A one-layer model with random weights stands in for a masked diffusion
language model.  For each block: a few denoising steps, in each of which the
block's keys and values are (re)appended to the cache, every query of the
block attends over everything cached, and the commit step places the most
confident tokens; when a sequence's cache is full, the tokens that drew the
least attention are evicted into fresh pages.  At the end the generated tokens
are scored under the model, with alternatives, and the score is differentiated.

    python examples/cached_block_decode.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import commit_step_gb300 as cs  # noqa: E402


class TinyBlockModel:
    """Embedding, one attention layer with shared key heads, and an LM head."""

    def __init__(self, vocab=1000, heads=8, kv_heads=2, head_dim=64, seed=0, device="cuda"):
        g = torch.Generator(device="cpu").manual_seed(seed)
        d = heads * head_dim

        def w(*shape):
            return (torch.randn(shape, generator=g) / math.sqrt(shape[-1])).to(torch.bfloat16).to(device)

        self.vocab, self.heads, self.kv_heads, self.head_dim, self.mask_id = vocab, heads, kv_heads, head_dim, vocab - 1
        self.embed = w(vocab, d) * math.sqrt(d)
        self.qkv = w(d + 2 * kv_heads * head_dim, d)
        self.proj, self.head = w(d, d), w(vocab, d) * 4

    def project(self, tokens):
        """Queries, keys and values of (B, L) tokens: slices of one product."""
        B, L = tokens.shape
        x = self.embed[tokens.long()]
        y = (x @ self.qkv.T).view(B, L, -1, self.head_dim)
        H, K = self.heads, self.kv_heads
        return x, y[:, :, :H], y[:, :, H:H + K], y[:, :, H + K:]

    def logits(self, x, attended):
        h = x + attended.reshape(x.shape) @ self.proj.T
        return h @ self.head.T


def decode(model, prompt, *, gen_len=64, block_len=16, steps=4, budget=48, page_size=16, attention=None):
    """Returns (tokens (B, gen_len), logits that scored them (B, gen_len, V),
    cached lengths (B,)).  ``attention``: by default ``cache_attention``."""
    attention = attention or cs.cache_attention
    dev = prompt.device
    B, P = prompt.shape
    # A sequence's cache never holds more than the larger of its prompt and its budget, and one block.
    width = -(-(max(P, budget) + block_len) // page_size)
    cache = cs.KVCache(2 * B * width, page_size, model.kv_heads, model.head_dim, device=dev)
    tables = torch.arange(2 * B * width, dtype=torch.int32, device=dev).view(2, B, width)
    table, spare = tables[0].contiguous(), tables[1].contiguous()
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    weights = torch.zeros((B, model.kv_heads, width * page_size), device=dev)

    _, _, k, v = model.project(prompt)
    cs.cache_append(cache, k, v, table, lens)
    lens = lens + P
    tokens, logits = [], []
    for _ in range(gen_len // block_len):
        block = torch.full((B, block_len), model.mask_id, dtype=torch.int32, device=dev)
        for step in range(steps):
            x, q, k, v = model.project(block)
            cs.cache_append(cache, k, v, table, lens)          # again at the same place: the block so far
            out, _ = attention(q, cache, table, lens + block_len)
            z = model.logits(x, out).contiguous()
            quota = block_len // steps if step < steps - 1 else block_len
            cs.commit_step(z, rule=cs.RULE_TOPK, k=quota, mask_id=model.mask_id, suppress_ids=[model.mask_id],
                           canvas=block)
        # The block as it was placed: what stays in the cache, what its tokens attend to, and its logits.
        x, q, k, v = model.project(block)
        cs.cache_append(cache, k, v, table, lens)
        lens = lens + block_len
        out, _ = attention(q, cache, table, lens, weights=weights, decay=0.9)
        tokens.append(block)
        logits.append(model.logits(x, out))
        if int(lens.max()) + block_len > width * page_size:
            # Full: keep the first tokens, the latest block and what drew most attention.
            _, lens, weights = cs.cache_evict(cache, table, lens, weights, budget, spare, keep_first=4,
                                              keep_last=block_len)
            table, spare = spare, table
    return torch.cat(tokens, 1), torch.cat(logits, 1), lens


def score(model, tokens, logits, advantage):
    """The policy-gradient loss of the tokens, their alternatives, and the logits' gradient."""
    logits = logits.detach().requires_grad_()
    logprob, entropy, top_ids, top_logprob = cs.score_tokens(logits, tokens, top=4, suppress_ids=(model.mask_id,))
    loss = -(advantage[:, None] * logprob).mean() - 0.01 * entropy.mean()
    loss.backward()
    return loss.detach(), logprob.detach(), top_ids, top_logprob.detach(), logits.grad


def main():
    torch.manual_seed(0)
    model = TinyBlockModel()
    prompt = torch.randint(0, model.vocab - 1, (2, 40), dtype=torch.int32).cuda()
    tokens, logits, lens = decode(model, prompt)
    loss, logprob, top_ids, top_logprob, grad = score(model, tokens, logits, torch.tensor([1.0, -0.5], device="cuda"))
    print("tokens", tokens[0, :8].tolist(), "... cached", lens.tolist())
    print("log probabilities", [round(v, 3) for v in logprob[0, :8].tolist()])
    print("alternatives of the first", top_ids[0, 0].tolist(), [round(v, 3) for v in top_logprob[0, 0].tolist()])
    print(f"loss {loss.item():.4f}, gradient norm {grad.float().norm().item():.4f}")


if __name__ == "__main__":
    main()
