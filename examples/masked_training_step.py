"""One training step of a masked diffusion language model whose embedding and LM head share a weight.

A batch of canvases is noised (tokens covered by the mask token, a share drawn
for each sequence), embedded, run through a small bidirectional mixer with random
weights, and scored at the covered positions only, straight from the hidden
states: the logits of the batch are never held.  The shared weight's gradient is
the sum of the head's and the embedding's.

    python examples/masked_training_step.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import commit_step_gb300 as cs  # noqa: E402


class TinyMaskedModel:
    """A shared embedding and head around one layer that mixes the positions and the features."""

    def __init__(self, vocab=1000, d=256, length=64, seed=0, device="cuda"):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.vocab, self.d, self.mask_id = vocab, d, vocab - 1
        self.weight = (torch.randn((vocab, d), generator=g) / math.sqrt(d)).to(torch.bfloat16).to(device).requires_grad_()
        self.mix = (torch.randn((length, length), generator=g) / length).to(torch.bfloat16).to(device).requires_grad_()
        self.dense = (torch.randn((d, d), generator=g) / math.sqrt(d)).to(torch.bfloat16).to(device).requires_grad_()

    def parameters(self):
        return [self.weight, self.mix, self.dense]

    def hidden(self, canvas):
        x = cs.embed_canvas(canvas, self.weight, scale=math.sqrt(self.d))
        y = x + torch.einsum("lm,bmd->bld", self.mix, x)
        return y + torch.tanh(y @ self.dense)


def noised(tokens, mask_id, generator):
    """(canvas, targets, weights): a share t of each sequence covered; targets -1 elsewhere; weights 1 / t."""
    B, L = tokens.shape
    t = torch.rand((B, 1), generator=generator) * 0.9 + 0.1
    covered = (torch.rand((B, L), generator=generator) < t).to(tokens.device)
    canvas = torch.where(covered, torch.full_like(tokens, mask_id), tokens)
    targets = torch.where(covered, tokens, torch.full_like(tokens, -1))
    return canvas, targets, (1.0 / t).to(tokens.device)


def loss(model, tokens, generator, entropy_bonus=0.0):
    canvas, targets, weight = noised(tokens, model.mask_id, generator)
    logprob, entropy = cs.score_hidden(model.hidden(canvas), model.weight, targets, suppress_ids=(model.mask_id,))
    return (-(weight * logprob).sum() - entropy_bonus * entropy.sum()) / tokens.numel()


def main():
    model = TinyMaskedModel()
    tokens = torch.randint(0, model.vocab - 1, (4, 64), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    value = loss(model, tokens, torch.Generator().manual_seed(2), entropy_bonus=0.01)
    value.backward()
    print(f"loss {value.item():.4f}; gradient norms", [round(p.grad.float().norm().item(), 4) for p in model.parameters()])
    with torch.no_grad():
        for p in model.parameters():
            p -= 0.1 * p.grad
    print(f"after a step {loss(model, tokens, torch.Generator().manual_seed(2)).item():.4f}")


if __name__ == "__main__":
    main()
