"""A language model small enough to read, trained with the library end to end.

One table E serves both ends: the hidden vector of token x is c E[x], the
logits of the next token are (c E[x]) E^T.  Every simulated rank draws its own
tokens; a step is, for each rank, the embedding lookup, the cross entropy over
the vocabulary with its gradients, and the embedding's gradient added onto the
head's, straight into the rank's 16-bit gradient vector; then one ZeRO-2 step
over the ranks, clipped by the global norm of their mean gradient.  The step's
16-bit working copy is the next step's table.

The text is synthetic: each word is followed by itself or by its partner, one
as likely as the other, so the loss falls from log(vocab) towards log(2).

    python -m examples.tied_lm [--vocab 4096 --width 256 --tokens 2048 --ranks 4 --steps 60]
"""

from __future__ import annotations

import argparse
import math

import torch

import zero_sharded_mixed_step_gb300 as zs

LR, BETA1, BETA2, EPS = 3e-3, 0.9, 0.95, 1e-8


class TiedLm:
    """The table as a ZeRO-2 context of one unit, and the operators around it."""

    def __init__(self, vocab, width, tokens, ranks, dtype="bf16", seed=0):
        self.vocab, self.width, self.tokens, self.ranks = vocab, width, tokens, ranks
        gen = torch.Generator(device="cuda").manual_seed(seed)
        theta0 = torch.randn(vocab * width, device="cuda", generator=gen) * 0.02
        self.zero = zs.ZeroStep(zs.ZERO_SCHEME_Z2, ranks, [vocab * width], dtype, theta0=theta0, with_grad_buffers=True)
        self.embedding = zs.Embedding(vocab, width, dtype, max_tokens=tokens, scale=1 / (0.02 * math.sqrt(width)))
        self.head = zs.LmLoss(vocab, width, dtype, max_tokens=tokens)
        self.t = 0

    def table(self):
        return self.zero.p16[: self.vocab * self.width].view(self.vocab, self.width)

    def table_grad(self, rank):
        return self.zero.grads[rank][: self.vocab * self.width].view(self.vocab, self.width)

    def backward(self, rank, inputs, targets):
        """The rank's mean loss; its gradient is left in the rank's gradient vector."""
        table = self.table()
        hidden = self.embedding.forward(inputs, table)
        loss, lse = self.head.loss(hidden, table, targets)
        grad = self.table_grad(rank)
        dhidden, _ = self.head.grad(hidden, table, targets, lse, 1.0 / self.tokens, dtable=grad)
        self.embedding.grad(inputs, dhidden, grad, accumulate=True)
        return loss.mean()

    def step(self, batches, max_norm=1.0):
        """One training step over the ranks' (inputs, targets); returns their losses."""
        losses = [self.backward(r, *batch) for r, batch in enumerate(batches)]
        self.t += 1
        self.zero.step(self.zero.grads, LR, BETA1, BETA2, EPS, self.t, max_norm=max_norm)
        return torch.stack(losses)


def batch(vocab, tokens, gen):
    """Words, each followed by itself or by its partner (the word whose number differs in the last bit)."""
    x = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
    other = torch.randint(0, 2, (tokens,), device="cuda", generator=gen)
    return x, x ^ other


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--vocab", type=int, default=4096)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args(argv)
    if a.vocab % 2:
        ap.error("--vocab must be even: every word has a partner")
    model = TiedLm(a.vocab, a.width, a.tokens, a.ranks)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for k in range(a.steps):
        losses = model.step([batch(a.vocab, a.tokens, gen) for _ in range(a.ranks)])
        if k % 10 == 0 or k == a.steps - 1:
            print(f"step {k + 1:4d}  loss {losses.mean().item():.4f}  gradient norm {model.zero.grad_norm.item():.4f}")
    model.head.status()
    return losses.mean().item()


if __name__ == "__main__":
    main()
