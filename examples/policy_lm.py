"""A policy over words small enough to read, trained by policy gradients with
the library end to end.

The model: the hidden vector of word x is c E[x] M, the logits of the answer
are (c E[x] M) E^T, with a tied table E and a square matrix M.  Every simulated
rank answers its own words, one of the likeliest alternatives each; an answer
is rewarded where it is as even or odd as its word.  A step is, for each rank,
the embedding lookup, the log probabilities with entropy and alternatives, the
gradients of -(advantage * logp) - bonus * entropy for the head, M and the
embedding; then, over the ranks, one clipped ZeRO-2 step for the table and one
orthogonalised step for M.

    python -m examples.policy_lm [--vocab 512 --width 192 --tokens 2048 --ranks 4 --steps 60]
"""

from __future__ import annotations

import argparse
import math

import torch

import zero_sharded_mixed_step_gb300 as zs

LR, BETA1, BETA2, EPS = 1e-3, 0.9, 0.95, 1e-8
LR_MATRIX, MU, BONUS = 2e-2, 0.9, 1e-2


class PolicyLm:
    """The table as a ZeRO-2 context, the matrix as an orthogonalised step, and the operators around them."""

    def __init__(self, vocab, width, tokens, ranks, dtype="bf16", alternatives=16, seed=0):
        self.vocab, self.width, self.tokens, self.ranks = vocab, width, tokens, ranks
        gen = torch.Generator(device="cuda").manual_seed(seed)
        theta0 = torch.randn(vocab * width, device="cuda", generator=gen) * 0.02
        matrix0 = torch.eye(width, device="cuda")
        self.zero = zs.ZeroStep(zs.ZERO_SCHEME_Z2, ranks, [vocab * width], dtype, theta0=theta0, with_grad_buffers=True)
        self.muon = zs.MuonStep([(width, width)], ranks, dtype, theta0=[matrix0])
        self.matrix_grads = self.muon.new_grad_buffers()
        self.embedding = zs.Embedding(vocab, width, dtype, max_tokens=tokens, scale=1 / (0.02 * math.sqrt(width)))
        self.head = zs.LmLogprobs(vocab, width, dtype, max_tokens=tokens, top=min(alternatives, vocab))
        self.t = 0

    def table(self):
        return self.zero.p16[: self.vocab * self.width].view(self.vocab, self.width)

    def matrix(self):
        return self.muon.views(self.muon.p16)[0]

    def table_grad(self, rank):
        return self.zero.grads[rank][: self.vocab * self.width].view(self.vocab, self.width)

    def hidden(self, words):
        embedded = self.embedding.forward(words, self.table())
        return embedded, embedded @ self.matrix()

    def answer(self, words, gen):
        """One of the likeliest alternatives of each word, as likely as they are among themselves."""
        _, hidden = self.hidden(words)
        top_logp, top_ids = self.head.logprobs(hidden, self.table(), words)[3:]
        pick = torch.multinomial(top_logp.exp(), 1, generator=gen)
        return top_ids.gather(1, pick)[:, 0].long()

    def backward(self, rank, words, answers, advantages):
        """The rank's mean entropy; the gradients of its mean objective are left in the rank's vectors."""
        table, matrix = self.table(), self.matrix()
        embedded, hidden = self.hidden(words)
        logp, entropy, lse = self.head.logprobs(hidden, table, answers)[:3]
        grad = self.table_grad(rank)
        bonus = torch.full_like(entropy, -BONUS / self.tokens)
        dhidden, _ = self.head.grad(hidden, table, answers, lse, advantages * (-1 / self.tokens), entropy, bonus, dtable=grad)
        self.matrix_grads[rank][0].copy_(embedded.T @ dhidden)
        self.embedding.grad(words, dhidden @ matrix.T, grad, accumulate=True)
        return entropy.mean()

    def step(self, batches, max_norm=1.0):
        """One training step over the ranks' (words, answers, advantages); returns their mean entropies."""
        entropies = [self.backward(r, *batch) for r, batch in enumerate(batches)]
        self.t += 1
        self.zero.step(self.zero.grads, LR, BETA1, BETA2, EPS, self.t, max_norm=max_norm)
        self.muon.step(self.matrix_grads, LR_MATRIX, MU)
        return torch.stack(entropies)

    def status(self):
        self.head.status()
        self.muon.status()


def rewards(words, answers):
    return ((words ^ answers) & 1 == 0).float()


def rollout(model, gen):
    """A rank's words, its answers to them, and how much better than the mean each one was."""
    words = torch.randint(0, model.vocab, (model.tokens,), device="cuda", generator=gen)
    answers = model.answer(words, gen)
    r = rewards(words, answers)
    return words, answers, r - r.mean()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--vocab", type=int, default=512)
    ap.add_argument("--width", type=int, default=192)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args(argv)
    model = PolicyLm(a.vocab, a.width, a.tokens, a.ranks)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for k in range(a.steps):
        batches = [rollout(model, gen) for _ in range(a.ranks)]
        reward = torch.stack([rewards(w, x).mean() for w, x, _ in batches]).mean()
        entropies = model.step(batches)
        if k % 10 == 0 or k == a.steps - 1:
            print(f"step {k + 1:4d}  reward {reward.item():.3f}  entropy {entropies.mean().item():.3f}")
    model.status()
    return reward.item()


if __name__ == "__main__":
    main()
