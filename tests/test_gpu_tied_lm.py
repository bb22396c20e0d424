"""The operators together, as examples/tied_lm.py uses them."""

import math

import pytest
import torch

from examples import tied_lm
from tests import lm_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def test_one_step_against_64_bits():
    """Gradients of both ends in one vector, their norm, and the clipped update."""
    vocab, width, tokens, ranks = 1000, 72, 300, 3
    model = tied_lm.TiedLm(vocab, width, tokens, ranks)
    gen = torch.Generator(device="cuda").manual_seed(5)
    batches = [tied_lm.batch(vocab, tokens, gen) for _ in range(ranks)]
    table16 = model.table().clone()
    theta = model.zero.master.clone()
    losses = model.step(batches, max_norm=0.05)
    u = ref.HALF_ULP[torch.bfloat16]
    c = model.embedding.scale
    grads = []
    for r, (x, y) in enumerate(batches):
        E = table16.double().requires_grad_(True)
        # the hidden vectors as the lookup rounds them, the rounding passed through
        h = E[x] * c
        h = h + (h.float().to(torch.bfloat16).double() - h).detach()
        loss = torch.nn.functional.cross_entropy(h @ E.T, y)
        loss.backward()
        assert abs(losses[r].item() - loss.item()) <= 1e-4 * loss.item()
        got = model.table_grad(r)
        # D, dhidden, the head's gradient and the sum are each rounded once: errors of independent signs
        assert ref.rel_norm(got, E.grad) <= 3 * u, r
        grads.append(model.zero.grads[r].double())
    mean = sum(grads) / ranks
    norm = torch.linalg.vector_norm(mean)
    assert abs(model.zero.grad_norm.item() - norm.item()) <= 1e-5 * norm.item() and norm > 0.05
    g = mean * (0.05 / (norm + 1e-6))
    # the first Adam step moves by lr g / (|g| + eps sqrt(1 - beta2)...): in 64 bits
    m_hat, v_hat = g, g * g
    want = theta.double() - tied_lm.LR * m_hat / (v_hat.sqrt() + tied_lm.EPS)
    assert ((model.zero.master.double() - want).abs() <= 1e-5 * want.abs() + 1e-5 * tied_lm.LR).all()
    model.zero.close()


def test_training_learns_the_pairs():
    loss = tied_lm.main(["--vocab", "1024", "--width", "128", "--tokens", "1024", "--ranks", "2", "--steps", "150"])
    assert math.log(2) - 0.02 <= loss <= 1.2, loss
