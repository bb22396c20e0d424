"""Log probabilities, their gradients and the orthogonalised step together, as examples/policy_lm.py uses them."""

import math

import pytest
import torch

from examples import policy_lm
from tests import lm_reference as lm
from tests import muon_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def test_one_step_against_64_bits():
    vocab, width, tokens, ranks = 600, 72, 300, 3
    model = policy_lm.PolicyLm(vocab, width, tokens, ranks)
    gen = torch.Generator(device="cuda").manual_seed(5)
    batches = [policy_lm.rollout(model, gen) for _ in range(ranks)]
    table16, matrix16 = model.table().clone(), model.matrix().clone()
    theta, master, momentum = model.zero.master.clone(), model.muon.master.clone(), model.muon.momentum.clone()
    entropies = model.step(batches, max_norm=1e9)
    model.status()
    u = lm.HALF_ULP[torch.bfloat16]
    c = model.embedding.scale

    def as_stored(x):
        # rounded as the model stores it, the rounding passed through
        return x + (x.float().to(torch.bfloat16).double() - x).detach()

    for r, (words, answers, advantages) in enumerate(batches):
        E, M = (x.double().requires_grad_(True) for x in (table16, matrix16))
        hidden = as_stored(as_stored(E[words] * c) @ M)
        logs = torch.log_softmax(hidden @ E.T, 1)
        entropy = -(logs.exp() * logs).sum(1)
        objective = -(advantages.double() * logs.gather(1, answers[:, None])[:, 0] + policy_lm.BONUS * entropy).mean()
        objective.backward()
        assert abs(entropies[r].item() - entropy.mean().item()) <= 1e-4 * entropy.mean().item()
        # the products' own rounding of D, dhidden, the embedding's rows and the sums, each once
        assert lm.rel_norm(model.table_grad(r), E.grad) <= 4 * u, r
        assert lm.rel_norm(model.matrix_grads[r][0], M.grad) <= 4 * u, r
    # the step of the matrix from the gradients as they lie there
    grads = [model.matrix_grads[r][0] for r in range(ranks)]
    m0, t0 = (model.muon.views(v)[0] for v in (momentum, master))
    want, m, direction = ref.step(grads, t0, m0, policy_lm.LR_MATRIX, policy_lm.MU, True, 0.0, 1.0)
    o = ref.orthogonal(direction)
    tol = ref.tolerance(direction, o, ref.COEFFICIENTS, 2, 2)
    got = model.muon.views(model.muon.master)[0]
    ref.assert_near((got.double() - t0.double()) / -policy_lm.LR_MATRIX, o,
                    tol + 3 * 2.0 ** -24 / policy_lm.LR_MATRIX * math.sqrt(width), "matrix")
    assert torch.equal(model.matrix(), got.to(torch.bfloat16))
    assert not torch.equal(model.zero.master, theta)
    model.zero.close()


def test_it_runs():
    reward = policy_lm.main(["--vocab", "256", "--width", "136", "--tokens", "500", "--ranks", "2", "--steps", "12"])
    assert 0.0 <= reward <= 1.0
