"""Log probabilities of rows with a logit of +infinity."""

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests import lm_reference as ref
from tests.test_gpu_lm_logprobs import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("N", [1, 50, 96, 97, 200, 5000])
@pytest.mark.parametrize("word", [0, 255, 1500, 2999])
def test_a_logit_of_infinity(N, word):
    """The row is no number, its likeliest word is that one; the other rows are what they are without it."""
    h, t, tg = make(N, 3000, 64, "bf16", ignored=0.1, seed=word)
    t[:, 0] = 0.0
    t[word, 0] = float("inf")
    h[:, 0] = -1.0                       # -infinity for that word
    rows = torch.arange(N, device="cuda") % 7 == 0
    h[rows, 0] = 1.0
    op = zs.LmLogprobs(3000, 64, "bf16", max_tokens=N, top=5, with_grad=False)
    logp, entropy, lse, values, ids = op.logprobs(h, t, tg)
    op.status()
    valid = ref.valid_mask(tg, 3000)
    assert torch.isnan(lse[rows]).all() and torch.isnan(entropy[rows]).all() and torch.isnan(values[rows]).all()
    assert torch.isnan(logp[rows & valid]).all() and (logp[~valid] == 0).all()
    assert (ids[rows, 0] == word).all() and (ids[rows] >= 0).all()
    others = t.clone()
    others[word] = 0.0
    want = ref.logprobs_reference(h[~rows], others, tg[~rows])
    # that word adds nothing: of the 64-bit sums it is taken out
    z = h[~rows].double() @ others.double().T
    z[:, word] = float("-inf")
    lse64 = torch.logsumexp(z, 1)
    assert ((lse[~rows].double() - lse64).abs() <= want["lse_bound"] + 1e-6).all()
    assert torch.isfinite(entropy[~rows]).all() and (ids[~rows] != word).all()
