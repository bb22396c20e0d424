"""What log probabilities hold after a lost block of operands: nothing that looks like a result and is none."""

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


@pytest.mark.parametrize("top", [0, 4, 16])
@pytest.mark.parametrize("N", [1, 40, 96, 97, 300, 4000])
def test_a_row_is_right_or_no_number(N, top):
    V = 5000
    h, t, tg = make(N, V, 128, "bf16")
    op = zs.LmLogprobs(V, 128, "bf16", max_tokens=N, top=top, with_grad=False)
    good = op.logprobs(h, t, tg)
    op.status()
    zs.zero_lm_inject_stall()
    bad = op.logprobs(h, t, tg)
    with pytest.raises(zs.ZeroError):
        op.status()
    with pytest.raises(zs.ZeroError):
        zs.zero_lm_status()
    whole = torch.stack([(x == y).view(N, -1).all(1) for x, y in zip(good, bad)]).all(0)
    none = torch.isnan(bad[2])
    assert none.any() and (whole | none).all()
    assert torch.isnan(bad[1][none]).all()
    valid = ref.valid_mask(tg, V)
    assert torch.isnan(bad[0][none & valid]).all() and (bad[0][~valid] == 0).all()
    if top:
        assert bad[4].dtype == torch.int32 and torch.isnan(bad[3][none]).all()
        assert (bad[4] >= -1).all() and (bad[4] < V).all()
    assert all(torch.equal(x, y) for x, y in zip(good, op.logprobs(h, t, tg)))
    op.status()
