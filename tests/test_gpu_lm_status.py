"""How the cross entropy reports a device wait that gave up: to the owner whose
call it was, in its results, and in the call that was asked to lose a copy."""

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs

pytestmark = pytest.mark.gpu

N, V, D = 400, 3000, 640


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def make(tokens=N, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(tokens, D, device="cuda", generator=gen).bfloat16()
    t = (torch.randn(V, D, device="cuda", generator=gen) * 0.1).bfloat16()
    tg = torch.randint(0, V, (tokens,), device="cuda", generator=gen)
    tg[::7] = -100
    return h, t, tg


@pytest.mark.parametrize("first", ["refused", "empty", "empty gradient"])
def test_an_injected_stall_is_spent_by_the_next_call(first):
    h, t, tg = make()
    op = zs.LmLoss(V, D, "bf16", max_tokens=N)
    loss, lse = op.loss(h, t, tg)
    op.status()
    zs.zero_lm_inject_stall()
    if first == "refused":
        with pytest.raises(zs.ZeroError):
            zs.zero_lm_loss(N, V, D, zs.ZERO_BF16, h, D, t, D, tg, 8, loss, lse, op.workspace, 64)
    elif first == "empty":
        op.loss(h[:0], t, tg[:0])
    else:
        op.grad(h[:0], t, tg[:0], lse[:0], 1.0)
    again = op.loss(h, t, tg)
    op.status()
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
