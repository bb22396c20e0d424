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


def failed(op):
    with pytest.raises(zs.ZeroError) as e:
        op.status()
    return e.value.code == zs.ZERO_E_STATE


@pytest.mark.parametrize("which", ["loss", "grad"])
def test_an_owner_learns_of_its_own_failures_only(which):
    h, t, tg = make()
    a, b = (zs.LmLoss(V, D, "bf16", max_tokens=N) for _ in range(2))
    lse = a.loss(h, t, tg)[1]
    a.status()
    zs.zero_lm_inject_stall()
    if which == "loss":
        a.loss(h, t, tg)
    else:
        a.grad(h, t, tg, lse, 1.0)
    b.loss(h, t, tg)
    b.status()                        # not b's failure, and not b's to report
    assert failed(a)
    a.status(), b.status()


def test_the_device_count_is_reported_once_beside_the_owners():
    h, t, tg = make()
    op = zs.LmLoss(V, D, "bf16", max_tokens=N)
    try:
        zs.zero_lm_status()           # what other tests left
    except zs.ZeroError:
        pass
    zs.zero_lm_inject_stall()
    op.loss(h, t, tg)
    with pytest.raises(zs.ZeroError) as e:
        zs.zero_lm_status()
    assert e.value.code == zs.ZERO_E_STATE
    zs.zero_lm_status()
    assert failed(op)


@pytest.mark.parametrize("tokens", [N, 40])
def test_what_a_failed_loss_could_not_compute_is_nan(tokens):
    """Every loss is either the right one or a NaN: never what an earlier call left in the workspace."""
    h, t, tg = make(tokens)
    op = zs.LmLoss(V, D, "bf16", max_tokens=N)
    loss, lse = op.loss(h, t, tg)
    h2, t2, _ = make(tokens, seed=1)
    op.loss(h2, t2, tg)
    zs.zero_lm_inject_stall()
    got, got_lse = op.loss(h, t, tg)
    assert failed(op)
    assert torch.isnan(got_lse).any()
    for x, y in ((got, loss), (got_lse, lse)):
        assert ((x == y) | torch.isnan(x)).all()
    again = op.loss(h, t, tg)         # and nothing of it is left
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


@pytest.mark.parametrize("accumulate", [False, True])
def test_failed_gradients_are_nan(accumulate):
    h, t, tg = make()
    op = zs.LmLoss(V, D, "bf16", max_tokens=N)
    lse = op.loss(h, t, tg)[1]
    wide = torch.zeros(V, D + 8, dtype=torch.bfloat16, device="cuda")
    want = [x.clone() for x in op.grad(h, t, tg, lse, 1.0, dtable=wide[:, :D], accumulate=accumulate)]
    wide.zero_()
    zs.zero_lm_inject_stall()
    dh, dt = op.grad(h, t, tg, lse, 1.0, dtable=wide[:, :D], accumulate=accumulate)
    assert failed(op)
    assert torch.isnan(dh).all() and torch.isnan(dt).all() and (wide[:, D:] == 0).all()
    wide.zero_()
    again = op.grad(h, t, tg, lse, 1.0, dtable=wide[:, :D], accumulate=accumulate)
    op.status()
    assert all(torch.equal(x, y) for x, y in zip(again, want))


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
