"""fp32 results after a lost block of operands: their tiles' sums go through several accumulators."""

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests.test_gpu_muon import gaussian

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("fine", [0, 3, 5])
@pytest.mark.parametrize("shapes", [[(300, 300), (200, 600)], [(1100, 700)], [(64, 600)]])
def test_a_wait_that_runs_out(shapes, fine):
    xs = [gaussian(*s) for s in shapes]
    op = zs.Orthogonalize(shapes, "fp32", fine_steps=fine)
    good = op.forward(xs)
    op.status()
    zs.zero_lm_inject_stall()
    bad = op.forward(xs)
    with pytest.raises(zs.ZeroError) as e:
        op.status()
    assert e.value.code == zs.ZERO_E_STATE
    with pytest.raises(zs.ZeroError):
        zs.zero_lm_status()
    assert all(torch.isnan(x).all() for x in bad)
    assert all(torch.equal(x, y) for x, y in zip(good, op.forward(xs)))
    op.status()


def test_small_matrices_beside_a_lost_one():
    """What the others hold is right or no number."""
    shapes = [(64, 700), (30, 20), (128, 256), (100, 2000)]
    xs = [gaussian(*s) for s in shapes]
    op = zs.Orthogonalize(shapes, "bf16")
    ys = [x.bfloat16() for x in xs]
    good = op.forward(ys)
    zs.zero_lm_inject_stall()
    bad = op.forward(ys)
    with pytest.raises(zs.ZeroError):
        op.status()
    with pytest.raises(zs.ZeroError):
        zs.zero_lm_status()
    lost = [bool(torch.isnan(x).all()) for x in bad]
    assert any(lost) and all(a or torch.equal(x, y) for a, x, y in zip(lost, good, bad))
    assert all(torch.equal(x, y) for x, y in zip(good, op.forward(ys)))
