"""Orthogonalisation of inputs of any size that fp32 holds: norms whose squares fp32 does not hold, and elements
that are far apart.  In shared memory, and through the kernels over tiles."""

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests import muon_reference as ref
from tests.test_gpu_muon import DT, check_step, few_directions, gaussian, make_step

pytestmark = pytest.mark.gpu

SHAPES = [(70, 90), (100, 700), (200, 300), (300, 140)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def away_from_zero(x):
    """Elements of at least 2^-4 and at most 2^5, so that 2^-120 times them are exact."""
    return torch.where(x < 0, -1.0, 1.0) * x.abs().clamp(2.0 ** -4, 2.0 ** 5)


def one_direction(rows, cols):
    return 1e-3 * gaussian(rows, cols) + gaussian(rows, 1, 1) @ gaussian(1, cols, 2)


def check(matrices, dtype, what):
    matrices = [x.to(DT[dtype]) for x in matrices]
    op = zs.Orthogonalize([tuple(x.shape) for x in matrices], dtype, fine_steps=5)
    out = op.forward(matrices)
    op.status()
    for x, got in zip(matrices, out):
        want = ref.orthogonal(x)
        tol = ref.tolerance(x, want, ref.COEFFICIENTS, 5, 2 if dtype == "fp32" else 1) + ref.HALF_ULP[DT[dtype]]
        ref.assert_near(got, want, tol, f"{what} {tuple(x.shape)} {dtype}")
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("e", [-120, -100, -80, -76, -72, -64, -46, -40, -20, 20, 54, 58, 64, 70, 90, 110, 120])
def test_the_inputs_size_does_not_matter(e, dtype):
    for kind in (gaussian, few_directions, one_direction):
        check([away_from_zero(kind(*s)) * 2.0 ** e for s in SHAPES], dtype, f"{kind.__name__} 2^{e}")


def test_far_from_one_the_bits_are_the_same():
    """A power of two changes no rounding."""
    xs = [away_from_zero(gaussian(*s)) for s in SHAPES]
    op = zs.Orthogonalize(SHAPES, "fp32")
    want = op.forward(xs)
    for e in (-120, -100, -60, 70, 100, 120):
        got = op.forward([x * 2.0 ** e for x in xs])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), e


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_elements_far_apart(dtype):
    """Blocks of elements whose squares vanish, fit and overflow in one matrix; the largest rule."""
    for sizes in ((1e-30, 1.0), (1e-25, 1e-22), (1.0, 1e25), (1e-30, 1e30), (1e19, 1e20), (1e-19, 1e-20, 1e-21)):
        xs = []
        for s in SHAPES:
            x = gaussian(*s)
            for k, size in enumerate(sizes):
                x[k::len(sizes)] *= size
            xs.append(x)
        check(xs, dtype, f"{sizes}")


def test_subnormal_elements():
    for s in SHAPES:
        x = (gaussian(*s) * 64).round() * 2.0 ** -149
        got = zs.Orthogonalize([s], "fp32").forward([x])[0]
        want = ref.orthogonal(x)
        ref.assert_near(got, want, ref.tolerance(x, want, ref.COEFFICIENTS, 5, 2), f"{s}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_largest_finite_elements(dtype):
    """A norm beyond fp32's range, of finite elements; and an infinity and a NaN beside them."""
    most = torch.finfo(DT[dtype]).max
    xs = [torch.where(gaussian(*s) < 0, -1.0, 1.0) * most for s in SHAPES]
    check(xs, dtype, "largest")
    for bad in (float("inf"), float("-inf"), float("nan")):
        for s, x in zip(SHAPES, xs):
            y = x.to(DT[dtype]).clone()
            y[s[0] - 1, s[1] - 1] = bad
            assert torch.isnan(zs.Orthogonalize([s], dtype).forward([y])[0]).all()


@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("size", [1e-37, 1e-30, 1e-23, 1e-20, 1e20, 1e30])
def test_a_momentum_that_fades_or_grows(size, W):
    """Gradients that stay 0 leave a momentum that shrinks step by step; the direction stays what it was."""
    op, grads = make_step(SHAPES, W, "bf16", unit=0.0)
    for m in op.views(op.momentum):
        m.copy_(away_from_zero(few_directions(*m.shape)) * size)
    check_step(op, grads, 0.02, 0.95, True, 0.1, f"momentum {size}")
    check_step(op, grads, 0.02, 0.9, False, 0.0, f"momentum {size}")
    assert torch.isfinite(op.master).all()


def test_a_momentum_that_fades_away():
    """From 1e-21 to nothing in steps of mu = 0.5: the master stays finite, and only decays at the end."""
    op, grads = make_step([(40, 60), (150, 200)], 3, "bf16", unit=0.0)
    for m in op.views(op.momentum):
        m.copy_(few_directions(*m.shape) * 1e-21)
    for _ in range(100):
        op.step(grads, 0.001, 0.5)
    op.status()
    assert torch.isfinite(op.master).all() and not op.momentum.any()
    theta = op.master.clone()
    op.step(grads, 0.001, 0.5)
    assert torch.equal(op.master, theta)
