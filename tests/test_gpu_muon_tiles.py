"""Matrices beyond what a cluster's shared memory takes (a smaller side above 128, or a larger one above 2048):
lists of many shapes, places, values that are not finite, recurrences and ranks through the kernels over tiles."""

import math

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests import muon_reference as ref
from tests.test_gpu_muon import DT, check, check_step, few_directions, gaussian, make_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def many_shapes(count):
    """So many shapes, wide, square and (as another one's transpose, which is no shape of its own) tall."""
    shapes = [(129 + 8 * k + k % 3, 131 + 21 * k) for k in range(count)]
    return shapes + [(c, r) for r, c in shapes[::2]] + shapes[1::3]


@pytest.mark.parametrize("count", [3, 4, 5, 12, 13, 25])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_lists_of_many_shapes(count, dtype):
    """Up to and beyond what one launch takes, with small ones between."""
    shapes = many_shapes(count) + [(40, 72), (100, 1000)]
    check([gaussian(r, c, seed=i) for i, (r, c) in enumerate(shapes)], dtype, what=f"{count} shapes")


@pytest.mark.parametrize("count", [4, 13])
@pytest.mark.parametrize("W", [2, 4])
def test_steps_of_many_shapes(count, W):
    shapes = many_shapes(count)
    op, grads = make_step(shapes, W, "bf16", scales=[0.2 * math.sqrt(max(s)) for s in shapes])
    check_step(op, grads, 0.02, 0.95, True, 0.1, f"{count} shapes")
    check_step(op, grads, 0.02, 0.9, False, 0.0, f"{count} shapes")


def test_wide_and_square_shapes_in_one_launch():
    """Steps by twos beside steps one by one, whose lists have other lengths."""
    shapes = [(130, 300), (200, 210), (150, 2100), (256, 256), (2100, 150)]
    for dtype in ("bf16", "fp32"):
        check([few_directions(r, c, seed=i) for i, (r, c) in enumerate(shapes)], dtype, what="mixed")


@pytest.mark.parametrize("cols,offset", [(192, 0), (192, 1), (189, 0), (189, 3)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_strides_and_places(dtype, cols, offset):
    for rows in (135, 400):          # as they are, and turned
        wide = torch.full((rows, cols + 16), 5.0, device="cuda", dtype=DT[dtype])
        x = gaussian(rows, cols).to(DT[dtype])
        wide[:, offset:offset + cols] = x
        out = torch.full((rows, cols + 32), 3.0, device="cuda", dtype=DT[dtype])
        op = zs.Orthogonalize([(rows, cols)], dtype)
        plain = op.forward([x])[0]
        got = op.forward([wide[:, offset:offset + cols]], out=[out[:, offset:offset + cols]])[0]
        assert torch.equal(got, plain)
        assert (out[:, :offset] == 3).all() and (out[:, offset + cols:] == 3).all()
        view = wide[:, offset:offset + cols]
        op.forward([view], out=[view])          # in place
        assert torch.equal(view, plain)
        assert (wide[:, offset + cols:] == 5).all() and (wide[:, :offset] == 5).all()


@pytest.mark.parametrize("shape", [(200, 300), (300, 200), (150, 700)])
def test_zero_and_values_that_are_not_finite(shape):
    op = zs.Orthogonalize([shape] * 5, "bf16")
    xs = [gaussian(*shape, seed=k).bfloat16() for k in range(5)]
    clean = op.forward(xs)
    xs[1].zero_()
    xs[2][3, 4] = float("inf")
    xs[3][-1, -1] = float("nan")
    out = op.forward(xs)
    assert torch.equal(out[0], clean[0]) and torch.equal(out[4], clean[4]) and not out[1].any()
    assert torch.isnan(out[2]).all() and torch.isnan(out[3]).all()


@pytest.mark.parametrize("W", [1, 2, 4])
def test_an_overflow_leaves_its_matrix_alone(W):
    op, grads = make_step([(200, 304), (304, 200), (150, 331), (140, 140)], W, "fp16")
    grads[W - 1][1][5, 6] = float("inf")
    grads[0][2][149, 330] = float("nan")
    before = [[x.clone() for x in op.views(v)] for v in (op.master, op.momentum, op.p16)]
    op.step(grads, 0.02, weight_decay=0.1)
    op.status()
    for old, now in zip(before, (op.master, op.momentum, op.p16)):
        now = op.views(now)
        assert torch.equal(old[1], now[1]) and torch.equal(old[2], now[2])
        for k in (0, 3):
            assert not torch.equal(old[k], now[k]) and torch.isfinite(now[k]).all()
    for g in op.views(op.momentum) + [x for rank in grads for x in rank]:
        g.zero_()
    theta = [x.clone() for x in op.views(op.master)]
    op.step(grads, 0.02, weight_decay=0.5)
    for old, now in zip(theta, op.views(op.master)):
        assert torch.equal(now, old * torch.tensor(1 - 0.02 * 0.5, dtype=torch.float32, device="cuda"))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_four_ranks(dtype):
    shapes = [(200, 304), (304, 200), (150, 331), (136, 1000)]
    op, grads = make_step(shapes, 4, dtype, scales=[0.2 * math.sqrt(max(s)) for s in shapes])
    check_step(op, grads, 0.02, 0.95, True, 0.1, "nesterov")
    check_step(op, grads, 0.02, 0.9, False, 0.0, "heavy ball")
    check_step(op, grads, 0.05, 0.0, True, 0.0, "no momentum")


@pytest.mark.parametrize("W", [1, 3, 4])
def test_gradients_in_any_place(W):
    """Gradients that start anywhere give what aligned ones give."""
    shapes = [(140, 264), (264, 136)]
    op, grads = make_step(shapes, W, "bf16")
    other, _ = make_step(shapes, W, "bf16")
    moved = []
    for rank in grads:
        buf = torch.zeros(sum(g.numel() for g in rank) + 8, dtype=torch.bfloat16, device="cuda")
        views, at = [], 3
        for g in rank:
            views.append(buf[at:at + g.numel()].view(g.shape))
            views[-1].copy_(g)
            at += g.numel() + 1
        moved.append(views)
    for _ in range(2):
        op.step(grads, 0.02)
        other.step(moved, 0.02)
    assert torch.equal(op.master, other.master) and torch.equal(op.momentum, other.momentum)


def test_lists_that_take_several_tables():
    check([gaussian(129, 130, seed=i) for i in range(300)], "fp16")
    op, grads = make_step([(129, 130)] * 120, 8, "bf16")
    check_step(op, grads, 0.02, 0.95, True, 0.1)


TWO_DIFFERENT = ((4.0, -6.0, 3.0), (3.0, -3.0, 1.0), (3.2, -4.1, 1.7), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0))
# |a| of the first two multiply to more than 64; singular values stay below 3.5 (from a scan of both polynomials)
LARGE_A = ((9.0, -24.0, 17.0), (7.2, -5.0, 0.72), (1.0, 0.0, 0.0))


@pytest.mark.parametrize("rows,cols", [(150, 200), (140, 400), (600, 140)])
def test_other_recurrences(rows, cols):
    """Matrices whose steps go one by one, and by twos: steps that differ, splits of the parts that are odd, a
    product of two a that does not fit."""
    xs = [gaussian(rows, cols), few_directions(rows, cols, seed=1)]
    for dtype in ("bf16", "fp32"):
        check(xs, dtype, coefficients=((1.5, -0.5, 0.0),) * 8, what="cubic")
        for fine in (None, 0, 1, 2, 3, 4):
            check(xs, dtype, fine=fine, coefficients=TWO_DIFFERENT, what=f"different, {fine} fine")
        check(xs, dtype, fine=3, coefficients=LARGE_A, what="large a")
    check(xs, "fp16", coefficients=((2.0, -1.5, 0.5),), what="one step")
    check(xs, "bf16", coefficients=((2.0, -1.5, 0.5),) * 2, fine=1, what="two steps, one fine")
    check(xs, "fp32", coefficients=((1.5, -0.5, 0.0),) * 32, what="as many as there may be")
