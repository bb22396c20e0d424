"""How far the default and the other numbers of fine steps are off for many kinds of spectra, held to the figures
that zero_step.h states."""

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests import muon_reference as ref
from tests.test_gpu_muon import DT, gaussian

pytestmark = pytest.mark.gpu

# zero_step.h: the difference's Frobenius norm over the result's with 0 to 5 of five steps in two parts, for any
# spectrum here but a matrix of rank one, and for that.  The recurrence in 64 bits with the kernels' roundings put in
# (one by one and by twos, sums cut to 24 bits after every 16 products) gives, for these sizes on a CPU, at most
# 4.3e-2, 2.8e-2, 7.1e-3, 3.9e-3, 9.3e-4, 5.2e-5 and 1.5e-1, 3.2e-2, 1.4e-2, 3.9e-3, 1.5e-3, 8.2e-5.  Here are 1.25
# times that for the rounded operands, another draw of the same size.  With all steps in two parts the sums' cuts are
# what is left.  All go one way, so that they grow with the sums' length L: 5.2e-5 is of L = 384 and 1.4e-7 L, 8.2e-5
# of it 2.1e-7 L, and a cut may come a bit earlier when 16 products of different sizes are added, which is up to twice
# as much.
STATED = (5e-2, 4e-2, 9e-3, 5e-3, 1.2e-3, 3e-7)
RANK_ONE = (2e-1, 4e-2, 1.8e-2, 5e-3, 2e-3, 4.5e-7)
GAUSSIAN = (1.6e-3, 1.6e-3, 1.6e-3, 1e-3, 6e-4, 8e-8)
# fp32 results' sums are cut within 64 products alone, 3e-7, 4.5e-7 and 8e-8 times 64; beside it come operands of 22
# bits, which leave twice what fp32's 24 do (a plain fp32 form is up to 2e-5, 8e-5 and 2.5e-6 off).
FP32 = {"rank one": 2e-4, "gaussian": 1e-5}


def stated(name, fine, rows, cols, dtype=None):
    if fine == 5 and dtype == "fp32":
        return FP32.get(name, 6e-5)
    row = {"rank one": RANK_ONE, "gaussian": GAUSSIAN}.get(name, STATED)
    return row[fine] * (max(rows, cols) if fine == 5 else 1)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def spectrum(rows, cols, s):
    q = [torch.linalg.qr(gaussian(n, len(s), seed=k).double())[0] for k, n in enumerate((rows, cols))]
    return (q[0] * s) @ q[1].T


def kinds(rows, cols):
    k = torch.arange(1, min(rows, cols) + 1, device="cuda", dtype=torch.float64)
    yield "gaussian", gaussian(rows, cols)
    yield "8 of 20", 0.05 * gaussian(rows, cols) + gaussian(rows, 8, 1) @ gaussian(8, cols, 2)
    yield "k^-1", spectrum(rows, cols, 1 / k)
    yield "k^-1.5", spectrum(rows, cols, k ** -1.5)
    yield "k^-2", spectrum(rows, cols, k ** -2)
    yield "exp(-k/20)", spectrum(rows, cols, torch.exp(-k / 20))
    for many, far in ((8, 1e-3), (8, 1e-4), (1, 1e-3), (len(k) // 2, 1e-2)):
        yield f"{many} of 1 above {far}", spectrum(rows, cols, torch.where(k <= many, 1.0, far))
    yield "rank one", spectrum(rows, cols, torch.where(k <= 1, 1.0, 0.0))


def off(got, want):
    return float(torch.linalg.vector_norm(got.double() - want) / torch.linalg.vector_norm(want))


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(128, 256), (100, 1500), (256, 512), (384, 384), (520, 264), (768, 768)])
def test_fine_steps(rows, cols, dtype):
    names, xs = zip(*kinds(rows, cols))
    xs = [(x / x.abs().max()).to(DT[dtype]) for x in xs]
    for fine in (0, 1, 2, 3, 4, 5, None):
        op = zs.Orthogonalize([(rows, cols)] * len(xs), dtype, fine_steps=fine)
        for name, x, got in zip(names, xs, op.forward(xs)):
            want = ref.orthogonal(x)
            own = off(want.to(DT[dtype]), want)          # the result's own rounding
            used = fine if fine is not None else 4 if dtype == "bf16" else 5
            assert off(got, want) <= stated(name, used, rows, cols, dtype) + 1.1 * own, (name, fine)
            if fine is None and dtype != "fp32":
                # by default the steps leave less than the result's own rounding: sqrt(1 + 1) of it together
                assert off(got, want) <= 1.42 * own, name
        op.status()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_the_steps_update(dtype):
    """The step writes an fp32 master: by default its direction is as exact as an fp32 result."""
    for rows, cols in ((100, 200), (256, 512), (384, 384)):
        names, xs = zip(*kinds(rows, cols))
        op = zs.MuonStep([(rows, cols)] * len(xs), 1, dtype)
        for m, x in zip(op.views(op.momentum), xs):
            m.copy_(x / x.abs().max())
        grads = op.new_grad_buffers()
        u = [m.double() * 0.5 for m in op.views(op.momentum)]
        op.step(grads, 1.0, 0.5, nesterov=False)       # of a master of 0: its new value is the direction
        op.status()
        for name, x, theta in zip(names, u, op.views(op.master)):
            assert off(-theta, ref.orthogonal(x)) <= stated(name, 5, rows, cols), name


@pytest.mark.parametrize("rows,cols", [(100, 900), (200, 300), (430, 1321), (1024, 2048), (2300, 700)])
def test_fp32_results_do_not_lose_with_the_size(rows, cols):
    """Long sums of one sign, whose cuts would add up: gradients with directions that many tokens share."""
    x = gaussian(rows, cols) + (gaussian(rows, 32, 1) * 0.3) @ gaussian(32, cols, 2) / 32 ** 0.5
    got = zs.Orthogonalize([(rows, cols)], "fp32").forward([x])[0]
    assert off(got, ref.orthogonal(x)) <= FP32["gaussian"]


@pytest.mark.parametrize("fine", [1, 2, 3, 4])
def test_steps_in_two_parts_beside_others(fine):
    """fp32 results with steps of both kinds: tiles of both follow one another through the same accumulators."""
    shapes = [(768, 768)] * 11 + [(300, 900)] * 7 + [(520, 264)] * 5
    xs = [gaussian(*s, seed=k) for k, s in enumerate(shapes)]
    op = zs.Orthogonalize(shapes, "fp32", fine_steps=fine)
    want = [ref.orthogonal(x) for x in xs]
    for _ in range(3):
        for k, got in enumerate(op.forward(xs)):
            assert off(got, want[k]) <= GAUSSIAN[fine], (fine, k)
    op.status()
