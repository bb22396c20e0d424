"""Newton-Schulz orthogonalisation and the step built on it, against plain
64-bit forms; the tolerances come from the recurrence with the kernels'
roundings put in (tests/muon_reference.py)."""

import math

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests import muon_reference as ref

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def gaussian(rows, cols, seed=0, unit=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 7 * rows + cols)
    return torch.randn(rows, cols, device="cuda", generator=gen) * unit


def few_directions(rows, cols, seed=0):
    """Few singular values far above the rest."""
    return 0.05 * gaussian(rows, cols, seed) + gaussian(rows, 8, seed + 1) @ gaussian(8, cols, seed + 2)


def check(matrices, dtype, fine=None, coefficients=ref.COEFFICIENTS, op=None, what=""):
    matrices = [x.to(DT[dtype]) for x in matrices]
    op = op or zs.Orthogonalize([tuple(x.shape) for x in matrices], dtype, coefficients=coefficients, fine_steps=fine)
    out = op.forward(matrices)
    op.status()
    steps = len(coefficients)
    used = fine if fine is not None else steps if dtype == "fp32" else max(0, steps - 3)
    for k, (x, got) in enumerate(zip(matrices, out)):
        want = ref.orthogonal(x, coefficients)
        tol = ref.tolerance(x, want, coefficients, used, 2 if dtype == "fp32" else 1) + ref.HALF_ULP[DT[dtype]]
        ref.assert_near(got, want, tol, f"{what} {k}: {tuple(x.shape)} {dtype}")
    return out


SHAPES = [(1, 1), (1, 2), (3, 1), (7, 5), (8, 8), (20, 64), (64, 64), (65, 63), (100, 300), (128, 257), (256, 256),
          (257, 256), (300, 520), (768, 200), (513, 1030)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_orthogonalize(rows, cols, dtype):
    check([gaussian(rows, cols)], dtype, what="gaussian")
    check([gaussian(cols, rows), few_directions(cols, rows)], dtype, what="few directions")


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(128, 256), (128, 272), (2048, 128), (64, 2048), (128, 1025), (1999, 17), (5, 700), (2049, 16), (129, 130)])
def test_around_what_one_cluster_takes(rows, cols, dtype):
    check([gaussian(rows, cols)], dtype, what="gaussian")
    check([few_directions(rows, cols)], dtype, what="few directions")


def test_mixed_sizes_in_one_call():
    """Matrices of one CTA, of clusters and beyond in one call, few of each and many."""
    shapes = [(30, 20), (128, 700), (300, 300), (9, 1500), (64, 64), (260, 140), (700, 128), (1, 1)]
    matrices = [gaussian(r, c, seed=i) for i, (r, c) in enumerate(shapes)]
    whole = check(matrices, "bf16")
    many = check(matrices * 20, "bf16")
    for i, (x, got) in enumerate(zip(matrices, whole)):
        # how many CTAs share a matrix goes by the call's other matrices, where SMs are left
        want = ref.orthogonal(x.bfloat16())
        tol = ref.tolerance(x.bfloat16(), want, ref.COEFFICIENTS, 2, 1) + ref.HALF_ULP[torch.bfloat16]
        ref.assert_near(got, want, tol, f"{i}")
        ref.assert_near(many[i + 8 * 13], want, tol, f"{i} of many")


@pytest.mark.parametrize("fine", [0, 1, 3, 5])
def test_fine_steps(fine):
    for dtype in ("bf16", "fp32"):
        check([gaussian(200, 333), few_directions(200, 333)], dtype, fine=fine, what=f"fine {fine}")


def test_singular_values_come_near_one():
    x = check([few_directions(300, 400)], "bf16")[0]
    s = torch.linalg.svdvals(x.double())
    assert 0.6 <= s[:8].min() and s.max() <= 1.3


def test_other_coefficients_and_counts():
    """Eight steps of the classical cubic, which converge to 1; steps of their own each; one step."""
    cubic = ((1.5, -0.5, 0.0),) * 8
    x = gaussian(64, 64)
    q = (torch.linalg.qr(x)[0] * torch.linspace(0.5, 1.0, 64, device="cuda")).contiguous()     # well conditioned
    check([q, x], "fp32", coefficients=cubic)
    check([x, gaussian(100, 40)], "bf16", coefficients=((4.0, -6.0, 3.0), (3.0, -3.0, 1.0), (1.875, -1.25, 0.375)))
    check([x], "fp16", coefficients=((2.0, -1.5, 0.5),))


def test_many_matrices_of_many_shapes():
    """More shapes than a launch takes, several of each, both ways round, in one call."""
    shapes = [(8 * k + r, 5 * k + 3) for k in range(1, 8) for r in (0, 3)] + [(40, 72), (72, 40), (72, 40), (40, 72)]
    matrices = [gaussian(r, c, seed=i) for i, (r, c) in enumerate(shapes)]
    whole = check(matrices, "bf16")
    # and each alone gives the same bits: nothing depends on its neighbours
    for x, got in list(zip(matrices, whole))[-5:]:
        alone = zs.Orthogonalize([tuple(x.shape)], "bf16").forward([x.bfloat16()])[0]
        assert torch.equal(alone, got)


def test_a_list_that_takes_several_tables():
    matrices = [gaussian(9, 17, seed=i) for i in range(400)]
    check(matrices, "fp16")


def test_sizes_of_the_input_do_not_matter():
    """Tiny and huge inputs: the result is that of the direction alone."""
    x = gaussian(70, 90)
    base = zs.Orthogonalize([(70, 90)], "fp32").forward([x])[0]
    for e in (-50, -10, 10, 55):
        assert torch.equal(zs.Orthogonalize([(70, 90)], "fp32").forward([x * 2.0 ** e])[0], base)


def test_zero_and_values_that_are_not_finite():
    op = zs.Orthogonalize([(70, 90)] * 4, "bf16")
    xs = [gaussian(70, 90, seed=k).bfloat16() for k in range(4)]
    clean = op.forward(xs)
    xs[1].zero_()
    xs[2][3, 4] = float("inf")
    xs[3][69, 89] = float("nan")
    out = op.forward(xs)
    assert torch.equal(out[0], clean[0]) and not out[1].any()
    assert torch.isnan(out[2]).all() and torch.isnan(out[3]).all()


@pytest.mark.parametrize("cols,offset", [(64, 0), (64, 1), (61, 0), (61, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides_and_places(dtype, cols, offset):
    for rows in (40, 130):
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
        assert torch.equal(view, plain) and (wide[:, offset + cols:] == 5).all()


def test_no_matrices():
    assert zs.Orthogonalize([], "bf16").forward([]) == []
    zs.MuonStep([], 2, "bf16").step([[], []], 0.1)


def make_step(shapes, W, dtype, seed=0, unit=1e-3, scales=None, **kw):
    theta = [gaussian(r, c, seed + 11, 0.02) for r, c in shapes]
    op = zs.MuonStep(shapes, W, dtype, theta0=theta, scales=scales, **kw)
    for k, m in enumerate(op.views(op.momentum)):
        m.copy_(gaussian(*m.shape, seed + 13, 3 * unit))
    grads = op.new_grad_buffers()
    for w, rank in enumerate(grads):
        for k, g in enumerate(rank):
            g.copy_(gaussian(*g.shape, seed + 17 * w + k, unit))
    return op, grads


def check_step(op, grads, lr, mu, nesterov, decay, what=""):
    before = [[x.clone() for x in op.views(v)] for v in (op.master, op.momentum)]
    op.step(grads, lr, mu, weight_decay=decay, nesterov=nesterov)
    op.status()
    steps = op.steps
    fine = op.fine_steps if op.fine_steps >= 0 else max(0, steps - 3)
    W = len(grads)
    for i, (theta0, m0) in enumerate(zip(*before)):
        scale = op.scales[i] if op.scales else 1.0
        theta, m, u = ref.step([rank[i] for rank in grads], theta0, m0, lr, mu, nesterov, decay, scale)
        got_m, got = op.views(op.momentum)[i], op.views(op.master)[i]
        # the mean's W roundings and the momentum's one, each 2^-24 of what is added
        size = sum(rank[i].double().abs() for rank in grads) / W + mu * m0.double().abs()
        assert ((got_m.double() - m).abs() <= (W + 3) * 2.0 ** -24 * size + 1e-37).all(), what
        o = ref.orthogonal(u)
        tol = ref.tolerance(u, o, ref.COEFFICIENTS, fine, 2)
        # the update's error, and theta's roundings
        ref.assert_near((got.double() - theta0.double() * (1 - lr * decay)) / (-lr * scale), o,
                        tol + float(theta0.double().abs().max()) * 3 * 2.0 ** -24 / (lr * scale) * o.numel() ** 0.5
                        / max(float(torch.linalg.vector_norm(o)), 1e-30), f"{what} matrix {i}")
        assert torch.equal(op.views(op.p16)[i], got.to(op.p16.dtype))
    used = torch.zeros(op.n, dtype=torch.bool, device="cuda")
    for v in op.views(used):
        v.fill_(True)
    for v in (op.master, op.momentum, op.p16):
        assert not v[~used].any()          # the padding between the matrices


STEP_SHAPES = [[(1, 1), (5, 3)], [(64, 96), (96, 64), (64, 64)], [(100, 37), (33, 130), (7, 7)], [(300, 200), (256, 512)],
               [(301, 203), (203, 301), (150, 1001)], [(520, 264), (30, 9), (131, 700)]]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("W", [1, 2, 3, 8, 11])
@pytest.mark.parametrize("shapes", STEP_SHAPES)
def test_step(shapes, W, dtype):
    op, grads = make_step(shapes, W, dtype, scales=[0.2 * math.sqrt(max(s)) for s in shapes])
    check_step(op, grads, 0.02, 0.95, True, 0.1, "nesterov")
    check_step(op, grads, 0.02, 0.9, False, 0.0, "heavy ball")
    check_step(op, grads, 0.05, 0.0, True, 0.0, "no momentum")


def test_mixed_formats_and_default_scales():
    op, grads = make_step([(64, 96), (33, 17)], 4, "fp16", work_dtype="bf16")
    assert op.p16.dtype == torch.bfloat16
    check_step(op, grads, 0.02, 0.95, True, 0.1)


def test_gradients_in_any_place():
    """Gradients that start anywhere give what aligned ones give."""
    shapes = [(40, 64), (64, 24)]
    op, grads = make_step(shapes, 3, "bf16")
    other, _ = make_step(shapes, 3, "bf16")
    moved = []
    for rank in grads:
        buf = torch.zeros(sum(g.numel() for g in rank) + 8, dtype=torch.bfloat16, device="cuda")
        views, at = [], 3
        for g in rank:
            views.append(buf[at:at + g.numel()].view(g.shape))
            views[-1].copy_(g)
            at += g.numel() + 1
        moved.append(views)
    op.step(grads, 0.02)
    other.step(moved, 0.02)
    assert torch.equal(op.master, other.master) and torch.equal(op.momentum, other.momentum)


def test_an_overflow_leaves_its_matrix_alone():
    op, grads = make_step([(40, 64), (64, 24), (30, 30)], 4, "fp16")
    grads[2][1][5, 6] = float("inf")
    grads[0][2][0, 0] = float("nan")
    before = [[x.clone() for x in op.views(v)] for v in (op.master, op.momentum, op.p16)]
    op.step(grads, 0.02, weight_decay=0.1)
    for old, now in zip(before, (op.master, op.momentum, op.p16)):
        now = op.views(now)
        assert torch.equal(old[1], now[1]) and torch.equal(old[2], now[2])
        assert not torch.equal(old[0], now[0]) and torch.isfinite(now[0]).all()
    for g in op.views(op.momentum) + [x for rank in grads for x in rank]:
        g.zero_()
    theta = [x.clone() for x in op.views(op.master)]
    op.step(grads, 0.02, weight_decay=0.5)
    for old, now in zip(theta, op.views(op.master)):
        assert torch.equal(now, old * torch.tensor(1 - 0.02 * 0.5, dtype=torch.float32, device="cuda"))


@pytest.mark.parametrize("what", ["orthogonalize", "step"])
def test_the_same_bits_every_time_and_in_a_graph(what):
    shapes = [(200, 300), (64, 64), (300, 40)]
    if what == "orthogonalize":
        op = zs.Orthogonalize(shapes, "bf16")
        xs = [gaussian(*s).bfloat16() for s in shapes]

        def once():
            return op.forward(xs)

        first = once()
        for _ in range(3):
            assert all(torch.equal(x, y) for x, y in zip(first, once()))
    else:
        op, grads = make_step(shapes, 3, "bf16")
        twin, _ = make_step(shapes, 3, "bf16")

        def once():
            op.step(grads, 0.02)

        once()
        twin.step(grads, 0.02)
        assert torch.equal(op.master, twin.master) and torch.equal(op.p16, twin.p16)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        once()
    if what == "step":
        twin.step(grads, 0.02)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = once()
    if what == "orthogonalize":
        for x in xs:
            x.mul_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, once()))
        return
    for _ in range(2):
        graph.replay()
        twin.step(grads, 0.02)
    torch.cuda.synchronize()
    assert torch.equal(op.master, twin.master) and torch.equal(op.momentum, twin.momentum)


@pytest.mark.parametrize("shapes", [[(300, 300), (200, 600)], [(64, 600)], [(64, 64)]])
def test_a_wait_that_runs_out_is_reported(shapes):
    xs = [gaussian(*s).bfloat16() for s in shapes]
    op, other = zs.Orthogonalize(shapes, "bf16"), zs.Orthogonalize(shapes, "bf16")
    good = op.forward(xs)
    op.status()
    zs.zero_lm_inject_stall()
    bad = op.forward(xs)
    other.forward(xs)
    other.status()
    assert all(torch.isnan(x).all() for x in bad)
    with pytest.raises(zs.ZeroError) as e:
        op.status()
    assert e.value.code == zs.ZERO_E_STATE
    with pytest.raises(zs.ZeroError):
        zs.zero_lm_status()
    assert all(torch.equal(x, y) for x, y in zip(good, op.forward(xs)))
    op.status()
    one = zs.Orthogonalize(shapes, "bf16", coefficients=ref.COEFFICIENTS[:1])
    step, grads = make_step(shapes, 1, "bf16")
    master = step.master.clone()
    zs.zero_lm_inject_stall()
    step.step(grads, 0.1)
    with pytest.raises(zs.ZeroError):
        step.status()
    assert torch.equal(step.master, master)        # the products were lost before the update
    one.forward(xs)
    one.status()
    with pytest.raises(zs.ZeroError):
        zs.zero_lm_status()


def test_streams_take_turns():
    """A call on another stream than the last one's waits for that one."""
    shapes = [(400, 700)] * 3
    op, grads = make_step(shapes, 3, "bf16")
    twin, _ = make_step(shapes, 3, "bf16")
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for k in range(9):
        with torch.cuda.stream(streams[k % 3]):
            op.step(grads, 0.01)
    torch.cuda.synchronize()
    for _ in range(9):
        twin.step(grads, 0.01)
    torch.cuda.synchronize()
    assert torch.equal(op.master, twin.master)


def test_calls_on_two_streams_at_once():
    """Small and large matrices, steps and log probabilities beside one another, each by owners of its own."""
    small = [gaussian(10, 1300, seed=k).bfloat16() for k in range(40)]
    large = [gaussian(300, 700, seed=k).bfloat16() for k in range(3)]
    h, t = gaussian(300, 128).bfloat16(), gaussian(5000, 128, 1, 0.1).bfloat16()
    tg = torch.arange(300, device="cuda")
    step, grads = make_step([(40, 64), (200, 300)], 3, "bf16")
    twin, _ = make_step([(40, 64), (200, 300)], 3, "bf16")
    ops = [zs.Orthogonalize([(10, 1300)] * 40, "bf16"), zs.Orthogonalize([(300, 700)] * 3, "bf16"),
           zs.LmLogprobs(5000, 128, "bf16", max_tokens=300, top=4)]

    def calls(k):
        return (ops[0].forward(small), ops[1].forward(large), ops[2].logprobs(h, t, tg))[k]

    want = [calls(k) for k in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [[], [], []]
    for _ in range(10):
        for k in range(3):
            with torch.cuda.stream(streams[k]):
                got[k].append(calls(k))
        with torch.cuda.stream(streams[3]):
            step.step(grads, 0.01)
    torch.cuda.synchronize()
    for k in range(3):
        ops[k].status()
        assert all(torch.equal(x, y) for out in got[k] for x, y in zip(out, want[k]))
    for _ in range(10):
        twin.step(grads, 0.01)
    torch.cuda.synchronize()
    assert torch.equal(step.master, twin.master)
