"""The global gradient norm over many tensors, clipping, and the clipped step."""

import math

import numpy as np
import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests import gpu_harness as gh
from tests import lm_reference as ref
from tests.canary import Arena

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
LR, B1, B2, EPS = 1e-3, 0.9, 0.95, 1e-8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def tensors(sizes, W, dtype, sigma=1e-2, seed=0, skew=0):
    """W lists of tensors; with skew each starts `skew` elements into its buffer."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [[(torch.randn(k + skew, device="cuda", generator=gen) * sigma).to(DT[dtype])[skew:] for k in sizes]
            for _ in range(W)]


def check(sizes, W, dtype, max_norm, **kw):
    grads = tensors(sizes, W, dtype, **kw)
    flat = [torch.cat(g) if g else torch.empty(0, device="cuda") for g in grads]
    norm64, want = ref.clip_reference(flat, W, max_norm)
    op = zs.GradClip(sizes, W, dtype)
    norm, out = op.norm_and_clip(grads, max_norm)
    # fp32 means (W roundings), fp32 squares of a thread's share (at most 8192 * 64 / 256 additions of them), fp64 beyond
    assert abs(norm.item() - norm64) <= norm64 * (W + 2048) * 2.0 ** -24, (norm.item(), norm64)
    u = ref.HALF_ULP.get(DT[dtype], 2.0 ** -24)
    size = sum(f.double().abs() for f in flat) / W
    bound = want.abs() * (u + (W + 2056) * 2.0 ** -24) + size * W * 2.0 ** -24 + ref.TINY16.get(DT[dtype], 0.0)
    ref.assert_within(out, want, bound, f"{len(sizes)} tensors, W={W}, {dtype}")
    assert torch.equal(op.clip(grads, norm, max_norm), out) and torch.equal(op.norm(grads), norm)
    return norm, out


SIZES = {"one": [1], "empty": [0, 0], "odd": [1, 2, 3, 7, 8, 9, 0, 15, 4097, 8191, 8192, 8193, 70001],
         "big": [3_000_000, 5, 1_000_001], "many": [(37 * k) % 211 + 1 for k in range(3000)]}


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("W", [1, 3, 8])
@pytest.mark.parametrize("sizes", list(SIZES), ids=list(SIZES))
def test_norm_and_clip(sizes, W, dtype):
    check(SIZES[sizes], W, dtype, 0.25)           # clipped (where there is anything to clip)
    check(SIZES[sizes], W, dtype, 1e6)            # not clipped


@pytest.mark.parametrize("skew", [1, 3, 8])
def test_alignments(skew):
    for dtype in ("fp16", "fp32"):
        check([5, 100, 8192, 20_003], 2, dtype, 0.5, skew=skew)
    # each rank's buffers placed differently
    sizes = [100, 20_003]
    a, b = tensors(sizes, 1, "bf16", skew=1)[0], tensors(sizes, 1, "bf16", skew=2, seed=1)[0]
    op = zs.GradClip(sizes, 2, "bf16")
    norm, out = op.norm_and_clip([a, b], 0.5)
    n64, want = ref.clip_reference([torch.cat(a), torch.cat(b)], 2, 0.5)
    assert abs(norm.item() - n64) <= 1e-4 * n64
    assert ref.rel_norm(out, want) <= 2.0 ** -8


def test_ranks_beyond_the_fixed_counts():
    check([1000, 77], 64, "bf16", 0.01)
    check([1000, 77], 5, "fp16", 0.01)


def test_in_place_and_guard_bytes():
    sizes = [33, 8192, 70_001]
    arena = Arena(16 << 20, "cuda")
    plain = tensors(sizes, 1, "bf16")[0]
    grads = []
    for g in plain:
        x = arena.zeros(g.numel(), torch.bfloat16)
        x.copy_(g)
        grads.append(x)
    op = zs.GradClip(sizes, 1, "bf16", alloc=arena)
    want = op.norm_and_clip([plain], 0.1)[1]
    norm = op.norm([grads])
    zs.zero_grad_clip(1, sizes, zs.ZERO_BF16, grads, norm, 0.1, grads)
    assert torch.equal(torch.cat(grads), want)
    arena.check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_norm_that_is_not_finite_scales_nothing(bad):
    grads = tensors([100, 9000], 2, "fp16")
    grads[1][1][4567] = bad
    op = zs.GradClip([100, 9000], 2, "fp16")
    norm, out = op.norm_and_clip(grads, 1e-3)
    assert not math.isfinite(norm.item())
    mean = (torch.cat(grads[0]).float() + torch.cat(grads[1]).float()) / 2
    keep = torch.isfinite(mean)
    assert torch.equal(out[keep], mean[keep].half())


# ---- the clipped step ------------------------------------------------------------------

def ranks(step, W, dtype, sigma, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for buf in step.new_grad_buffers():
        step.place_(buf, (torch.randn(step.n, device="cuda", generator=gen) * sigma).to(buf.dtype))
        out.append(buf)
    return out


def state(step):
    torch.cuda.synchronize()
    return [x.clone() for x in (step.master, step.m, step.v, step.working_copy())]


CONFIGS = [(zs.ZERO_SCHEME_DP, 1, [1], "fp16"), (zs.ZERO_SCHEME_Z1, 4, [37], "bf16"),
           (zs.ZERO_SCHEME_Z2, 8, [300_007], "bf16"), (zs.ZERO_SCHEME_Z2, 16, [65_536], "fp16"),
           (zs.ZERO_SCHEME_Z2, 3, [10_001], "fp16"), (zs.ZERO_SCHEME_Z3, 4, [70_001, 0, 5, 65_536], "bf16"),
           (zs.ZERO_SCHEME_Z3, 8, [4096, 4096, 4096], "fp16"), (zs.ZERO_SCHEME_Z2, 2, [0], "fp16")]


@pytest.mark.parametrize("scheme,W,units,dtype", CONFIGS)
def test_clipped_step_against_the_oracle(scheme, W, units, dtype):
    n = sum(units)
    theta0 = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)) * 0.02
    step = zs.ZeroStep(scheme, W, units, dtype, theta0=theta0)
    idx = step.real_index()
    master = theta0.double().cpu().numpy()
    m, v = np.zeros(n), np.zeros(n)
    for t in range(1, 5):
        grads = ranks(step, W, dtype, 1e-2, seed=t)
        max_norm = 0.05 if t % 2 else 1e9
        step.step(grads, LR, B1, B2, EPS, t, max_norm=max_norm)
        norm, g = ref.clip_reference([b[idx] for b in grads], W, max_norm)
        assert abs(step.grad_norm.item() - norm) <= norm * (W + 2048) * 2.0 ** -24
        g = g.cpu().numpy()
        m = B1 * m + (1 - B1) * g
        v = B2 * v + (1 - B2) * g * g
        master = master - LR / (1 - B1 ** t) * m / (np.sqrt(v / (1 - B2 ** t)) + EPS)
        got = [x[idx].cpu().numpy() for x in (step.master, step.m, step.v)]
        for what, a, b in zip(("master", "m", "v"), got, (master, m, v)):
            # the clipping coefficient's error (the norm's) enters m once and v twice
            tol = 1e-5 * np.abs(b) + 2 * (W + 2056) * 2.0 ** -24 * np.abs(b) + 1e-6 * np.abs(b).max(initial=0.0)
            assert (np.abs(a - b) <= tol).all(), (what, t)
        own = step.master[idx].to(step.work_torch_dtype)
        assert np.array_equal(gh.bits_of(step.working_copy()[idx]), gh.bits_of(own))
    mask = torch.ones(step.n_pad, dtype=torch.bool, device="cuda")
    mask[idx] = False
    assert all((x[mask] == 0).all() for x in (step.master, step.m, step.v))
    step.close()


@pytest.mark.parametrize("scheme,W,units,dtype", CONFIGS)
def test_a_norm_below_the_limit_changes_no_bit(scheme, W, units, dtype):
    theta0 = torch.randn(sum(units), device="cuda") * 0.02
    a = zs.ZeroStep(scheme, W, units, dtype, theta0=theta0)
    b = zs.ZeroStep(scheme, W, units, dtype, theta0=theta0)
    for t in range(1, 4):
        grads = ranks(a, W, dtype, 1e-3, seed=t)
        a.step(grads, LR, B1, B2, EPS, t)
        b.step(grads, LR, B1, B2, EPS, t, max_norm=1e9)
    assert all(torch.equal(x, y) for x, y in zip(state(a), state(b)))
    assert a.stat(zs.ZERO_STAT_COMM_BYTES) == b.stat(zs.ZERO_STAT_COMM_BYTES)
    assert a.stat(zs.ZERO_STAT_GATHERS) == b.stat(zs.ZERO_STAT_GATHERS)
    assert a.stat(zs.ZERO_STAT_SCATTERS) == b.stat(zs.ZERO_STAT_SCATTERS)
    a.close(), b.close()


def test_schemes_agree_bit_for_bit():
    theta0 = torch.randn(100_000, device="cuda") * 0.02
    got = []
    for scheme in (zs.ZERO_SCHEME_DP, zs.ZERO_SCHEME_Z2, zs.ZERO_SCHEME_Z3):
        s = zs.ZeroStep(scheme, 8, [100_000], "bf16", theta0=theta0)
        for t in range(1, 4):
            s.step(ranks(s, 8, "bf16", 1e-2, seed=t), LR, B1, B2, EPS, t, max_norm=0.1)
        got.append(state(s) + [s.grad_norm.clone()])
        s.close()
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))


@pytest.mark.parametrize("scheme", [zs.ZERO_SCHEME_Z2, zs.ZERO_SCHEME_Z3])
def test_overflow_leaves_the_state(scheme):
    units = [5000] if scheme != zs.ZERO_SCHEME_Z3 else [3000, 2000]
    s = zs.ZeroStep(scheme, 4, units, "fp16", theta0=torch.randn(5000, device="cuda"))
    s.step(ranks(s, 4, "fp16", 1e-2, 1), LR, B1, B2, EPS, 1, max_norm=1.0)
    before = state(s)
    grads = ranks(s, 4, "fp16", 1e-2, 2)
    grads[2][1234] = float("inf")
    s.step(grads, LR, B1, B2, EPS, 2, max_norm=1.0)
    assert all(torch.equal(x, y) for x, y in zip(before, state(s))) and math.isinf(s.grad_norm.item())
    s.step(ranks(s, 4, "fp16", 1e-2, 3), LR, B1, B2, EPS, 3, max_norm=1.0)
    assert not torch.equal(before[0], state(s)[0])
    s.close()


def test_zero3_with_a_hook_that_makes_the_gradients():
    """The hook fills each unit's gradients in the backward pass: the norm has to wait for all of them."""
    units, W = [3000, 70_001, 512], 4
    theta0 = torch.randn(sum(units), device="cuda") * 0.02
    main, gather = torch.cuda.Stream(), torch.cuda.Stream()
    a = zs.ZeroStep(zs.ZERO_SCHEME_Z3, W, units, "bf16", theta0=theta0)
    grads = ranks(a, W, "bf16", 1e-2, 5)
    torch.cuda.synchronize()
    b = zs.ZeroStep(zs.ZERO_SCHEME_Z3, W, units, "bf16", theta0=theta0, stream=main, gather_stream=gather)
    late = b.new_grad_buffers()
    torch.cuda.synchronize()
    seen = []

    def hook(user, phase, unit, buf, stream):
        seen.append((phase, unit))
        if phase == 1:
            with torch.cuda.stream(main):
                lo, hi = b.off[unit], b.off[unit] + b.shard[unit] * W
                for x, y in zip(late, grads):
                    x[lo:hi].copy_(y[lo:hi])

    b.set_unit_hook(hook)
    for t in (1, 2):
        a.step(grads, LR, B1, B2, EPS, t, max_norm=0.1)
        with torch.cuda.stream(main):
            for x in late:
                x.zero_()
        b.step(late, LR, B1, B2, EPS, t, max_norm=0.1)
    b.sync()
    assert seen == 2 * ([(0, u) for u in range(3)] + [(1, u) for u in (2, 1, 0)])
    assert all(torch.equal(x, y) for x, y in zip(state(a), state(b)))
    assert torch.equal(a.grad_norm, b.grad_norm)
    assert a.stat(zs.ZERO_STAT_COMM_BYTES) == b.stat(zs.ZERO_STAT_COMM_BYTES)
    a.close(), b.close()


def test_graph_replay_and_clipped_steps_mix():
    units, W = [4096] * 4, 8
    theta0 = torch.randn(sum(units), device="cuda") * 0.02
    main = torch.cuda.Stream()
    a = zs.ZeroStep(zs.ZERO_SCHEME_Z3, W, units, "bf16", theta0=theta0)
    torch.cuda.synchronize()
    b = zs.ZeroStep(zs.ZERO_SCHEME_Z3, W, units, "bf16", theta0=theta0, stream=main)
    b.set_graph(True)
    for t in range(1, 7):
        grads = ranks(a, W, "bf16", 1e-2, t)
        torch.cuda.synchronize()
        limit = 0.1 if t % 3 == 0 else None
        a.step(grads, LR, B1, B2, EPS, t, max_norm=limit)
        b.step(grads, LR, B1, B2, EPS, t, max_norm=limit)
        b.sync()
    assert all(torch.equal(x, y) for x, y in zip(state(a), state(b)))
    a.close(), b.close()


def test_step_guard_bytes():
    for scheme, units in ((zs.ZERO_SCHEME_Z2, [100_003]), (zs.ZERO_SCHEME_Z3, [5, 0, 17, 4096, 99_991])):
        arena = Arena(96 << 20, "cuda")
        theta0 = torch.randn(sum(units), device="cuda") * 0.02
        a = zs.ZeroStep(scheme, 5, units, "fp16", theta0=theta0, alloc=arena)
        b = zs.ZeroStep(scheme, 5, units, "fp16", theta0=theta0)
        for t in (1, 2):
            ga = ranks(a, 5, "fp16", 1e-2, t)
            gb = ranks(b, 5, "fp16", 1e-2, t)
            a.step(ga, LR, B1, B2, EPS, t, max_norm=0.1)
            b.step(gb, LR, B1, B2, EPS, t, max_norm=0.1)
        assert all(torch.equal(x, y) for x, y in zip(state(a), state(b)))
        arena.check()
        a.close(), b.close()


def test_refusals():
    s = zs.ZeroStep(zs.ZERO_SCHEME_Z2, 2, [100], "fp16")
    g = s.new_grad_buffers()
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(zs.ZeroError):
            s.step(g, LR, B1, B2, EPS, 1, max_norm=bad)
    with pytest.raises(zs.ZeroError):
        s.step(g, LR, B1, B2, EPS, 2, max_norm=1.0)       # out of order, as without clipping
    s.step(g, LR, B1, B2, EPS, 1, max_norm=1.0)
    op = zs.GradClip([10, 20], 1, "fp16")
    ok = tensors([10, 20], 1, "fp16")
    for wrong in (tensors([10, 21], 1, "fp16"), tensors([10], 1, "fp16"), tensors([10, 20], 2, "fp16"),
                  tensors([10, 20], 1, "bf16"), [[ok[0][0], torch.zeros(40, dtype=torch.float16, device="cuda")[::2]]]):
        with pytest.raises(ValueError):
            op.norm(wrong)


@pytest.mark.parametrize("scheme,units", [(zs.ZERO_SCHEME_Z2, [300_007]), (zs.ZERO_SCHEME_Z3, [4096, 70_001, 5])])
def test_timing_shows_the_norm_pass(scheme, units):
    s = zs.ZeroStep(scheme, 4, units, "bf16", theta0=torch.randn(sum(units), device="cuda"))
    zs.zero_enable_timing(s.ctx, True)
    for t in (1, 2, 3):
        s.step(ranks(s, 4, "bf16", 1e-2, t), LR, B1, B2, EPS, t, max_norm=1.0)
    s.step(ranks(s, 4, "bf16", 1e-2, 4), LR, B1, B2, EPS, 4)
    ms, n = zs.zero_read_timing(s.ctx, zs.ZERO_KERNEL_NORM)
    assert n == 3 and ms > 0
    ms, n = zs.zero_read_timing(s.ctx, zs.ZERO_KERNEL_FUSED)
    assert n == 4 * len(units) and ms > 0
    assert zs.zero_read_timing(s.ctx, zs.ZERO_KERNEL_NORM) == (0.0, 0)
    s.close()


@pytest.mark.parametrize("W", [1, 2])
def test_few_ranks_step_without_a_mean(W):
    """Their workspace has no room for one; guards lie around all of it."""
    n = 100_003
    arena = Arena(96 << 20, "cuda")
    theta0 = torch.randn(n, device="cuda") * 0.02
    a = zs.ZeroStep(zs.ZERO_SCHEME_Z2, W, [n], "fp16", theta0=theta0, alloc=arena)
    b = zs.ZeroStep(zs.ZERO_SCHEME_Z2, W, [n], "fp16", theta0=theta0)
    for t in (1, 2):
        grads = ranks(a, W, "fp16", 1e-2, t)
        a.step(grads, LR, B1, B2, EPS, t, max_norm=0.1)
        b.step(grads, LR, B1, B2, EPS, t, max_norm=0.1)
    assert all(torch.equal(x, y) for x, y in zip(state(a), state(b))) and torch.equal(a.grad_norm, b.grad_norm)
    arena.check()
    a.close(), b.close()


def test_a_norm_just_below_the_limit():
    """The factor is limit / (norm + 1e-6): 1 from norm + 1e-6 <= limit on, below 1 for a limit equal to the norm."""
    theta0 = torch.randn(1000, device="cuda") * 0.02
    a, b = (zs.ZeroStep(zs.ZERO_SCHEME_Z2, 4, [1000], "bf16", theta0=theta0) for _ in range(2))
    grads = ranks(a, 4, "bf16", 1e-5, 1)
    a.step(grads, LR, B1, B2, EPS, 1)
    b.step(grads, LR, B1, B2, EPS, 1, max_norm=1e9)
    norm = np.float32(b.grad_norm.item())
    for limit, same in ((np.float32(norm + np.float32(1e-6)), True), (norm, False)):
        c = zs.ZeroStep(zs.ZERO_SCHEME_Z2, 4, [1000], "bf16", theta0=theta0)
        c.step(grads, LR, B1, B2, EPS, 1, max_norm=float(limit))
        assert torch.equal(c.m, a.m) == same
        factor = 1.0 if same else float(limit) / (float(norm) + 1e-6)
        assert torch.allclose(c.m.double(), a.m.double() * factor, rtol=1e-6, atol=0)
        c.close()
    a.close(), b.close()
