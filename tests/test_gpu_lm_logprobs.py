"""Log probabilities, entropy and alternatives over a large vocabulary, and
their gradients, against a plain 64-bit form inside derived bounds."""

import math

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests import lm_reference as ref

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def make(N, V, d, dtype, seed=0, ignored=0.2, h_sigma=1.0, t_sigma=None, grid=False, ids=torch.int64):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(N, d, device="cuda", generator=gen) * h_sigma
    t = torch.randn(V, d, device="cuda", generator=gen) * (t_sigma or min(0.3, 2 / d ** 0.5))
    if grid:
        # sums of products that are exact in fp32 in any order, so that the order of the logits is known
        h, t = (h * 8).round().clamp(-32, 32) / 8, (t * 64).round().clamp(-32, 32) / 64
    tg = torch.randint(0, V, (N,), device="cuda", generator=gen)
    tg[torch.rand(N, device="cuda", generator=gen) < ignored] = -100
    return h.to(DT[dtype]), t.to(DT[dtype]), tg.to(ids)


def check(h, t, tg, scale=1.0, top=0, op=None, what=""):
    N, V, d = h.shape[0], t.shape[0], t.shape[1]
    name = "fp16" if h.dtype == torch.float16 else "bf16"
    op = op or zs.LmLogprobs(V, d, name, max_tokens=N, scale=scale, top=top, with_grad=False)
    want = ref.logprobs_reference(h, t, tg, scale)
    got = op.logprobs(h, t, tg)
    op.status()
    for x, k in zip(got, ("logp", "entropy", "lse")):
        ref.assert_within(x, want[k], want[k + "_bound"], f"{what} {k}")
    assert (got[0][~ref.valid_mask(tg, V)] == 0).all()
    if top:
        values, ids = got[3].double(), got[4].long()
        assert ids.dtype == torch.int64 and ids.min() >= 0 and ids.max() < V
        assert all(len(set(row)) == top for row in ids.tolist())
        at = want["logs"].gather(1, ids)
        slack = (2 * want["z_bound"] + want["lse_bound"])[:, None] + (at.abs() + 1) * 2.0 ** -22
        ref.assert_within(values, at, slack, f"{what} top_logp")
        # no other word's logit is larger than the least of the list by more than two logits' errors
        best = torch.topk(want["logs"], top, dim=1).values
        assert (at >= best - 2 * want["z_bound"][:, None]).all(), what
        assert (values[:, 1:] <= values[:, :-1]).all()
    return got, want


SIZES = [(1, 1, 8), (1, 2, 8), (2, 31, 16), (3, 257, 72), (31, 1000, 136), (32, 513, 64), (33, 513, 64), (96, 513, 264),
         (97, 513, 264), (97, 1, 8), (127, 255, 64), (129, 1031, 264), (255, 511, 136), (257, 2048, 128),
         (300, 4099, 520), (1, 50257, 768), (130, 50257, 64), (515, 777, 2056), (20_000, 300, 16)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("N,V,d", SIZES)
def test_logprobs(N, V, d, dtype):
    h, t, tg = make(N, V, d, dtype, seed=N + V + d)
    for top in sorted({0, min(V, 3), min(V, 8), min(V, 16)}):
        check(h, t, tg, scale=(0.5, 1.0, 1.25)[top % 3], top=top, what=f"{N}x{V}x{d} top {top}")


def in_order(logits, top):
    return torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top]


@pytest.mark.parametrize("top", [1, 5, 8, 16])
@pytest.mark.parametrize("N", [1, 16, 96, 97, 300, 5000])
def test_alternatives_are_exact_where_the_logits_are(N, top):
    """The ids in order, the lower of equal logits' first; the same logit many times over."""
    h, t, tg = make(N, 3001, 64, "bf16", seed=N, grid=True)
    t[100:140] = t[2000:2040]
    t[1500] = t[7]
    got, want = check(h, t, tg, top=top)
    assert torch.equal(got[4].long(), in_order(want["logits"], top))
    same = torch.zeros_like(t)
    got, _ = check(h, same, tg, top=top, what="all equal")
    assert torch.equal(got[4], torch.arange(top, device="cuda", dtype=torch.int32).expand(N, top))
    up = torch.zeros_like(t)
    up[:, 0] = torch.arange(3001, device="cuda").div(16, rounding_mode="floor")     # rising: every column enters the list
    ones = torch.ones_like(h)
    got, want = check(ones, up, tg, top=top, what="rising")
    assert torch.equal(got[4].long(), in_order(want["logits"], top))


@pytest.mark.parametrize("top", [3, 8, 9, 16])
@pytest.mark.parametrize("V", [16384, 65536, 65537, 131072, 131073, 300_001])
def test_alternatives_of_large_vocabularies(V, top):
    """The largest logits next to one another, far apart, and at every distance that one thread's groups may have."""
    h, t, tg = make(3, V, 8, "bf16", seed=V, grid=True)
    h[0] = 1
    for step in (1, 31, 32, 512, 4096, 8192, 16384, 32768):
        u = t.clone() / 64
        at = (torch.arange(40, device="cuda") * step + 5) % V
        u[at] = torch.arange(40, device="cuda").div(3, rounding_mode="floor")[:, None].to(u.dtype) + 1
        got, want = check(h, u, tg, top=top, what=f"step {step}")
        assert torch.equal(got[4].long(), in_order(want["logits"], top)), step
    got, _ = check(h, torch.zeros_like(t), tg, top=top, what="all equal")
    assert torch.equal(got[4], torch.arange(top, device="cuda", dtype=torch.int32).expand(3, top))


@pytest.mark.parametrize("N", [5, 150])
def test_fewer_numbers_than_alternatives(N):
    """Logits of -infinity and NaN are not listed."""
    h, t, tg = make(N, 40, 64, "bf16", grid=True)
    h = h.abs() + 1
    t[3:] = 0
    t[3:, 0] = float("-inf")
    op = zs.LmLogprobs(40, 64, "bf16", max_tokens=N, top=8, with_grad=False)
    logp, entropy, lse, values, ids = op.logprobs(h, t, tg)
    want = ref.logprobs_reference(h, t[:3], torch.full_like(tg, -1))
    assert torch.equal(ids[:, :3].long(), in_order(want["logits"], 3)) and (ids[:, 3:] == -1).all()
    assert (values[:, 3:] == float("-inf")).all()
    ref.assert_within(lse, want["lse"], want["lse_bound"], "lse")
    ref.assert_within(entropy, want["entropy"], want["entropy_bound"], "entropy")
    t[7, 0] = float("nan")
    logp, entropy, lse, values, ids = op.logprobs(h, t, tg)
    assert torch.isnan(lse).all() and torch.isnan(entropy).all() and torch.isnan(values[:, :3]).all()
    assert torch.equal(ids[:, :3].long(), in_order(want["logits"], 3)) and (ids[:, 3:] == -1).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_sharp_and_flat_distributions(dtype):
    """Logits of hundreds (an entropy of almost 0) and logits that are all equal (log of the vocabulary)."""
    for N in (40, 200):
        h, t, tg = make(N, 700, 64, dtype, h_sigma=3.0, t_sigma=2.0)
        got, _ = check(h, t, tg, top=4, what="sharp")
        assert (got[1] >= 0).all()
        got, _ = check(torch.zeros_like(h), t, tg, scale=0.5, what="flat")
        assert ((got[1].double() - math.log(700)).abs() <= 1e-5).all()


def test_more_tokens_than_a_slab():
    """Over 32768 tokens, with 50 left over for the few tokens' form."""
    h, t, tg = make(32768 + 50, 300, 16, "bf16", grid=True, seed=3)
    got, want = check(h, t, tg, top=3)
    assert torch.equal(got[4].long(), in_order(want["logits"], 3))


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("N", [60, 150])
def test_targets_outside_the_vocabulary(N, ids):
    h, t, tg = make(N, 300, 64, "bf16", ids=ids)
    tg[::3], tg[1::3] = 300, -1
    tg[5] = 2 ** 31 - 1
    if ids == torch.int64:
        tg[6], tg[7] = 2 ** 32 + 5, -2 ** 63
    check(h, t, tg, top=2)


def test_a_row_that_is_not_finite_stays_one_row():
    for N in (50, 200):
        h, t, tg = make(N, 400, 64, "bf16", ignored=0.0)
        h[17, 3] = float("nan")
        op = zs.LmLogprobs(400, 64, "bf16", max_tokens=N, top=2)
        logp, entropy, lse, values, ids = op.logprobs(h, t, tg)
        keep = torch.arange(N, device="cuda") != 17
        for x in (logp, entropy, lse, values):
            assert torch.isnan(x[17]).all() and torch.isfinite(x[keep]).all()
        assert (ids[17] == -1).all() and (ids[keep] >= 0).all()
        dh, _ = op.grad(h, t, tg, lse, torch.ones(N, device="cuda"))
        assert torch.isnan(dh[17]).all() and torch.isfinite(dh[keep]).all()


def check_grad(h, t, tg, a, b=None, scale=1.0, what=""):
    N, V, d = h.shape[0], t.shape[0], t.shape[1]
    op = zs.LmLogprobs(V, d, "fp16" if h.dtype == torch.float16 else "bf16", max_tokens=N, scale=scale)
    want = ref.logprobs_reference(h, t, tg, scale, a, b)
    logp, entropy, lse = op.logprobs(h, t, tg)
    dh, dt = op.grad(h, t, tg, lse, a, entropy, b)
    op.status()
    ref.assert_within(dh, want["dhidden"], want["dhidden_bound"], f"{what} dhidden")
    ref.assert_within(dt, want["dtable"], want["dtable_bound"], f"{what} dtable")
    return dh, dt, want


def weights(N, seed=0, unit=1.0, zeros=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed + 99)
    a = torch.randn(N, device="cuda", generator=gen) * unit
    a[torch.rand(N, device="cuda", generator=gen) < zeros] = 0.0
    return a, torch.rand(N, device="cuda", generator=gen) * (-0.1 * unit)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("N,V,d", [(1, 1, 8), (2, 31, 16), (33, 513, 64), (129, 1031, 264), (300, 4099, 520),
                                   (1, 50257, 768), (515, 777, 2056)])
def test_gradients(N, V, d, dtype):
    h, t, tg = make(N, V, d, dtype, seed=N + V + d)
    unit = 2048.0 / N if dtype == "fp16" else 1.0 / N
    a, b = weights(N, unit=unit)
    for scale, given in ((1.0, None), (1.25, b)):
        dh, dt, want = check_grad(h, t, tg, a, given, scale, f"{N}x{V}x{d}")
        if N >= 64:
            assert ref.rel_norm(dh, want["dhidden"]) <= 2 * ref.HALF_ULP[h.dtype]
            assert ref.rel_norm(dt, want["dtable"]) <= 2 * ref.HALF_ULP[h.dtype]


def test_pieces_of_the_vocabulary():
    h, t, tg = make(5000, 20011, 72, "bf16", seed=3)
    a, b = weights(5000, unit=1 / 5000)
    dh, dt, want = check_grad(h, t, tg, a, b)
    assert ref.rel_norm(dh, want["dhidden"]) <= 2 * ref.HALF_ULP[h.dtype]
    assert ref.rel_norm(dt, want["dtable"]) <= 2 * ref.HALF_ULP[h.dtype]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_weights_of_many_sizes(dtype):
    """From 1e-3 of the largest up, a largest far from 1, and of both signs."""
    h, t, tg = make(200, 700, 64, dtype)
    for unit in (1e-2, 1.0, 3e3) if dtype == "fp16" else (1e-20, 1.0, 1e20):
        gen = torch.Generator(device="cuda").manual_seed(5)
        a = torch.exp(torch.rand(200, device="cuda", generator=gen) * math.log(1e3)) * 1e-3 * unit
        a[::2] *= -1
        check_grad(h, t, tg, a, None, what=f"{unit}")


def test_the_cross_entropy_is_a_special_case():
    """a = -scale for every token: the gradients of zero_lm_loss_grad, each within its own bound."""
    h, t, tg = make(200, 700, 64, "bf16")
    want = ref.lm_reference(h, t, tg, 0.25)
    op = zs.LmLogprobs(700, 64, "bf16", max_tokens=200)
    logp, entropy, lse = op.logprobs(h, t, tg)
    dh, dt = op.grad(h, t, tg, lse, torch.full((200,), -0.25, device="cuda"))
    ref.assert_within(-logp, want["loss"], want["loss_bound"] + want["loss"].abs() * 2.0 ** -22, "loss")
    ref.assert_within(dh, want["dhidden"], want["dhidden_bound"], "dhidden")
    ref.assert_within(dt, want["dtable"], want["dtable_bound"], "dtable")


def test_against_differences():
    """The gradients against central differences of the 64-bit form, along directions."""
    h, t, tg = make(40, 90, 32, "fp16", seed=4, t_sigma=0.3)
    a, b = weights(40, unit=8.0, zeros=0.0)
    op = zs.LmLogprobs(90, 32, "fp16", max_tokens=40, scale=0.5)
    logp, entropy, lse = op.logprobs(h, t, tg)
    dh, dt = op.grad(h, t, tg, lse, a, entropy, b)
    valid = ref.valid_mask(tg, 90)

    def value(x, y):
        logs = torch.log_softmax(0.5 * (x @ y.T), 1)
        picked = logs.gather(1, torch.where(valid, tg, 0)[:, None])[:, 0]
        return ((a.double() * picked - b.double() * (logs.exp() * logs).sum(1)) * valid).sum()

    gen = torch.Generator(device="cuda").manual_seed(8)
    x, y, e = h.double(), t.double(), 1e-4
    bound = ref.logprobs_reference(h, t, tg, 0.5, a, b)
    for _ in range(4):
        u = torch.randn(x.shape, device="cuda", generator=gen, dtype=torch.float64)
        w = torch.randn(y.shape, device="cuda", generator=gen, dtype=torch.float64)
        numeric = (value(x + e * u, y + e * w) - value(x - e * u, y - e * w)) / (2 * e)
        mine = (dh.double() * u).sum() + (dt.double() * w).sum()
        # the outputs' own bounds, and the differences' third order: e^2 times derivatives of some thousands
        slack = (bound["dhidden_bound"] * u.abs()).sum() + (bound["dtable_bound"] * w.abs()).sum() + 1e-3
        assert (mine - numeric).abs() <= slack


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_nothing_leaks_from_tokens_without_target_or_weight(bad):
    for dtype in ("fp16", "bf16"):
        h, t, tg = make(140, 400, 64, dtype)
        a, b = weights(140)
        b[a == 0] = 0.0
        skipped = ~ref.valid_mask(tg, 400) | (a == 0)
        assert skipped.any() and not skipped.all()
        a[~ref.valid_mask(tg, 400)] = bad          # weights of tokens without target are not looked at
        op = zs.LmLogprobs(400, 64, dtype, max_tokens=140)
        clean = op.logprobs(h, t, tg)
        dh0, dt0 = op.grad(h, t, tg, clean[2], a, clean[1], b)
        h[skipped] = bad
        logp, entropy, lse = op.logprobs(h, t, tg)
        dh, dt = op.grad(h, t, tg, lse, a, entropy, b)
        assert (dh[skipped] == 0).all() and torch.equal(dh, dh0) and torch.equal(dt, dt0)


def test_all_weights_zero():
    for dtype in ("fp16", "bf16"):
        h, t, tg = make(140, 400, 64, dtype)
        zero = torch.zeros(140, device="cuda")
        dh, dt, _ = check_grad(h, t, tg, zero, zero)
        assert not dh.any() and not dt.any()


def test_strides_accumulation_and_buffers():
    N, V, d = 133, 517, 72
    h0, t0, tg = make(N, V, d, "bf16", seed=5)
    h, t = (torch.full((n, d + w), 7.0, dtype=h0.dtype, device="cuda") for n, w in ((N, 24), (V, 8)))
    h[:, 8:8 + d], t[:, :d] = h0, t0
    a, b = weights(N)
    op = zs.LmLogprobs(V, d, "bf16", max_tokens=200, top=5)
    plain = op.logprobs(h0, t0, tg)
    wide = op.logprobs(h[:, 8:8 + d], t[:, :d], tg)
    assert all(torch.equal(x, y) for x, y in zip(plain, wide))
    dh0, dt0 = op.grad(h0, t0, tg, plain[2], a, plain[1], b)
    dhb = torch.full((N, d + 16), 3.0, dtype=h0.dtype, device="cuda")
    dtb = torch.full((V, d + 40), 3.0, dtype=h0.dtype, device="cuda")
    op.grad(h[:, 8:8 + d], t[:, :d], tg, plain[2], a, plain[1], b, dhidden=dhb[:, 16:], dtable=dtb[:, 40:])
    assert torch.equal(dhb[:, 16:], dh0) and torch.equal(dtb[:, 40:], dt0)
    assert (dhb[:, :16] == 3).all() and (dtb[:, :40] == 3).all()
    old = torch.randn(V, d, device="cuda").to(h0.dtype)
    got = op.grad(h0, t0, tg, plain[2], a, plain[1], b, dtable=old.clone(), accumulate=True)[1]
    want = ref.logprobs_reference(h0, t0, tg, 1.0, a, b)
    total = want["dtable"] + old.double()
    ref.assert_within(got, total, want["dtable_bound"] + total.abs() * (ref.HALF_ULP[h0.dtype] + 2.0 ** -23), "added")


def test_no_tokens():
    op = zs.LmLogprobs(50, 16, "bf16", max_tokens=8, top=4)
    h, t = torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(50, 16, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    out = op.logprobs(h, t, none)
    assert [tuple(x.shape) for x in out] == [(0,), (0,), (0,), (0, 4), (0, 4)]
    empty = torch.zeros(0, device="cuda")
    dh, dt = op.grad(h, t, none, empty, empty)
    assert dh.shape == (0, 16) and not dt.any()


@pytest.mark.parametrize("N", [40, 300])
def test_the_same_bits_every_time_and_in_a_graph(N):
    h, t, tg = make(N, 5000, 128, "bf16", seed=2)
    a, b = weights(N)
    op = zs.LmLogprobs(5000, 128, "bf16", max_tokens=N, top=8)

    def once():
        out = op.logprobs(h, t, tg)
        return out + op.grad(h, t, tg, out[2], a, out[1], b)

    first = once()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, once()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        once()
    side.synchronize()
    with torch.cuda.graph(graph):
        out = once()
    h2, t2, tg2 = make(N, 5000, 128, "bf16", seed=7)
    h.copy_(h2), t.copy_(t2), tg.copy_(tg2)
    graph.replay()
    torch.cuda.synchronize()
    fresh = once()
    assert all(torch.equal(x, y) for x, y in zip(out, fresh))
    op.status()


@pytest.mark.parametrize("N,which", [(40, "logprobs"), (300, "logprobs"), (300, "grad")])
def test_a_wait_that_runs_out_is_reported(N, which):
    h, t, tg = make(N, 5000, 128, "bf16")
    op, other = (zs.LmLogprobs(5000, 128, "bf16", max_tokens=N, top=4) for _ in range(2))
    a = torch.ones(N, device="cuda")
    good = op.logprobs(h, t, tg)
    grads = op.grad(h, t, tg, good[2], a)
    op.status()
    zs.zero_lm_inject_stall()
    if which == "logprobs":
        out = op.logprobs(h, t, tg)
        assert torch.isnan(out[2]).any()
    else:
        out = op.grad(h, t, tg, good[2], a)
        assert torch.isnan(out[0]).all() and torch.isnan(out[1]).all()
    other.logprobs(h, t, tg)
    other.status()
    with pytest.raises(zs.ZeroError) as e:
        op.status()
    assert e.value.code == zs.ZERO_E_STATE
    with pytest.raises(zs.ZeroError):
        zs.zero_lm_status()
    zs.zero_lm_status()
    assert all(torch.equal(x, y) for x, y in zip(good, op.logprobs(h, t, tg)))
    assert all(torch.equal(x, y) for x, y in zip(grads, op.grad(h, t, tg, good[2], a)))
    op.status()
