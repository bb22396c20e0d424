"""The cross entropy over a large vocabulary and its gradients against a plain
64-bit form, inside bounds derived from the kernels' arithmetic."""

import math

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests import lm_reference as ref
from tests.canary import Arena

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def make(N, V, d, dtype, seed=0, ignored=0.2, h_sigma=1.0, t_sigma=0.1, ids=torch.int64):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h = (torch.randn(N, d, device="cuda", generator=gen) * h_sigma).to(DT[dtype])
    t = (torch.randn(V, d, device="cuda", generator=gen) * t_sigma).to(DT[dtype])
    tg = torch.randint(0, V, (N,), device="cuda", generator=gen)
    tg[torch.rand(N, device="cuda", generator=gen) < ignored] = -100
    return h, t, tg.to(ids)


def check(h, t, tg, scale=1.0, op=None, what=""):
    N, V, d = h.shape[0], t.shape[0], t.shape[1]
    name = "fp16" if h.dtype == torch.float16 else "bf16"
    op = op or zs.LmLoss(V, d, name, max_tokens=N)
    want = ref.lm_reference(h, t, tg, scale)
    loss, lse = op.loss(h, t, tg)
    dh, dt = op.grad(h, t, tg, lse, scale)
    op.status()
    valid = ref.valid_mask(tg, V)
    assert (loss[~valid] == 0).all() and (dh[~valid] == 0).all(), what
    ref.assert_within(loss, want["loss"], want["loss_bound"], f"{what} loss")
    ref.assert_within(lse[valid], want["lse"][valid], want["lse_bound"][valid], f"{what} lse")
    ref.assert_within(dh, want["dhidden"], want["dhidden_bound"], f"{what} dhidden")
    ref.assert_within(dt, want["dtable"], want["dtable_bound"], f"{what} dtable")
    return loss, lse, dh, dt, want


SIZES = [(1, 1, 8), (1, 2, 8), (2, 31, 16), (3, 257, 72), (31, 1000, 136), (32, 513, 64), (33, 513, 64), (127, 255, 64), (128, 256, 64), (129, 1031, 264),
         (255, 511, 136), (257, 2048, 128), (300, 4099, 520), (64, 5000, 1600), (1, 50257, 768), (515, 777, 2056)]


# each width of tile that a few tokens as columns take, and the counts around its changes
FEW = [(48, 4099, 64), (64, 257, 72), (65, 1000, 136), (95, 255, 64), (96, 513, 264), (97, 513, 264)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("N,V,d", SIZES + FEW)
def test_loss_and_gradients(N, V, d, dtype):
    h, t, tg = make(N, V, d, dtype, seed=N + V + d, t_sigma=min(0.3, 2 / d ** 0.5))
    loss, lse, dh, dt, want = check(h, t, tg, scale=2048.0 / N if dtype == "fp16" else 1.0 / N, what=f"{N}x{V}x{d}")
    if want["dtable"].abs().max() > 0 and N >= 64:
        # errors that are rounding noise: well inside twice half a unit in the 2-norm
        assert ref.rel_norm(dh, want["dhidden"]) <= 2 * ref.HALF_ULP[h.dtype]
        assert ref.rel_norm(dt, want["dtable"]) <= 2 * ref.HALF_ULP[h.dtype]


def test_pieces_of_the_vocabulary():
    """Enough tokens that the gradient takes several pieces of the vocabulary."""
    h, t, tg = make(5000, 20011, 72, "bf16", seed=3)
    *_, dh, dt, want = check(h, t, tg, scale=1 / 5000)
    assert ref.rel_norm(dh, want["dhidden"]) <= 2 * ref.HALF_ULP[h.dtype]
    assert ref.rel_norm(dt, want["dtable"]) <= 2 * ref.HALF_ULP[h.dtype]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_sharp_and_flat_distributions(dtype):
    """Logits of tens (probabilities of 0 and 1) and logits that are all equal."""
    h, t, tg = make(200, 700, 64, dtype, h_sigma=3.0, t_sigma=2.0)
    check(h, t, tg, what="sharp")
    tg[:100] = (h.double() @ t.double().T).argmax(1)[:100]     # the likeliest word: losses near 0
    check(h, t, tg, what="right")
    check(torch.zeros_like(h), t, tg, what="flat")


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
def test_targets_outside_the_vocabulary(ids):
    h, t, tg = make(150, 300, 64, "bf16", ids=ids)
    tg[::3] = 300
    tg[1::3] = -1
    tg[5] = 2 ** 31 - 1
    if ids == torch.int64:
        tg[6] = 2 ** 32 + 5          # 5 if it were cut to 32 bits
        tg[7] = -2 ** 63
    check(h, t, tg)
    check(h, t, torch.full_like(tg, -100), what="no target at all")


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_nothing_leaks_from_tokens_without_target(bad):
    h, t, tg = make(140, 400, 64, "fp16")
    skipped = ~ref.valid_mask(tg, 400)
    assert skipped.any()
    h[skipped] = bad
    loss, lse, dh, dt, _ = check(h, t, tg)
    assert torch.isfinite(dh).all() and torch.isfinite(dt).all() and torch.isfinite(loss).all()


def test_a_row_that_is_not_finite_stays_one_row():
    h, t, tg = make(140, 400, 64, "bf16", ignored=0.0)
    h[17, 3] = float("nan")
    op = zs.LmLoss(400, 64, "bf16", max_tokens=140)
    loss, lse = op.loss(h, t, tg)
    dh, _ = op.grad(h, t, tg, lse, 1.0)
    assert torch.isnan(loss[17]) and torch.isnan(dh[17]).all()
    keep = torch.arange(140, device="cuda") != 17
    assert torch.isfinite(loss[keep]).all() and torch.isfinite(dh[keep]).all()


def test_strides_accumulation_and_buffers():
    """Rows inside wider buffers on both sides, and a gradient added onto one."""
    N, V, d = 133, 517, 72
    h0, t0, tg = make(N, V, d, "bf16", seed=5)
    h, t = torch.full((N, d + 24), 7.0, dtype=h0.dtype, device="cuda"), torch.full((V, d + 8), 7.0, dtype=h0.dtype, device="cuda")
    h[:, 8:8 + d], t[:, :d] = h0, t0
    op = zs.LmLoss(V, d, "bf16", max_tokens=200)
    loss0, lse0 = op.loss(h0, t0, tg)
    loss, lse = op.loss(h[:, 8:8 + d], t[:, :d], tg)
    assert torch.equal(loss, loss0) and torch.equal(lse, lse0)
    dh0, dt0 = op.grad(h0, t0, tg, lse, 0.5)
    dhb = torch.full((N, d + 16), 3.0, dtype=h0.dtype, device="cuda")
    dtb = torch.full((V, d + 40), 3.0, dtype=h0.dtype, device="cuda")
    op.grad(h[:, 8:8 + d], t[:, :d], tg, lse, 0.5, dhidden=dhb[:, 16:], dtable=dtb[:, 40:])
    assert torch.equal(dhb[:, 16:], dh0) and torch.equal(dtb[:, 40:], dt0)
    assert (dhb[:, :16] == 3).all() and (dtb[:, :40] == 3).all()
    want = ref.lm_reference(h0, t0, tg, 0.5)
    old = torch.randn(V, d, device="cuda").to(h0.dtype)
    got = op.grad(h0, t0, tg, lse, 0.5, dtable=old.clone(), accumulate=True)[1]
    total = want["dtable"] + old.double()
    bound = want["dtable_bound"] + total.abs() * ref.HALF_ULP[h0.dtype] + old.double().abs() * 2.0 ** -23
    ref.assert_within(got, total, bound, "accumulated dtable")


def test_no_tokens():
    h, t, tg = make(0, 40, 16, "fp16")
    op = zs.LmLoss(40, 16, "fp16", max_tokens=4)
    loss, lse = op.loss(h, t, tg)
    dt = torch.ones(40, 16, dtype=torch.float16, device="cuda")
    op.grad(h, t, tg, lse, 1.0, dtable=dt, accumulate=True)
    assert (dt == 1).all()
    op.grad(h, t, tg, lse, 1.0, dtable=dt)
    assert (dt == 0).all() and loss.numel() == 0


def test_repeats_are_bitwise_and_an_owner_serves_smaller_calls():
    big = zs.LmLoss(3001, 200, "bf16", max_tokens=3000)
    for N in (3000, 2999, 700, 130, 1):
        h, t, tg = make(N, 3001, 200, "bf16", seed=N)
        own = zs.LmLoss(3001, 200, "bf16", max_tokens=N)
        outs = []
        for op in (big, big, own):
            loss, lse = op.loss(h, t, tg)
            outs.append((loss, lse) + op.grad(h, t, tg, lse, 1.0 / N))
        big.status()
        for other in outs[1:]:
            assert all(torch.equal(x, y) for x, y in zip(outs[0], other)), N


def test_gradients_against_differences():
    """(L(x + s) - L(x - s)) / 2 along steps s that the 16-bit formats hold
    exactly.  Third-order terms: |L'''| <= 2 max|dl|^3 per token, dl = s t."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    N, V, d = 40, 90, 32
    h = torch.randint(-16, 17, (N, d), device="cuda", generator=gen).half() / 8
    t = torch.randint(-16, 17, (V, d), device="cuda", generator=gen).half() / 64
    tg = torch.randint(0, V, (N,), device="cuda", generator=gen)
    tg[::5] = -1
    op = zs.LmLoss(V, d, "fp16", max_tokens=N)
    lse = op.loss(h, t, tg)[1]
    dh, dt = op.grad(h, t, tg, lse, 1.0)
    total = lambda a, b: op.loss(a, b, tg)[0].double().sum()  # noqa: E731
    for which in ("hidden", "table"):
        for k in range(6):
            x = h if which == "hidden" else t
            s = torch.randint(-1, 2, x.shape, device="cuda", generator=gen).half() / (64 if which == "hidden" else 512)
            if which == "hidden":
                num = (total(h + s, t) - total(h - s, t)) / 2
                dl = (s.double() @ t.double().T).abs().amax(1)
            else:
                num = (total(h, t + s) - total(h, t - s)) / 2
                dl = (h.double() @ s.double().T).abs().amax(1)
            ana = ((dh if which == "hidden" else dt).double() * s.double()).sum()
            want = ref.lm_reference(h, t, tg)
            g = want["dhidden_bound"] if which == "hidden" else want["dtable_bound"]
            tol = (2 * dl ** 3 / 6).sum() + want["loss_bound"].sum() + (g * s.double().abs()).sum()
            assert abs(num - ana) <= tol, (which, k, float(num), float(ana), float(tol))


def test_guard_bytes():
    """Every buffer between guards, at the least alignment the ABI accepts."""
    for N, V, d in ((130, 517, 72), (33, 1000, 264)):
        arena = Arena(64 << 20, "cuda", seed=1)
        h0, t0, tg0 = make(N, V, d, "fp16", seed=N)
        h = arena.zeros(N * d, torch.float16).view(N, d)
        t = arena.zeros(V * d, torch.float16).view(V, d)
        h.copy_(h0), t.copy_(t0)
        tg = arena.zeros(N * 8, torch.uint8).view(torch.int64)
        tg.copy_(tg0)
        dh = arena.zeros(N * d, torch.float16).view(N, d)
        dt = arena.zeros(V * d, torch.float16).view(V, d)
        loss, lse = arena.zeros(N, torch.float32), arena.zeros(N, torch.float32)
        op = zs.LmLoss(V, d, "fp16", max_tokens=N, alloc=arena)
        op.loss(h, t, tg, loss=loss, lse=lse)
        op.grad(h, t, tg, lse, 1.0, dhidden=dh, dtable=dt)
        op.status()
        arena.check()
        plain = zs.LmLoss(V, d, "fp16", max_tokens=N)
        loss1, lse1 = plain.loss(h0, t0, tg0)
        dh1, dt1 = plain.grad(h0, t0, tg0, lse1, 1.0)
        assert torch.equal(loss, loss1) and torch.equal(dh, dh1) and torch.equal(dt, dt1)


def test_another_stream_than_the_current_one():
    h, t, tg = make(600, 5000, 256, "bf16")
    side = torch.cuda.Stream()
    op = zs.LmLoss(5000, 256, "bf16", max_tokens=600, stream=side)
    base = zs.LmLoss(5000, 256, "bf16", max_tokens=600)
    want = base.loss(h, t, tg)
    torch.cuda.synchronize()
    got = op.loss(h, t, tg)
    grads = op.grad(h, t, tg, got[1], 1.0)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(x, y) for x, y in zip(grads, base.grad(h, t, tg, want[1], 1.0)))


def test_owner_refusals():
    h, t, tg = make(20, 40, 16, "fp16")
    op = zs.LmLoss(40, 16, "fp16", max_tokens=20)
    lse = op.loss(h, t, tg)[1]
    with pytest.raises(ValueError):
        op.loss(h.bfloat16(), t, tg)
    with pytest.raises(ValueError):
        op.loss(h[:, :8], t, tg)
    with pytest.raises(ValueError):
        op.loss(h, t[:39], tg)
    with pytest.raises(ValueError):
        op.loss(h, t, tg.short())
    with pytest.raises(ValueError):
        op.loss(h.T.contiguous().T, t, tg)
    with pytest.raises(ValueError):
        op.grad(h, t, tg, lse.double(), 1.0)
    with pytest.raises(ValueError):
        op.grad(h, t, tg, lse, 1.0, accumulate=True)
    with pytest.raises(ValueError):
        op.loss(torch.cat([h, h]), t, torch.cat([tg, tg]))
    with pytest.raises(ValueError):
        zs.LmLoss(40, 16, "fp16", max_tokens=20, with_grad=False).grad(h, t, tg, lse, 1.0)
    with pytest.raises(zs.ZeroError):
        zs.LmLoss(40, 12, "fp16")
    with pytest.raises(zs.ZeroError):
        op.loss(torch.empty(20, 20, dtype=torch.float16, device="cuda")[:, :16], t, tg)   # rows of 40 bytes


def test_more_tokens_than_one_slab():
    """The loss goes over the tokens in slabs of 32768."""
    h, t, tg = make(33_000, 70, 16, "bf16", seed=8)
    *_, dh, dt, want = check(h, t, tg, scale=1 / 33_000)
    assert ref.rel_norm(dh, want["dhidden"]) <= 2 * ref.HALF_ULP[h.dtype]


@pytest.mark.parametrize("which", ["loss", "grad"])
def test_a_lost_copy_is_reported(which):
    """A block of operands that never arrives: the waits run out, the status
    says so, and the next call works."""
    h, t, tg = make(400, 3000, 640, "bf16")
    op = zs.LmLoss(3000, 640, "bf16", max_tokens=400)
    loss, lse = op.loss(h, t, tg)
    grads = [x.clone() for x in op.grad(h, t, tg, lse, 1.0)]
    op.status()
    zs.zero_lm_inject_stall()
    if which == "loss":
        op.loss(h, t, tg)
    else:
        op.grad(h, t, tg, lse, 1.0)
    with pytest.raises(zs.ZeroError) as e:
        op.status()
    assert e.value.code == zs.ZERO_E_STATE
    op.status()                                   # reported once
    loss2, lse2 = op.loss(h, t, tg)
    assert torch.equal(loss2, loss) and torch.equal(lse2, lse)
    assert all(torch.equal(x, y) for x, y in zip(op.grad(h, t, tg, lse, 1.0), grads))
    op.status()


def test_calls_in_a_cuda_graph():
    """Loss and gradients captured once and replayed on new contents."""
    N, V, d = 300, 5000, 256
    h, t, tg = make(N, V, d, "bf16", seed=21)
    op = zs.LmLoss(V, d, "bf16", max_tokens=N)
    emb = zs.Embedding(V, d, "bf16", max_tokens=N)
    ids = tg.clamp(min=0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def run():
        loss, lse = op.loss(h, t, tg)
        dh, dt = op.grad(h, t, tg, lse, 1.0 / N)
        return loss, dh, emb.grad(ids, dh, dt, accumulate=True), emb.forward(ids, t)

    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = run()
    for seed in (22, 23):
        h2, t2, tg2 = make(N, V, d, "bf16", seed=seed)
        h.copy_(h2), t.copy_(t2), tg.copy_(tg2), ids.copy_(tg2.clamp(min=0))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        assert all(torch.equal(x, y) for x, y in zip(got, run()))


@pytest.mark.parametrize("N", [96, 200])
def test_large_logits_lose_nothing_to_the_change_of_base(N):
    """Two equal logits l, exact in fp32: lse = l + log 2.  Exponents are formed
    in base 2 and back: the two constants' product is within 1.2e-8 of 1, the
    result is rounded once (half a unit in its last place), and the two
    exponentials and the logarithm are good to 1e-6.  A rounding of l log2(e)
    by itself would show here."""
    a = torch.linspace(17, 32, N, device="cuda").half()
    h, t = torch.zeros(N, 8, device="cuda").half(), torch.zeros(2, 8, device="cuda").half()
    h[:, 0], t[:, 0] = a, 31.78125
    want = a.double() * 31.78125 + math.log(2)
    ulp = 2.0 ** (torch.floor(torch.log2(want)) - 23)
    loss, lse = zs.LmLoss(2, 8, "fp16", max_tokens=N).loss(h, t, torch.zeros(N, dtype=torch.int64, device="cuda"))
    ref.assert_within(lse, want, ulp / 2 + want * 1.2e-8 + 1e-6, "lse")
    # the subtraction of the logit is exact (within a factor of 2 of lse)
    ref.assert_within(loss, torch.full_like(want, math.log(2)), ulp / 2 + want * 1.2e-8 + 1e-6, "loss")


def test_four_pieces_of_the_vocabulary():
    """Enough pieces that both buffers of D are used again and dh is added to
    more than once; the last piece is shorter than the others."""
    h, t, tg = make(9000, 25_001, 16, "bf16", seed=4, t_sigma=0.3)
    *_, dh, dt, want = check(h, t, tg, scale=1 / 9000)
    assert ref.rel_norm(dh, want["dhidden"]) <= 2 * ref.HALF_ULP[h.dtype]
    assert ref.rel_norm(dt, want["dtable"]) <= 2 * ref.HALF_ULP[h.dtype]


@pytest.mark.parametrize("tail", [1, 96, 97])
def test_a_short_last_slab(tail):
    """After a slab of 32768 tokens, one small enough for exchanged operands (and one just not)."""
    h, t, tg = make(32_768 + tail, 300, 24, "fp16", seed=tail)
    op = zs.LmLoss(300, 24, "fp16", max_tokens=len(tg), with_grad=False)
    loss, lse = op.loss(h, t, tg)
    op.status()
    want = ref.lm_reference(h, t, tg)
    valid = ref.valid_mask(tg, 300)
    ref.assert_within(loss, want["loss"], want["loss_bound"], "loss")
    ref.assert_within(lse[valid], want["lse"][valid], want["lse_bound"][valid], "lse")
    last = zs.LmLoss(300, 24, "fp16", max_tokens=tail).loss(h[-tail:].contiguous(), t, tg[-tail:].contiguous())
    assert torch.equal(loss[-tail:], last[0]) and torch.equal(lse[-tail:], last[1])


@pytest.mark.parametrize("N,V,d", [(133, 517, 72), (5000, 20_011, 72), (40, 3000, 64)])
def test_a_table_gradient_added_in_fp16(N, V, d):
    """D carries a factor of 2^14 in fp16, which has to be undone before the old value is added."""
    h, t, tg = make(N, V, d, "fp16", seed=N)
    scale = 2048.0 / N
    op = zs.LmLoss(V, d, "fp16", max_tokens=N)
    lse = op.loss(h, t, tg)[1]
    want = ref.lm_reference(h, t, tg, scale)
    old = torch.randn(V, d, device="cuda").half()
    dh, got = op.grad(h, t, tg, lse, scale, dtable=old.clone(), accumulate=True)
    total = want["dtable"] + old.double()
    bound = want["dtable_bound"] + total.abs() * ref.HALF_ULP[h.dtype] + old.double().abs() * 2.0 ** -23
    ref.assert_within(got, total, bound, "accumulated dtable")
    ref.assert_within(dh, want["dhidden"], want["dhidden_bound"], "dhidden")
