"""The embedding lookup and its gradient against a plain 64-bit form."""

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


def draw(N, V, d, dtype, seed=0, kind="uniform", ids=torch.int64):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "uniform":
        x = torch.randint(0, V, (N,), device="cuda", generator=gen)
    elif kind == "one":
        x = torch.full((N,), V - 1, device="cuda")
    elif kind == "words":
        u = torch.rand(N, device="cuda", generator=gen, dtype=torch.float64)
        x = ((V + 1.0) ** u).long().sub_(1).clamp_(0, V - 1)
    else:
        x = torch.randint(-V, 2 * V, (N,), device="cuda", generator=gen)      # two thirds outside
    rows = torch.randn(N, d, device="cuda", generator=gen).to(DT[dtype])
    table = torch.randn(V, d, device="cuda", generator=gen).to(DT[dtype])
    return x.to(ids), rows, table


CASES = [(1, 1, 8, "uniform"), (1, 50257, 768, "uniform"), (2, 3, 16, "one"), (15, 7, 40, "uniform"),
         (16, 100, 64, "words"), (17, 100, 64, "words"), (31, 300, 2056, "outside"), (33, 255, 8, "one"),
         (64, 256, 264, "words"), (1000, 257, 72, "words"), (4097, 65537, 24, "uniform"), (4096, 5000, 136, "one"),
         (20000, 50257, 48, "words"), (9999, 400, 88, "outside")]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("N,V,d,kind", CASES)
def test_lookup_and_gradient(N, V, d, kind, dtype):
    ids, rows, table = draw(N, V, d, dtype, seed=N, kind=kind, ids=torch.int32 if N % 2 else torch.int64)
    emb = zs.Embedding(V, d, dtype, max_tokens=N, scale=1.7)
    y = emb.forward(ids, table)
    valid = ref.valid_mask(ids, V)
    want = torch.where(valid[:, None], table[torch.where(valid, ids, 0).long()].float() * torch.tensor(1.7).cuda(), 0.0)
    assert torch.equal(y, want.to(DT[dtype]))                   # one fp32 product, one rounding
    got = emb.grad(ids, rows)
    total, bound = ref.embedding_grad_reference(ids, rows, 1.7, V)
    ref.assert_within(got, total, bound, "dtable")
    old = (table * 0.5).contiguous()
    got2 = emb.grad(ids, rows, old.clone(), accumulate=True)
    total, bound = ref.embedding_grad_reference(ids, rows, 1.7, V, old)
    ref.assert_within(got2, total, bound, "accumulated dtable")
    assert torch.equal(emb.grad(ids, rows), got)                # the same bits every time


def test_rows_of_ids_outside_the_table_do_not_matter():
    ids, rows, table = draw(500, 60, 64, "bf16", kind="outside")
    emb = zs.Embedding(60, 64, "bf16", max_tokens=500)
    want = emb.grad(ids, rows)
    rows[~ref.valid_mask(ids, 60)] = float("nan")
    assert torch.equal(emb.grad(ids, rows), want)
    ids[:] = 2 ** 32 + 3         # 3 if it were cut to 32 bits
    assert (emb.grad(ids, rows) == 0).all() and (emb.forward(ids, table) == 0).all()


def test_strides_empty_calls_and_guard_bytes():
    V, d, N = 97, 72, 333
    ids, rows, table = draw(N, V, d, "fp16")
    arena = Arena(32 << 20, "cuda")
    wide_t = arena.zeros(V * (d + 8), torch.float16).view(V, d + 8)
    wide_y = arena.zeros(N * (d + 16), torch.float16).view(N, d + 16)
    wide_r = arena.zeros(N * (d + 24), torch.float16).view(N, d + 24)
    wide_g = arena.zeros(V * (d + 8), torch.float16).view(V, d + 8)
    wide_t[:, 8:].copy_(table), wide_r[:, :d].copy_(rows), wide_g.fill_(9.0), wide_y.fill_(9.0)
    emb = zs.Embedding(V, d, "fp16", max_tokens=N, scale=0.5, alloc=arena)
    plain = zs.Embedding(V, d, "fp16", max_tokens=N, scale=0.5)
    emb.forward(ids, wide_t[:, 8:], out=wide_y[:, 16:])
    emb.grad(ids, wide_r[:, :d], wide_g[:, :d])
    assert torch.equal(wide_y[:, 16:], plain.forward(ids, table)) and (wide_y[:, :16] == 9).all()
    assert torch.equal(wide_g[:, :d], plain.grad(ids, rows)) and (wide_g[:, d:] == 9).all()
    arena.check()
    none = ids[:0]
    assert plain.forward(none, table).shape == (0, d)
    g = torch.ones(V, d, dtype=torch.float16, device="cuda")
    assert (plain.grad(none, rows[:0], g, accumulate=True) == 1).all()
    assert (plain.grad(none, rows[:0], g) == 0).all()


def test_gradient_against_differences():
    """The lookup is linear: its difference along a step is exact in fp32."""
    ids, rows, table = draw(200, 50, 32, "fp16", kind="words")
    rows = (rows * 8).round() / 8
    step = torch.randint(-2, 3, table.shape, device="cuda").half() / 4
    base = torch.randint(-8, 9, table.shape, device="cuda").half() / 4
    emb = zs.Embedding(50, 32, "fp16", max_tokens=200, scale=2.0)
    f = lambda t: (emb.forward(ids, t).double() * rows.double()).sum()  # noqa: E731
    num = (f(base + step) - f(base - step)) / 2
    total, bound = ref.embedding_grad_reference(ids, rows, 2.0, 50)
    ana = (emb.grad(ids, rows).double() * step.double()).sum()
    assert abs(num - ana) <= (bound * step.double().abs()).sum() + 1e-9


def test_refusals():
    ids, rows, table = draw(20, 40, 16, "fp16")
    emb = zs.Embedding(40, 16, "fp16", max_tokens=20)
    with pytest.raises(ValueError):
        emb.forward(ids, table.float())
    with pytest.raises(ValueError):
        emb.forward(ids.float(), table)
    with pytest.raises(ValueError):
        emb.grad(ids, rows[:19])
    with pytest.raises(ValueError):
        emb.grad(ids, rows, accumulate=True)
    with pytest.raises(ValueError):
        emb.grad(torch.cat([ids, ids]), torch.cat([rows, rows]))
    with pytest.raises(zs.ZeroError):
        zs.Embedding(40, 20, "fp16")


@pytest.mark.parametrize("kind", ["words", "uniform", "one", "outside"])
@pytest.mark.parametrize("N", [1, 700, 3000])
def test_rows_that_no_id_names_are_zero_in_a_large_table(N, kind):
    """A table of 61 MB: part of its rows is filled beside the sort, the rest beside the sums."""
    V, d = 59_999, 512
    ids, rows, table = draw(N, V, d, "bf16", seed=N, kind=kind)
    ids[-1] = V - 1
    emb = zs.Embedding(V, d, "bf16", max_tokens=N)
    wide = torch.full((V, d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    total, bound = ref.embedding_grad_reference(ids, rows, 1.0, V)
    got = emb.grad(ids, rows, torch.full((V, d), 5.0, dtype=torch.bfloat16, device="cuda"))
    ref.assert_within(got, total, bound, "dtable")
    emb.grad(ids, rows, wide[:, :d])
    assert torch.equal(wide[:, :d], got) and (wide[:, d:] == 3).all()


def _gradient_time(ids, rows, V):
    """Median device time of the table's gradient, in us."""
    emb = zs.Embedding(V, rows.shape[1], "bf16", max_tokens=len(ids))
    table = torch.empty(V, rows.shape[1], dtype=torch.bfloat16, device="cuda")
    times = []
    for _ in range(13):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda._sleep(200_000)        # the call is queued whole before it runs
        a.record()
        emb.grad(ids, rows, table)
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return sorted(times[3:])[5]


@pytest.mark.parametrize("N,V,d,share", [(65_535, 1 << 20, 64, 1), (47_000, 50_257, 768, 1), (8192, 50_257, 768, 2)])
def test_a_frequent_id_costs_the_same_wherever_it_stands(N, V, d, share):
    """One token in `share` has one id, as padding has: the first of the table, or the last."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(0, V, (N,), device="cuda", generator=gen)
    rows = torch.randn(N, d, device="cuda", generator=gen).bfloat16()
    us = []
    for frequent in (0, V - 1):
        ids[::share] = frequent
        us.append(_gradient_time(ids, rows, V))
    assert us[1] <= 1.3 * us[0] + 3, us
