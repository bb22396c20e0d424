"""The operators on a table of more than 2^31 values: offsets past 32 bits."""

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests import lm_reference as ref

pytestmark = pytest.mark.gpu

V, D = 1_400_000, 1600          # 2.24e9 values


@pytest.fixture(scope="module")
def table():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    gen = torch.Generator(device="cuda").manual_seed(1)
    t = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, V, 100_000):
        t[lo:lo + 100_000] = torch.randn(100_000, D, device="cuda", generator=gen) * 0.05
    return t


IDS = [0, V - 1, V - 2, V - 1, 1_342_177, 1_342_178, 700_000, V]


def test_lookup(table):
    ids = torch.tensor(IDS, device="cuda")
    got = zs.Embedding(V, D, "bf16", max_tokens=8).forward(ids, table)
    assert torch.equal(got[:-1], table[ids[:-1]]) and (got[-1] == 0).all()


@pytest.mark.parametrize("accumulate", [False, True])
def test_lookup_gradient(table, accumulate):
    ids = torch.tensor(IDS, device="cuda")
    rows = torch.randn(8, D, device="cuda").bfloat16()
    got = table.clone() if accumulate else torch.full_like(table, 3.0)
    zs.Embedding(V, D, "bf16", max_tokens=8).grad(ids, rows, got, accumulate=accumulate)
    named = sorted(set(IDS[:-1]))
    at = torch.tensor(named, device="cuda")
    where = {v: k for k, v in enumerate(named)}
    local = torch.tensor([where.get(v, -1) for v in IDS], device="cuda")
    old = table[at] if accumulate else None
    want, bound = ref.embedding_grad_reference(local, rows, 1.0, len(named), old)
    ref.assert_within(got[at], want, bound, "named rows")
    got[at] = table[at] if accumulate else 0
    for lo in range(0, V, 100_000):
        part = got[lo:lo + 100_000]
        assert torch.equal(part, table[lo:lo + 100_000]) if accumulate else not part.any()


@pytest.mark.parametrize("N", [5, 130])
def test_loss_and_gradients(table, N):
    gen = torch.Generator(device="cuda").manual_seed(N)
    h = torch.randn(N, D, device="cuda", generator=gen).bfloat16()
    tg = torch.randint(0, V, (N,), device="cuda", generator=gen)
    tg[0], tg[1], tg[2] = V - 1, 1_342_178, -1
    op = zs.LmLoss(V, D, "bf16", max_tokens=N)
    loss, lse = op.loss(h, table, tg)
    dh, dt = op.grad(h, table, tg, lse, 1.0)
    op.status()
    # the 64-bit form over stretches of the vocabulary
    h64, valid = h.double(), tg >= 0
    parts, picked = [], torch.zeros(N, dtype=torch.float64, device="cuda")
    for lo in range(0, V, 100_000):
        l = h64 @ table[lo:lo + 100_000].double().T
        parts.append(torch.logsumexp(l, 1))
        here = valid & (tg >= lo) & (tg < lo + 100_000)
        picked[here] = l[here, tg[here] - lo]
    want = torch.logsumexp(torch.stack(parts), 0)
    # sums of 1600 products in the tensor core, each step truncated: 105 roundings of 2^-23 of at most 200 in all
    tol = 105 * 2.0 ** -23 * 200 + 20 * 2.0 ** -22
    assert ((lse.double() - want).abs() <= tol).all()
    assert ((loss.double() - torch.where(valid, want - picked, 0.0)).abs() <= 2 * tol).all() and loss[2] == 0
    dh64 = torch.zeros(N, D, dtype=torch.float64, device="cuda")
    u = ref.HALF_ULP[torch.bfloat16]
    for lo in range(0, V, 100_000):
        t64 = table[lo:lo + 100_000].double()
        d = torch.exp(h64 @ t64.T - want[:, None])
        here = valid & (tg >= lo) & (tg < lo + 100_000)
        d[here, tg[here] - lo] -= 1.0
        d *= valid[:, None]
        dh64 += d @ t64
        if lo in (0, 1_300_000):
            assert ref.rel_norm(dt[lo:lo + 100_000], d.T @ h64) <= 2 * u
    assert ref.rel_norm(dh, dh64) <= 2 * u and (dh[2] == 0).all()
