"""The log probabilities on a table of more than 2^31 values, and long and large matrices: offsets past 32 bits."""

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests import lm_reference as lm
from tests import muon_reference as ref

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
        t[lo:lo + 100_000] = torch.randn(100_000, D, device="cuda", generator=gen) * 0.02
    return t


@pytest.mark.parametrize("N", [5, 130])
def test_logprobs(table, N):
    gen = torch.Generator(device="cuda").manual_seed(N)
    h = torch.randn(N, D, device="cuda", generator=gen).bfloat16()
    tg = torch.randint(0, V, (N,), device="cuda", generator=gen)
    tg[0], tg[1], tg[2] = V - 1, 1_342_178, -1
    # rows far up that answer to one hidden vector each, among the likeliest therefore
    table[V - 1] = h[3] * 0.02
    table[1_342_177] = h[4] * 0.02
    op = zs.LmLogprobs(V, D, "bf16", max_tokens=N, top=4)
    logp, entropy, lse, values, ids = op.logprobs(h, table, tg)
    dh, dt = op.grad(h, table, tg, lse, torch.ones(N, device="cuda"), entropy, torch.full((N,), 0.1, device="cuda"))
    op.status()
    assert ids[3, 0] == V - 1 and ids[4, 0] == 1_342_177
    h64 = h.double()
    parts, best = [], []
    for lo in range(0, V, 100_000):
        l = h64 @ table[lo:lo + 100_000].double().T
        parts.append(torch.logsumexp(l, 1))
        best.append(torch.topk(l, 4, dim=1).values)
    want = torch.logsumexp(torch.stack(parts), 0)
    # sums of 1600 products, each step truncated (105 roundings of 2^-23 of at most 200 in all), and of exponentials
    tol = 105 * 2.0 ** -23 * 200 + 20 * 2.0 ** -22 + (V / 64 + 100) * 2.0 ** -24
    assert ((lse.double() - want).abs() <= tol).all()
    top = torch.topk(torch.cat(best, 1), 4, dim=1).values - want[:, None]
    assert ((values.double() - top).abs() <= 2 * tol).all()
    H = torch.zeros(N, dtype=torch.float64, device="cuda")
    picked = torch.zeros_like(H)
    valid = tg >= 0
    for lo in range(0, V, 100_000):
        logs = h64 @ table[lo:lo + 100_000].double().T - want[:, None]
        H -= (logs.exp() * logs).sum(1)
        here = valid & (tg >= lo) & (tg < lo + 100_000)
        picked[here] = logs[here, tg[here] - lo]
    assert ((entropy.double() - H).abs() <= (2 * H + 2) * 2 * tol).all()
    assert ((logp.double() - torch.where(valid, picked, 0.0)).abs() <= 2 * tol).all() and logp[2] == 0
    u = lm.HALF_ULP[torch.bfloat16]
    dh64 = torch.zeros(N, D, dtype=torch.float64, device="cuda")
    for lo in range(0, V, 100_000):
        t64 = table[lo:lo + 100_000].double()
        logs = h64 @ t64.T - want[:, None]
        p = logs.exp()
        d = -p - 0.1 * p * (logs + H[:, None])
        here = valid & (tg >= lo) & (tg < lo + 100_000)
        d[here, tg[here] - lo] += 1.0
        d *= valid[:, None]
        dh64 += d @ t64
        if lo in (0, 1_300_000):
            assert lm.rel_norm(dt[lo:lo + 100_000], d.T @ h64) <= 2 * u
    assert lm.rel_norm(dh, dh64) <= 2 * u and (dh[2] == 0).all()


@pytest.mark.parametrize("rows,cols", [(1, 32768), (32768, 2), (130, 9000), (20_000, 200), (3001, 2999)])
def test_long_matrices(rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols, device="cuda", generator=gen).bfloat16()
    op = zs.Orthogonalize([(rows, cols)], "bf16")
    got = op.forward([x])[0]
    op.status()
    want = ref.orthogonal(x)
    ref.assert_near(got, want, ref.tolerance(x, want, ref.COEFFICIENTS, 2, 1) + 2.0 ** -8, f"{rows}x{cols}")


def test_a_matrix_of_more_than_2_31_bytes_a_part():
    """One part of X alone holds 1.1e9 values."""
    rows, cols = 32768, 32768
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    # blocks along the diagonal, the last at the far end: each block's result is its own, at the whole norm
    for at in (0, 16_384, rows - 512):
        x[at:at + 512, at:at + 512] = torch.randn(512, 512, device="cuda", generator=gen)
    co = ref.COEFFICIENTS[:2]
    op = zs.Orthogonalize([(rows, cols)], "bf16", coefficients=co, fine_steps=1)
    got = op.forward([x])[0]
    op.status()
    norm = torch.linalg.vector_norm(x, dtype=torch.float64)
    left = got.clone()
    for at in (0, 16_384, rows - 512):
        block = x[at:at + 512, at:at + 512].double()
        share = torch.linalg.vector_norm(block) / norm
        want = block / norm
        for a, b, c in co:
            gram = want @ want.T
            want = a * want + (b * gram + c * gram @ gram) @ want
        assert share > 0.1
        # one fine step and one of one part: three operands rounded by half a step of fp16, their errors' sizes added
        assert lm.rel_norm(got[at:at + 512, at:at + 512], want) <= 2.0 ** -8 + 4 * 3 * 2.0 ** -11
        left[at:at + 512, at:at + 512] = 0
    assert not left.any()
