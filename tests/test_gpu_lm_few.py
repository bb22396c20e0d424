"""Log probabilities on both sides of the counts of tokens at which the operands change places."""

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests.test_gpu_lm_logprobs import check, check_grad, in_order, make, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("N", [95, 96, 97, 112, 127, 128, 129, 160])
def test_around_the_limits(N, dtype):
    for V, d in ((40, 8), (3001, 72), (20_011, 136)):
        h, t, tg = make(N, V, d, dtype, seed=N, grid=True)
        for top in (0, 1, 8, 16):
            got, want = check(h, t, tg, scale=1.25, top=top, what=f"{N} {V} {top}")
            if top:
                assert torch.equal(got[4].long(), in_order(want["logits"], top))


@pytest.mark.parametrize("top", [0, 5, 16])
def test_one_workspace_for_all_counts(top):
    """An owner of many tokens on both sides of every limit, one call after another."""
    V, d = 2000, 64
    h, t, tg = make(40_000, V, d, "bf16", seed=1)
    op = zs.LmLogprobs(V, d, "bf16", max_tokens=40_000, top=top, with_grad=False)
    for N in (40_000, 128, 32768 + 128, 97, 129, 1, 32768 + 129):
        check(h[:N], t, tg[:N], top=top, op=op, what=f"{N}")


@pytest.mark.parametrize("N", [1023, 1024, 1025, 4097])
def test_the_largest_weight(N):
    """In fp16 D is scaled by its largest bound, which one block or many find; it stands at either end."""
    h, t, tg = make(N, 300, 64, "fp16", seed=N, ignored=0.0)
    for at in (0, N - 1):
        a, b = weights(N, unit=1e-3)
        a[at] = 4.0
        check_grad(h, t, tg, a, b, what=f"{N} {at}")
