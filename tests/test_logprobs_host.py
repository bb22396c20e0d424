"""Argument checks of the log probabilities, without a GPU: every refusal happens before any CUDA call."""

import pytest

import zero_sharded_mixed_step_gb300 as zs
from tests.test_lm_ops_host import COMMON_BAD, code, fake

FORWARD = dict(tokens=4, vocab=10, width=16, dtype=zs.ZERO_FP16, hidden=fake(1), hidden_stride=16, table=fake(2),
               table_stride=16, targets=fake(3), id_bytes=8, scale=1.0, top=2, logp=fake(4), entropy=fake(9),
               lse=fake(5), top_logp=fake(10), top_ids=fake(11), workspace=fake(6), workspace_bytes=1 << 20)
GRAD = dict({k: v for k, v in FORWARD.items() if k not in ("top", "logp", "entropy", "lse", "top_logp", "top_ids",
                                                          "workspace", "workspace_bytes")},
            lse=fake(5), dlogp=fake(12), entropy=fake(9), dentropy=fake(13), dhidden=fake(7), dhidden_stride=16,
            dtable=fake(8), dtable_stride=16, accumulate=0, workspace=fake(6), workspace_bytes=1 << 20)
SCALES = [("scale", x, zs.ZERO_E_ARG) for x in (0.0, -1.0, float("nan"), float("inf"), 1e60, 3e38, 1e-60)]


@pytest.mark.parametrize("name,value,want", COMMON_BAD + SCALES + [
    ("logp", None, zs.ZERO_E_ARG), ("logp", fake(4) + 1, zs.ZERO_E_ALIGN), ("entropy", None, zs.ZERO_E_ARG),
    ("entropy", fake(9) + 2, zs.ZERO_E_ALIGN), ("top", -1, zs.ZERO_E_ARG), ("top", 17, zs.ZERO_E_ARG),
    ("top", 11, zs.ZERO_E_ARG), ("top_logp", None, zs.ZERO_E_ARG), ("top_ids", None, zs.ZERO_E_ARG),
    ("top_ids", fake(11) + 2, zs.ZERO_E_ALIGN)])
def test_refusals(zlib, name, value, want):
    assert code(zs.zero_lm_logprobs, **dict(FORWARD, **{name: value})) == want


@pytest.mark.parametrize("name,value,want", COMMON_BAD + SCALES + [
    ("dlogp", None, zs.ZERO_E_ARG), ("dlogp", fake(12) + 2, zs.ZERO_E_ALIGN), ("entropy", None, zs.ZERO_E_ARG),
    ("dentropy", fake(13) + 2, zs.ZERO_E_ALIGN), ("dhidden", None, zs.ZERO_E_ARG), ("dhidden_stride", 8, zs.ZERO_E_ARG),
    ("dtable", None, zs.ZERO_E_ARG), ("dtable", fake(8) + 2, zs.ZERO_E_ALIGN), ("dtable_stride", 17, zs.ZERO_E_ALIGN)])
def test_grad_refusals(zlib, name, value, want):
    assert code(zs.zero_lm_logprobs_grad, **dict(GRAD, **{name: value})) == want


def test_nothing_touches_nothing(zlib):
    zs.zero_lm_logprobs(**dict(FORWARD, tokens=0))
    zs.zero_lm_logprobs_grad(**dict(GRAD, tokens=0, accumulate=1))


def test_workspace(zlib):
    assert code(zs.zero_lm_logprobs_workspace_bytes, -1, 10, 16) == zs.ZERO_E_ARG
    assert code(zs.zero_lm_logprobs_workspace_bytes, 4, 10, 16, 11) == zs.ZERO_E_ARG
    for with_grad in (False, True):
        last = 0
        for tokens in (0, 1, 96, 97, 5000, 100_000):
            for top in (0, 8, 16):
                assert zs.zero_lm_logprobs_workspace_bytes(tokens, 50257, 768, top, with_grad) >= \
                    zs.zero_lm_logprobs_workspace_bytes(tokens, 50257, 768, 0, with_grad)
            assert zs.zero_lm_logprobs_workspace_bytes(tokens, 50257, 768, 16, with_grad) >= last
            last = zs.zero_lm_logprobs_workspace_bytes(tokens, 50257, 768, 16, with_grad)
    # the logits of a large batch are not kept
    assert zs.zero_lm_logprobs_workspace_bytes(8192, 50257, 768, 16, False) < 8192 * 50257 * 4 / 50


def test_owner_checks(zlib):
    import torch
    op = zs.LmLogprobs(10, 16, "bf16", max_tokens=4, top=2, with_grad=False, device="cpu")
    h, t = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(10, 16, dtype=torch.bfloat16)
    tg = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        op.logprobs(torch.zeros(5, 16, dtype=torch.bfloat16), t, torch.zeros(5, dtype=torch.int64))
    with pytest.raises(ValueError):
        op.logprobs(h.half(), t, tg)
    with pytest.raises(ValueError):
        op.logprobs(h, t, tg.float())
    with pytest.raises(ValueError):
        op.grad(h, t, tg, torch.zeros(4), torch.zeros(4))
    op = zs.LmLogprobs(10, 16, "bf16", max_tokens=4, device="cpu")
    with pytest.raises(ValueError):
        op.grad(h, t, tg, torch.zeros(4), torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        op.grad(h, t, tg, torch.zeros(4), torch.zeros(4), dentropy=torch.zeros(4))
    with pytest.raises(ValueError):
        op.grad(h, t, tg, torch.zeros(4), torch.zeros(4), accumulate=True)
    with pytest.raises(zs.ZeroError):
        zs.LmLogprobs(10, 16, "bf16", top=17, device="cpu")
