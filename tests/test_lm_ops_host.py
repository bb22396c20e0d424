"""Argument checks of the language-model operators, without a GPU: every refusal
happens before any CUDA call."""

import pytest

import zero_sharded_mixed_step_gb300 as zs

A = 0x7F0000000000          # fake device addresses


def fake(k):
    return A + k * (1 << 30)


def code(fn, *args, **kw):
    with pytest.raises(zs.ZeroError) as e:
        fn(*args, **kw)
    return e.value.code


LOSS = dict(tokens=4, vocab=10, width=16, dtype=zs.ZERO_FP16, hidden=fake(1), hidden_stride=16, table=fake(2),
            table_stride=16, targets=fake(3), id_bytes=8, loss=fake(4), lse=fake(5), workspace=fake(6),
            workspace_bytes=1 << 20)
GRAD = dict({k: v for k, v in LOSS.items() if k != "loss"}, scale=1.0, dhidden=fake(7), dhidden_stride=16,
            dtable=fake(8), dtable_stride=16, accumulate=0)
COMMON_BAD = [("tokens", -1, zs.ZERO_E_ARG), ("tokens", (1 << 24) + 1, zs.ZERO_E_ARG), ("vocab", 0, zs.ZERO_E_ARG),
              ("vocab", (1 << 24) + 1, zs.ZERO_E_ARG), ("width", 0, zs.ZERO_E_ARG), ("width", 12, zs.ZERO_E_ARG),
              ("width", 1 << 17, zs.ZERO_E_ARG), ("dtype", zs.ZERO_FP32, zs.ZERO_E_ARG), ("id_bytes", 2, zs.ZERO_E_ARG),
              ("hidden", None, zs.ZERO_E_ARG), ("hidden", fake(1) + 8, zs.ZERO_E_ALIGN),
              ("hidden_stride", 8, zs.ZERO_E_ARG), ("hidden_stride", 20, zs.ZERO_E_ALIGN), ("table", None, zs.ZERO_E_ARG),
              ("table_stride", 8, zs.ZERO_E_ARG), ("table_stride", 1 << 33, zs.ZERO_E_ARG),
              ("targets", None, zs.ZERO_E_ARG), ("targets", fake(3) + 4, zs.ZERO_E_ALIGN),
              ("lse", None, zs.ZERO_E_ARG), ("lse", fake(5) + 2, zs.ZERO_E_ALIGN), ("workspace", None, zs.ZERO_E_ARG),
              ("workspace", fake(6) + 128, zs.ZERO_E_ALIGN), ("workspace_bytes", 100, zs.ZERO_E_ARG)]


@pytest.mark.parametrize("name,value,want", COMMON_BAD + [("loss", None, zs.ZERO_E_ARG)])
def test_loss_refusals(zlib, name, value, want):
    assert code(zs.zero_lm_loss, **dict(LOSS, **{name: value})) == want


@pytest.mark.parametrize("name,value,want", COMMON_BAD + [
    ("scale", float("nan"), zs.ZERO_E_ARG), ("scale", 1e60, zs.ZERO_E_ARG), ("dhidden", None, zs.ZERO_E_ARG),
    ("dhidden_stride", 8, zs.ZERO_E_ARG), ("dtable", None, zs.ZERO_E_ARG), ("dtable", fake(8) + 2, zs.ZERO_E_ALIGN),
    ("dtable_stride", 17, zs.ZERO_E_ALIGN)])
def test_loss_grad_refusals(zlib, name, value, want):
    assert code(zs.zero_lm_loss_grad, **dict(GRAD, **{name: value})) == want


def test_loss_of_nothing_touches_nothing(zlib):
    zs.zero_lm_loss(**dict(LOSS, tokens=0))
    zs.zero_lm_loss_grad(**dict(GRAD, tokens=0, accumulate=1))


def test_lm_workspace(zlib):
    assert code(zs.zero_lm_workspace_bytes, -1, 10, 16) == zs.ZERO_E_ARG
    assert code(zs.zero_lm_workspace_bytes, 4, 10, 12) == zs.ZERO_E_ARG
    last = 0
    for tokens in (0, 1, 100, 5000, 8192, 100_000):
        small, full = (zs.zero_lm_workspace_bytes(tokens, 50257, 768, g) for g in (False, True))
        assert 256 <= small <= full and full >= last
        last = full
    # never the logits: 8192 tokens of 50257 fp32 values would be 1.65 GB
    assert zs.zero_lm_workspace_bytes(8192, 50257, 768) < 8192 * 50257 * 4 / 4


EMB = dict(tokens=4, vocab=10, width=16, dtype=zs.ZERO_BF16, ids=fake(1), id_bytes=4, table=fake(2), table_stride=16,
           scale=1.0, out=fake(3), out_stride=16)
EMB_GRAD = dict(tokens=4, vocab=10, width=16, dtype=zs.ZERO_BF16, ids=fake(1), id_bytes=4, dout=fake(2),
                dout_stride=16, scale=1.0, dtable=fake(3), dtable_stride=16, accumulate=0, workspace=fake(4),
                workspace_bytes=1 << 20)
EMB_BAD = [("tokens", -1, zs.ZERO_E_ARG), ("tokens", (1 << 24) + 1, zs.ZERO_E_ARG), ("vocab", 0, zs.ZERO_E_ARG),
           ("width", 12, zs.ZERO_E_ARG), ("dtype", 7, zs.ZERO_E_ARG), ("ids", None, zs.ZERO_E_ARG),
           ("ids", fake(1) + 2, zs.ZERO_E_ALIGN), ("id_bytes", 1, zs.ZERO_E_ARG), ("scale", float("inf"), zs.ZERO_E_ARG)]


@pytest.mark.parametrize("name,value,want", EMB_BAD + [
    ("table", None, zs.ZERO_E_ARG), ("table", fake(2) + 8, zs.ZERO_E_ALIGN), ("table_stride", 15, zs.ZERO_E_ARG),
    ("table_stride", 18, zs.ZERO_E_ALIGN), ("out", None, zs.ZERO_E_ARG), ("out_stride", 8, zs.ZERO_E_ARG)])
def test_embedding_refusals(zlib, name, value, want):
    assert code(zs.zero_embedding, **dict(EMB, **{name: value})) == want


@pytest.mark.parametrize("name,value,want", EMB_BAD + [
    ("dout", None, zs.ZERO_E_ARG), ("dout_stride", 15, zs.ZERO_E_ARG), ("dtable", None, zs.ZERO_E_ARG),
    ("dtable", fake(3) + 2, zs.ZERO_E_ALIGN), ("workspace", None, zs.ZERO_E_ARG),
    ("workspace", fake(4) + 16, zs.ZERO_E_ALIGN), ("workspace_bytes", 64, zs.ZERO_E_ARG)])
def test_embedding_grad_refusals(zlib, name, value, want):
    assert code(zs.zero_embedding_grad, **dict(EMB_GRAD, **{name: value})) == want


def test_embedding_of_nothing_touches_nothing(zlib):
    zs.zero_embedding(**dict(EMB, tokens=0))
    zs.zero_embedding_grad(**dict(EMB_GRAD, tokens=0, accumulate=1))
    assert zs.zero_embedding_workspace_bytes(0, 16) >= 256
    assert code(zs.zero_embedding_workspace_bytes, -1, 16) == zs.ZERO_E_ARG
    assert code(zs.zero_embedding_workspace_bytes, 4, 20) == zs.ZERO_E_ARG


NORM = dict(W=2, numels=[5, 0], dtype=zs.ZERO_BF16, grads=[fake(1), None, fake(2), None], norm=fake(3),
            workspace=fake(4), workspace_bytes=1 << 20)
CLIP = dict(W=2, numels=[5, 0], dtype=zs.ZERO_BF16, grads=[fake(1), None, fake(2), None], norm=fake(3), max_norm=1.0,
            out=[fake(5), None])
LIST_BAD = [("W", 0, zs.ZERO_E_ARG), ("W", 65, zs.ZERO_E_ARG), ("dtype", 3, zs.ZERO_E_ARG),
            ("numels", [-1, 0], zs.ZERO_E_ARG), ("grads", [None, None, fake(2), None], zs.ZERO_E_ARG),
            ("grads", [fake(1), None, fake(2) + 1, None], zs.ZERO_E_ALIGN), ("norm", None, zs.ZERO_E_ARG),
            ("norm", fake(3) + 2, zs.ZERO_E_ALIGN)]


@pytest.mark.parametrize("name,value,want", LIST_BAD + [
    ("workspace", None, zs.ZERO_E_ARG), ("workspace", fake(4) + 32, zs.ZERO_E_ALIGN),
    ("workspace_bytes", zs.ZERO_BF16, zs.ZERO_E_ARG)])
def test_grad_norm_refusals(zlib, name, value, want):
    if name == "numels":
        value = [2 ** 64 - 1, 0]        # -1 as the 64-bit word that crosses the ABI
    assert code(zs.zero_grad_norm, **dict(NORM, **{name: value})) == want


@pytest.mark.parametrize("name,value,want", LIST_BAD + [
    ("max_norm", 0.0, zs.ZERO_E_ARG), ("max_norm", float("nan"), zs.ZERO_E_ARG), ("max_norm", 1e50, zs.ZERO_E_ARG),
    ("out", [None, None], zs.ZERO_E_ARG), ("out", [fake(5) + 1, None], zs.ZERO_E_ALIGN)])
def test_grad_clip_refusals(zlib, name, value, want):
    if name == "numels":
        value = [2 ** 64 - 1, 0]
    assert code(zs.zero_grad_clip, **dict(CLIP, **{name: value})) == want


def test_clipped_step_refusals(zlib):
    ctx = zs.zero_init(1, 4, 37, [37], 0, 0, fake(1), fake(2), fake(3), fake(4))
    nbytes = zs.zero_step_clipped_workspace_bytes(ctx)
    assert nbytes >= 4 * 40
    ok = dict(ctx=ctx, scheme=1, W=4, n=37, grads=[fake(10 + r) for r in range(4)], lr=1e-3, beta1=0.9, beta2=0.95,
              eps=1e-8, t=1, max_norm=1.0, norm=fake(5), workspace=fake(6), workspace_bytes=nbytes)
    for name, value, want in (("max_norm", 0.0, zs.ZERO_E_ARG), ("max_norm", -1.0, zs.ZERO_E_ARG),
                              ("max_norm", float("inf"), zs.ZERO_E_ARG), ("max_norm", float("nan"), zs.ZERO_E_ARG),
                              ("max_norm", 1e-60, zs.ZERO_E_ARG), ("norm", None, zs.ZERO_E_ARG),
                              ("norm", fake(5) + 1, zs.ZERO_E_ALIGN), ("workspace", None, zs.ZERO_E_ARG),
                              ("workspace", fake(6) + 128, zs.ZERO_E_ALIGN), ("workspace_bytes", nbytes - 1, zs.ZERO_E_ARG),
                              ("t", 2, zs.ZERO_E_STATE), ("n", 36, zs.ZERO_E_ARG), ("eps", 0.0, zs.ZERO_E_ARG),
                              ("grads", [fake(10) + 8, fake(11), fake(12), fake(13)], zs.ZERO_E_ALIGN)):
        assert code(zs.zero_step_clipped, **dict(ok, **{name: value})) == want, name
    zs.zero_mark_rank(ctx, 2, False)
    assert code(zs.zero_step_clipped, **ok) == zs.ZERO_E_RANK
    zs.zero_destroy(ctx)
    assert code(zs.zero_step_clipped, **dict(ok, ctx=None)) == zs.ZERO_E_ARG
