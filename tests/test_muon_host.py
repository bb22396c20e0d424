"""Argument checks of the orthogonalised updates, without a GPU: every refusal happens before any CUDA call."""

import pytest

import zero_sharded_mixed_step_gb300 as zs
from tests.test_lm_ops_host import code, fake

CO = zs.MUON_COEFFICIENTS
ORTH = dict(shapes=[(4, 6), (8, 3)], dtype=zs.ZERO_BF16, matrices=[fake(1), fake(2)], in_strides=None,
            out=[fake(3), fake(4)], out_strides=None, coefficients=CO, fine_steps=-1, workspace=fake(5),
            workspace_bytes=1 << 20)
STEP = dict(W=2, shapes=[(4, 6), (8, 3)], grad_dtype=zs.ZERO_FP16, work_dtype=zs.ZERO_BF16,
            grads=[[fake(1), fake(2)], [fake(3), fake(4)]], master=[fake(5), fake(6)], momentum=[fake(7), fake(8)],
            p16=[fake(9), fake(10)], lr=0.1, mu=0.9, nesterov=True, weight_decay=0.0, scales=None, coefficients=CO,
            fine_steps=-1, workspace=fake(11), workspace_bytes=1 << 20)
E = zs.ZERO_E_ARG
COMMON = [("shapes", [(4, 6), (0, 3)], E), ("shapes", [(4, 6), (8, -3)], E), ("shapes", [(4, 6), (8, 32769)], E),
          ("coefficients", (), E), ("coefficients", CO * 7, E), ("coefficients", ((1.0, 65.0, 0.0),), E),
          ("coefficients", ((1.0, float("nan"), 0.0),), E), ("fine_steps", -2, E), ("fine_steps", 6, E),
          ("workspace", None, E), ("workspace", fake(11) + 128, zs.ZERO_E_ALIGN), ("workspace_bytes", 100, E)]


@pytest.mark.parametrize("name,value,want", COMMON + [
    ("dtype", 3, E), ("matrices", [fake(1), None], E), ("matrices", [fake(1) + 1, fake(2)], zs.ZERO_E_ALIGN),
    ("out", [None, fake(4)], E), ("out", [fake(3), fake(4) + 1], zs.ZERO_E_ALIGN), ("in_strides", [5, 3], E),
    ("out_strides", [6, 1 << 33], E), ("in_strides", [-6, 3], E)])
def test_orthogonalize_refusals(zlib, name, value, want):
    assert code(zs.zero_orthogonalize, **dict(ORTH, **{name: value})) == want


@pytest.mark.parametrize("name,value,want", COMMON + [
    ("W", 0, E), ("W", 65, E), ("grad_dtype", zs.ZERO_FP32, E), ("work_dtype", zs.ZERO_FP32, E),
    ("grads", [[fake(1), fake(2)], [fake(3), None]], E),
    ("grads", [[fake(1), fake(2)], [fake(3) + 1, fake(4)]], zs.ZERO_E_ALIGN), ("master", [None, fake(6)], E),
    ("master", [fake(5) + 2, fake(6)], zs.ZERO_E_ALIGN), ("momentum", [fake(7), fake(8) + 2], zs.ZERO_E_ALIGN),
    ("momentum", [fake(7), None], E), ("p16", [fake(9), None], E), ("p16", [fake(9) + 1, fake(10)], zs.ZERO_E_ALIGN),
    ("lr", float("nan"), E), ("lr", 1e60, E), ("mu", 1.0, E), ("mu", -0.1, E), ("mu", float("nan"), E),
    ("weight_decay", float("inf"), E), ("scales", [1.0, float("nan")], E), ("scales", [1e50, 1.0], E)])
def test_step_refusals(zlib, name, value, want):
    assert code(zs.zero_muon_step, **dict(STEP, **{name: value})) == want


def test_nothing_touches_nothing(zlib):
    zs.zero_orthogonalize(**dict(ORTH, shapes=[], matrices=[], out=[], workspace=None, workspace_bytes=0))
    zs.zero_muon_step(**dict(STEP, shapes=[], grads=[[], []], master=[], momentum=[], p16=[], workspace=None,
                             workspace_bytes=0))


def test_workspace(zlib):
    assert code(zs.zero_orthogonalize_workspace_bytes, [(0, 1)]) == E
    assert code(zs.zero_muon_workspace_bytes, 0, [(1, 1)]) == E
    one, two = (zs.zero_orthogonalize_workspace_bytes([(256, 512)] * k) for k in (1, 2))
    assert 256 * 512 * 8 < one < two <= 2 * one
    assert zs.zero_orthogonalize_workspace_bytes([(512, 256)]) == one
    assert zs.zero_muon_workspace_bytes(8, [(256, 512)]) >= zs.zero_muon_workspace_bytes(2, [(256, 512)]) + 256 * 512 * 4
    assert zs.zero_orthogonalize_workspace_bytes([]) > 0


def test_owner_checks(zlib):
    import torch
    op = zs.Orthogonalize([(4, 6)], "bf16", device="cpu")
    x = torch.zeros(4, 6, dtype=torch.bfloat16)
    for bad in ([], [x, x], [x.T], [x.float()], [torch.zeros(4, 12, dtype=torch.bfloat16)[:, ::2]]):
        with pytest.raises(ValueError):
            op.forward(bad)
    with pytest.raises(ValueError):
        op.forward([x], out=[x.half()])
    with pytest.raises(ValueError):
        zs.Orthogonalize([(4, 6)], coefficients=((1.0, 2.0),), device="cpu")
    theta = torch.arange(24.0).view(4, 6)
    step = zs.MuonStep([(4, 6), (3, 3)], 2, "bf16", theta0=[theta, torch.ones(3, 3)], device="cpu")
    assert step.starts == [0, 24] and step.n == 40
    assert torch.equal(step.views(step.master)[0], theta) and torch.equal(step.views(step.p16)[1].float(), torch.ones(3, 3))
    grads = step.new_grad_buffers()
    assert len(grads) == 2 and [tuple(g.shape) for g in grads[0]] == [(4, 6), (3, 3)]
    for bad in (grads[:1], [grads[0], grads[1][:1]], [[g.float() for g in rank] for rank in grads],
                [[g.T.contiguous() for g in rank] for rank in grads]):
        with pytest.raises(ValueError):
            step.step(bad, 0.1)
    with pytest.raises(ValueError):
        zs.MuonStep([(4, 6)], scales=[1.0, 2.0], device="cpu")
