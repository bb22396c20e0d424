"""What the owners of the language-model operators refuse and prepare before
anything reaches a GPU."""

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs


def on_host(numel, dtype):
    return torch.full((numel * dtype.itemsize,), 0xFF, dtype=torch.uint8).view(dtype)


def clip_owner(numels, W=1, dtype="fp16", **kw):
    return zs.GradClip(numels, W, dtype, device="cuda:0", alloc=on_host, **kw)


def test_gradients_on_the_host_are_refused(zlib):
    op = clip_owner([4, 5], W=2)
    grads = [[torch.zeros(4).half(), torch.zeros(5).half()] for _ in range(2)]
    with pytest.raises(ValueError, match="cuda:0"):
        op.norm(grads)
    with pytest.raises(ValueError, match="cuda:0"):
        op.norm_and_clip(grads, 1.0)
    with pytest.raises(ValueError, match="cuda:0"):
        op.norm([[x.to("meta") for x in rank] for rank in grads])


def test_lists_of_unequal_ranks_are_refused(zlib):
    op = clip_owner([4, 5], W=2)
    a, b = torch.zeros(4).half(), torch.zeros(5).half()
    for grads in ([[a, b, a], [b]], [[a], [b, a, b]], [[a, b, a, b], []]):
        with pytest.raises(ValueError, match="2 lists"):
            op.norm(grads)


class Placed(zs.GradClip):
    """An owner past the check of its gradients."""

    def _pointers(self, grads):
        return zs._u64_array([0] * len(self._expected))


@pytest.mark.parametrize("norm", [torch.zeros(1), torch.zeros(1, dtype=torch.float64), torch.zeros(2),
                                  torch.zeros(1).half(), torch.zeros(0)])
def test_a_norm_that_is_not_one_value_on_the_device_is_refused(zlib, norm):
    op = Placed([4], 1, "fp16", device="cuda:0", alloc=on_host)
    with pytest.raises(ValueError, match="norm"):
        op.clip([[None]], norm, 1.0, out=torch.zeros(4).half())


def test_an_output_on_the_host_is_refused(zlib, monkeypatch):
    op = Placed([4], 1, "fp16", device="cuda:0", alloc=on_host)
    monkeypatch.setattr(op, "_raw_stream", lambda: None)
    monkeypatch.setattr(op, "_norm", lambda *a: None)
    with pytest.raises(ValueError, match="out"):
        op.norm_and_clip([[None]], 1.0, out=torch.zeros(4).half())


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_matrices_ids_and_vectors_off_the_device_are_refused(zlib, device):
    op = zs.LmLoss(40, 16, "fp16", max_tokens=8, device="cuda:0", alloc=on_host)
    emb = zs.Embedding(40, 16, "fp16", max_tokens=8, device="cuda:0", alloc=on_host)
    h, t = torch.zeros(8, 16, device=device).half(), torch.zeros(40, 16, device=device).half()
    ids = torch.zeros(8, dtype=torch.int64, device=device)
    with pytest.raises(ValueError, match="cuda:0"):
        op.loss(h, t, ids)
    with pytest.raises(ValueError, match="cuda:0"):
        op._vector(torch.zeros(8, device=device), 8)
    with pytest.raises(ValueError, match="cuda:0"):
        emb.forward(ids, t)
    with pytest.raises(ValueError, match="cuda:0"):
        emb.grad(ids, h)
    with pytest.raises(ValueError, match="cuda:0"):
        zs._ids(ids, "tokens", op.device)
