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


class Devices:
    """Stands for the current device and for torch.cuda.device()."""

    def __init__(self, current):
        self.current, self.entered = current, []

    def get(self):
        return self.current

    def device(self, index):
        import contextlib

        @contextlib.contextmanager
        def scope():
            before, self.current = self.current, index
            self.entered.append(index)
            yield
            self.current = before
        return scope()


def test_calls_run_under_the_owners_device(zlib, monkeypatch):
    """The C entry points launch on the current device: it has to be the owner's at the call."""
    devices, seen = Devices(0), []

    class Library:
        @staticmethod
        def zero_lm_loss(*args):
            seen.append(devices.current)
            return 0

        zero_lm_loss_grad = zero_lm_workspace_status = zero_lm_loss

        @staticmethod
        def zero_lm_workspace_bytes(*args):
            return 256

    monkeypatch.setattr(zs, "lib", lambda: Library)
    monkeypatch.setattr(zs, "_current_device", devices.get)
    monkeypatch.setattr(torch.cuda, "device", devices.device)
    here = zs.LmLoss(40, 16, "fp16", max_tokens=8, device="cuda:0", alloc=on_host)
    there = zs.LmLoss(40, 16, "fp16", max_tokens=8, device="cuda:1", alloc=on_host)
    here._loss(), there._loss(), there._grad(), here._grad()
    assert seen == [0, 1, 1, 0] and devices.current == 0 and devices.entered == [1, 1]


def test_errors_under_another_device_are_raised(zlib, monkeypatch):
    devices = Devices(1)
    monkeypatch.setattr(zs, "_current_device", devices.get)
    monkeypatch.setattr(torch.cuda, "device", devices.device)
    op = zs.LmLoss(40, 16, "fp16", max_tokens=8, device="cuda:0", alloc=on_host)
    with pytest.raises(zs.ZeroError):
        op._loss(-1, 40, 16, zs.ZERO_FP16, None, 16, None, 16, None, 8, None, None, None, 0, None)
    assert devices.entered == [0] and devices.current == 1


def test_the_norms_workspace_is_zero_whatever_alloc_returns(zlib):
    """Its count of finished blocks has to start at 0."""
    op = clip_owner([4, 5])
    assert op.workspace.numel() == zs.zero_grad_norm_workspace_bytes() and (op.workspace == 0).all()


def test_the_loss_owners_count_of_failures_starts_at_zero(zlib):
    op = zs.LmLoss(40, 16, "fp16", max_tokens=8, device="cuda:0", alloc=on_host)
    assert (op.workspace[:4] == 0).all()


def test_workspace_status_refusals(zlib):
    for workspace, want in ((None, zs.ZERO_E_ARG), (0x7F0000000080, zs.ZERO_E_ALIGN)):
        with pytest.raises(zs.ZeroError) as e:
            zs.zero_lm_workspace_status(workspace)
        assert e.value.code == want


@pytest.mark.parametrize("W,keeps_mean", [(1, False), (2, False), (3, True), (8, True)])
def test_the_clipped_steps_workspace_holds_a_mean_only_where_one_is_written(zlib, W, keeps_mean):
    """With 1 and 2 ranks the update reads the gradients again."""
    n, norm = 1_000_003, zs.zero_grad_norm_workspace_bytes()
    fake = 0x7F0000000000
    ctx = zs.zero_init(zs.ZERO_SCHEME_Z1, W, n, [n], 0, 0, fake, fake + (1 << 30), fake + (2 << 30), fake + (3 << 30))
    nbytes = zs.zero_step_clipped_workspace_bytes(ctx)
    assert (nbytes >= norm + 4 * n) if keeps_mean else (nbytes == norm)
    zs.zero_destroy(ctx)
