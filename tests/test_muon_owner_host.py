"""What MuonStep takes as its first parameters, without a GPU."""

import pytest

import zero_sharded_mixed_step_gb300 as zs


def test_theta0_has_to_fit(zlib):
    import torch
    shapes = [(4, 6), (3, 3)]
    right = [torch.arange(24.0).view(4, 6), torch.ones(3, 3)]
    step = zs.MuonStep(shapes, 2, "bf16", theta0=right, device="cpu")
    assert all(torch.equal(a, b) for a, b in zip(step.views(step.master), right))
    step = zs.MuonStep(shapes, 2, "bf16", theta0=[x.tolist() for x in right], device="cpu")
    assert all(torch.equal(a, b) for a, b in zip(step.views(step.master), right))
    # fewer, more, and what would be spread over a matrix
    for bad in (right[:1], right + [torch.ones(3, 3)], [], [right[0], torch.ones(3)], [right[0], torch.ones(3, 1)],
                [right[0], 1.0], [right[0].T, right[1]], [right[0].reshape(-1), right[1]]):
        with pytest.raises(ValueError, match="theta0"):
            zs.MuonStep(shapes, 2, "bf16", theta0=bad, device="cpu")
