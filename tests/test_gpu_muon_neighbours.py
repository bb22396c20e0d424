"""A small matrix's result does not depend on the other matrices of the call, which decide how many CTAs a launch
gives each."""

import math

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests.test_gpu_muon import gaussian, make_step

pytestmark = pytest.mark.gpu

SHAPES = [(30, 20), (128, 700), (9, 1500), (64, 64), (700, 128), (1, 1), (128, 256), (257, 16), (100, 2048)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_orthogonalize(dtype):
    xs = [gaussian(*s, seed=k).to(torch.bfloat16 if dtype == "bf16" else torch.float32) for k, s in enumerate(SHAPES)]
    alone = [zs.Orthogonalize([s], dtype).forward([x])[0] for s, x in zip(SHAPES, xs)]
    together = zs.Orthogonalize(SHAPES, dtype).forward(xs)
    many = zs.Orthogonalize(SHAPES * 20, dtype).forward(xs * 20)
    for k, one in enumerate(alone):
        assert torch.equal(one, together[k]), SHAPES[k]
        for copy in (0, 7, 19):
            assert torch.equal(one, many[k + copy * len(SHAPES)]), SHAPES[k]


def test_step():
    scales = [0.2 * math.sqrt(max(s)) for s in SHAPES]
    whole, grads = make_step(SHAPES, 3, "bf16", scales=scales)
    alone = []
    for k, s in enumerate(SHAPES):
        one = zs.MuonStep([s], 3, "bf16", scales=scales[k:k + 1])
        for v, w in ((one.master, whole.master), (one.momentum, whole.momentum)):
            one.views(v)[0].copy_(whole.views(w)[k])
        alone.append(one)
    for _ in range(2):
        whole.step(grads, 0.02)
        for k, one in enumerate(alone):
            one.step([rank[k:k + 1] for rank in grads], 0.02)
    for k, one in enumerate(alone):
        assert torch.equal(one.views(one.master)[0], whole.views(whole.master)[k]), SHAPES[k]
        assert torch.equal(one.views(one.p16)[0], whole.views(whole.p16)[k]), SHAPES[k]
