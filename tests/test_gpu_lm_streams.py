"""The owners' workspaces where the current stream changes between calls: the
work on one stream follows that on the other, and the allocator does not hand
the memory out again while either uses it."""

import pytest
import torch

import zero_sharded_mixed_step_gb300 as zs
from tests import lm_reference as ref

pytestmark = pytest.mark.gpu

DELAY = 200_000_000         # cycles of a sleeping kernel: some 0.1 s, longer than the host takes over a test
LR, B1, B2, EPS = 1e-3, 0.9, 0.95, 1e-8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from zero_sharded_mixed_step_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def test_a_norm_on_another_stream_than_the_owner_was_made_on():
    """The fill of the workspace is still to run when the first call is made."""
    g = [torch.randn(50_000, device="cuda").half() * 0.01]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    nbytes = zs.zero_grad_norm_workspace_bytes()
    with torch.cuda.stream(a):
        dirty = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(DELAY)
        del dirty                       # the owner gets this memory
        op = zs.GradClip([50_000], 1, "fp16")
    with torch.cuda.stream(b):
        norm, out = op.norm_and_clip([g], 0.1)
    torch.cuda.synchronize()
    want, clipped = ref.clip_reference(g, 1, 0.1)
    assert abs(norm.item() - want) <= 1e-4 * want
    assert ref.rel_norm(out, clipped) <= 2.0 ** -11


def test_a_call_follows_the_last_one_on_another_stream():
    """A gradient of the loss on one stream and the next on another: the second
    must not write the workspace while the first, held up, still reads it."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    N, V, d = 300, 5000, 256
    data = [((torch.randn(N, d, device="cuda", generator=gen)).bfloat16(),
             (torch.randn(V, d, device="cuda", generator=gen) * 0.1).bfloat16(),
             torch.randint(0, V, (N,), device="cuda", generator=gen)) for _ in range(2)]
    op = zs.LmLoss(V, d, "bf16", max_tokens=N)
    lse = [op.loss(*x)[1] for x in data]
    want = [op.grad(*x, y, 1.0) for x, y in zip(data, lse)]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for k in (0, 1):
        with torch.cuda.stream(streams[k]):
            if k == 0:
                torch.cuda._sleep(DELAY)
            got.append(op.grad(*data[k], lse[k], 1.0))
            done = torch.cuda.Event()
            done.record()
            assert not done.query()     # the second waits for the first, which is held up
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_calls_without_the_workspace_wait_for_none():
    """The lookup and the clipping do not use it: they run beside a gradient or a norm on another stream."""
    h, t = torch.randn(64, 64, device="cuda").half(), torch.randn(100, 64, device="cuda").half()
    ids, g = torch.zeros(64, dtype=torch.int64, device="cuda"), [torch.ones(100, device="cuda").half()]
    emb, clip = zs.Embedding(100, 64, "fp16", max_tokens=64), zs.GradClip([100], 1, "fp16")
    norm = clip.norm([g])
    emb.grad(ids, h), emb.forward(ids, t), clip.clip([g], norm, 1.0)      # kernels loaded
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    held, free = torch.cuda.Event(), torch.cuda.Event()
    with torch.cuda.stream(a):
        torch.cuda._sleep(DELAY)
        emb.grad(ids, h), clip.norm([g])
        held.record()
    with torch.cuda.stream(b):
        y, out = emb.forward(ids, t), clip.clip([g], norm, 1.0)
        free.record()
    free.synchronize()
    beside = not held.query()
    torch.cuda.synchronize()
    assert beside and torch.equal(y, t[ids]) and torch.allclose(out, (g[0].float() / 10).half())


@pytest.mark.parametrize("make", [lambda: zs.GradClip([100], 1, "fp16"),
                                  lambda: zs.Embedding(100, 64, "fp16", max_tokens=5000),
                                  lambda: zs.LmLoss(100, 64, "fp16", max_tokens=64)])
def test_the_workspace_of_a_dropped_owner_is_not_handed_out_early(make):
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    h, t = torch.randn(64, 64, device="cuda").half(), torch.randn(100, 64, device="cuda").half()
    ids, g = torch.zeros(64, dtype=torch.int64, device="cuda"), torch.zeros(100, device="cuda").half()

    def call(op):
        if isinstance(op, zs.GradClip):
            return op.norm([[g]])
        return op.grad(ids, h) if isinstance(op, zs.Embedding) else op.loss(h, t, ids)

    call(make())                        # kernels loaded at their first call wait for the device
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        op = make()
    with torch.cuda.stream(b):
        torch.cuda._sleep(DELAY)
        call(op)
        done = torch.cuda.Event()
        done.record()
    at, nbytes = op.workspace.data_ptr(), op.workspace.numel()
    del op
    with torch.cuda.stream(a):
        again = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    early, busy = again.data_ptr() == at, not done.query()
    torch.cuda.synchronize()
    assert busy and not early


def test_a_capture_on_another_stream_than_the_calls_before():
    """Capturing must not make the captured work wait for work outside of it."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn(200, 64, device="cuda", generator=gen).half()
    t = torch.randn(700, 64, device="cuda", generator=gen).half() * 0.2
    tg = torch.randint(0, 700, (200,), device="cuda", generator=gen)
    op = zs.LmLoss(700, 64, "fp16", max_tokens=200)
    want = op.loss(h, t, tg)
    grads = op.grad(h, t, tg, want[1], 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse = op.loss(h, t, tg)
        dh, dt = op.grad(h, t, tg, lse, 1.0)
    for x in (loss, lse, dh, dt):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((loss, lse, dh, dt), want + grads))
    assert torch.equal(op.loss(h, t, tg)[0], loss)


@pytest.mark.parametrize("as_handle", [False, True])
def test_the_clipped_steps_workspace_belongs_to_the_steps_stream(as_handle):
    """Made in the order of the step's stream, however that is given, while another one is current."""
    n, W = 50_000, 4
    theta0 = torch.randn(n, device="cuda") * 0.02
    side = torch.cuda.Stream()
    a = zs.ZeroStep(zs.ZERO_SCHEME_Z2, W, [n], "bf16", theta0=theta0)
    grads = a.new_grad_buffers()
    for k, x in enumerate(grads):
        x.copy_(torch.randn(a.n_pad, device="cuda") * 0.01 * (k + 1))
    torch.cuda.synchronize()
    b = zs.ZeroStep(zs.ZERO_SCHEME_Z2, W, [n], "bf16", theta0=theta0, stream=side.cuda_stream if as_handle else side)
    torch.cuda.synchronize()
    a.step(grads, LR, B1, B2, EPS, 1, max_norm=0.1)
    nbytes = zs.zero_step_clipped_workspace_bytes(b.ctx)
    dirty = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del dirty
    torch.cuda._sleep(DELAY)            # on the current stream, which the step does not use
    b.step(grads, LR, B1, B2, EPS, 1, max_norm=0.1)
    b.sync()
    got = b.grad_norm.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, a.grad_norm) and torch.equal(b.master, a.master) and torch.equal(b.p16, a.p16)
    a.close(), b.close()


def test_owners_take_a_stream_by_its_handle():
    side = torch.cuda.Stream()
    h = torch.randn(40, 64, device="cuda").half()
    t, tg = torch.randn(90, 64, device="cuda").half(), torch.arange(40, device="cuda")
    want = zs.LmLoss(90, 64, "fp16", max_tokens=40).loss(h, t, tg)
    torch.cuda.synchronize()
    got = zs.LmLoss(90, 64, "fp16", max_tokens=40, stream=side.cuda_stream).loss(h, t, tg)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
