"""Plain 64-bit forms of the orthogonalised update, and the tolerance for a
kernel that rounds its operands to fp16: the same recurrence in 64 bits with
those roundings put in shows how far they carry a given matrix; a kernel whose
sums differ in their last bits rounds some operands the other way, so that its
error is another draw of the same size."""

import torch

HALF_ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
COEFFICIENTS = ((3.4445, -4.7750, 2.0315),) * 5


def orthogonal(g, coefficients=COEFFICIENTS):
    """The recurrence on a 64-bit matrix over its norm."""
    x = g.double()
    norm = torch.linalg.vector_norm(x)
    x = x / norm if norm > 0 else x
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for a, b, c in coefficients:
        gram = x @ x.T
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.T if tall else x


def _parts(x, scale, count):
    hi = (x * scale).half().double()
    lo = (x * scale - hi).half().double() if count > 1 else torch.zeros_like(hi)
    return hi / scale, lo / scale


def _product(x, y):
    return (x[0] @ y[0] + x[0] @ y[1] + x[1] @ y[0]).float().double()


def rounded(g, coefficients, fine, first_parts):
    """The same with X, A and P rounded to one or two fp16 values as the kernels hold them."""
    x = g.double()
    norm = torch.linalg.vector_norm(x)
    x = x.T if x.shape[0] > x.shape[1] else x
    x = x / norm if norm > 0 else x
    for k, (a, b, c) in enumerate(coefficients):
        parts = 2 if k < fine else 1
        if k == 0 and first_parts == 1:
            xs = (x, torch.zeros_like(x))      # a 16-bit input is exact in one part
        else:
            xs = _parts(x, 4096.0, parts)
        gram = _parts(_product(xs, (xs[0].T, xs[1].T)), 4096.0, parts)
        p = a * torch.eye(len(x), device=x.device, dtype=x.dtype) + b * (gram[0] + gram[1]) + c * _product(gram, gram)
        x = _product(_parts(p, 512.0, parts), xs)
    return x.T if g.shape[0] > g.shape[1] else x


def tolerance(g, want, coefficients, fine, first_parts):
    """Of the result's 2-norm: twice what the roundings carry this matrix off, and what sums in fp32 leave: each of
    the three products of a step is truncated by 2^-23 of the sums' sizes some K / 16 times at random, times the
    steps' slopes, together at most the 64 below of 2^-23 sqrt(K)."""
    size = torch.linalg.vector_norm(want)
    if size == 0:
        return 0.0
    off = torch.linalg.vector_norm(rounded(g, coefficients, fine, first_parts) - want)
    return float(2 * off / size) + 64 * 2.0 ** -23 * max(g.shape) ** 0.5


def assert_near(got, want, tol, what):
    """Within tol of the 2-norm, and no element 16 times the mean error further off."""
    err = got.double() - want
    norm = float(torch.linalg.vector_norm(want))
    assert float(torch.linalg.vector_norm(err)) <= tol * norm, \
        f"{what}: {float(torch.linalg.vector_norm(err)) / max(norm, 1e-300):.3g} off, {tol:.3g} allowed"
    assert float(err.abs().max()) <= 16 * tol * max(norm / want.numel() ** 0.5, float(want.abs().max()) / 16), what


def step(grads, master, momentum, lr, mu, nesterov, decay, scale, coefficients=COEFFICIENTS):
    """(master, momentum, U) of one matrix after a step, in 64 bits; grads: one matrix of each rank."""
    g = sum(x.double() for x in grads) / len(grads)
    m = mu * momentum.double() + g
    u = g + mu * m if nesterov else m
    o = orthogonal(u, coefficients)
    return master.double() * (1 - lr * decay) - lr * scale * o, m, u
