"""Plain 64-bit forms of the language-model operators, and error bounds for the
kernels derived from how they compute (16-bit operands, fp32 sums).

Half a unit in the last place of the 16-bit formats, relative to the value:
at most 2^-11 for fp16 (11 significant bits), 2^-8 for bf16 (8).  A matrix product over K terms adds
16 products at a time to an fp32 accumulator, so it takes at most K / 16 + 5
roundings of 2^-23 (truncation) of at most the sum of the products' absolute
values.  exp2 on the device is good to 2^-22, and its argument l log2(e), formed
with one rounding, to 2^-23 of |l|."""

import math

import torch

HALF_ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY16 = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}     # half the smallest subnormal
PROB_SCALE = {torch.float16: 2.0 ** 14, torch.bfloat16: 1.0}          # what the kernels store D times


def valid_mask(targets, vocab):
    return (targets >= 0) & (targets < vocab)


def lm_reference(hidden, table, targets, scale=1.0):
    """dict of the 64-bit loss, lse, dhidden, dtable and elementwise bounds for each."""
    dtype = hidden.dtype
    u = HALF_ULP[dtype]
    vocab, d = table.shape
    valid = valid_mask(targets, vocab)
    # a token without target contributes nothing, whatever its hidden vector holds
    h = torch.where(valid[:, None], hidden.double(), 0.0)
    t = table.double()
    logits = h @ t.T
    lse = torch.logsumexp(logits, 1)
    at = torch.where(valid, targets, 0).long()
    picked = logits.gather(1, at[:, None])[:, 0]
    onehot = torch.zeros_like(logits)
    onehot[torch.arange(len(at), device=at.device), at] = valid.double()
    p = torch.exp(logits - lse[:, None])
    D = torch.where(valid[:, None], p - onehot, 0.0)
    out = dict(loss=torch.where(valid, lse - picked, 0.0), lse=lse, dhidden=scale * D @ t, dtable=scale * D.T @ h)
    mass = (h.abs() @ t.abs().T).amax(1) if vocab else torch.zeros_like(lse)
    logit_err = (d / 16 + 5) * 2.0 ** -23 * mass
    top = logits.abs().amax(1)
    # the sum of exponentials: 2^-22 each, the arguments' rounding, at most 300 additions of 2^-24 one after another
    rel_sum = 2.0 ** -22 + (top + 1) * 2.0 ** -22 + 300 * 2.0 ** -24
    out["lse_bound"] = logit_err + rel_sum + (lse.abs() + 1) * 2.0 ** -22
    out["loss_bound"] = torch.where(valid, out["lse_bound"] + logit_err + (picked.abs() + 1) * 2.0 ** -23, 0.0)
    rel_p = logit_err + out["lse_bound"] + 2.0 ** -22 + (top + lse.abs() + 1) * 2.0 ** -22
    size = torch.where(valid[:, None], p + onehot, 0.0)
    Derr = p * rel_p[:, None] * valid[:, None] + size * u + TINY16[dtype] / PROB_SCALE[dtype]
    out["dhidden_bound"] = scale * (Derr @ t.abs() + (vocab / 16 + 64) * 2.0 ** -23 * (size @ t.abs())) * (1 + u) + \
        out["dhidden"].abs() * u + TINY16[dtype]
    N = h.shape[0]
    out["dtable_bound"] = scale * (Derr.T @ h.abs() + (N / 16 + 64) * 2.0 ** -23 * (size.T @ h.abs())) * (1 + u) + \
        out["dtable"].abs() * u + TINY16[dtype]
    return out


def assert_within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first at {i}: "
                             f"{got.flatten()[i].item()!r} want {want.flatten()[i].item()!r} "
                             f"bound {bound.flatten()[i].item():.3g}")


def rel_norm(got, want):
    n = torch.linalg.vector_norm(want)
    e = torch.linalg.vector_norm(got.double() - want)
    return float(e / n) if n > 0 else float(e)


def embedding_grad_reference(ids, dout, scale, vocab, old=None):
    """64-bit gradient of the table and a bound: fp32 sums one after another, one rounding."""
    u = HALF_ULP[dout.dtype]
    valid = valid_mask(ids, vocab)
    rows = torch.where(valid[:, None], dout.double(), 0.0)
    at = torch.where(valid, ids, 0).long()
    total = torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device=dout.device).index_add_(0, at, rows)
    size = torch.zeros_like(total).index_add_(0, at, rows.abs())
    count = torch.bincount(at[valid], minlength=vocab).double()
    want = total * scale + (old.double() if old is not None else 0.0)
    bound = (count[:, None] + 2) * 2.0 ** -24 * size * abs(scale) + want.abs() * (u + 2.0 ** -23) + TINY16[dout.dtype]
    if old is not None:
        bound = bound + old.double().abs() * 2.0 ** -23
        untouched = count == 0
        bound[untouched] = 0.0
    return want, bound


def clip_reference(grads, W, max_norm):
    """(norm, clipped mean) in 64 bits from W flat vectors."""
    mean = sum(g.double() for g in grads) / W
    norm = float(torch.linalg.vector_norm(mean))
    coef = min(1.0, max_norm / (norm + 1e-6)) if math.isfinite(norm) else 1.0
    return norm, mean * coef
