"""The language-model operators next to the ZeRO step, as measured cases.

Five calls of three operators: the loss over a large vocabulary with its
gradient (``lm_loss``, ``lm_grad``), the embedding lookup and its gradient
(``embed``, ``embed_grad``), and the global gradient norm with clipping, by
itself over many tensors and inside the step (``clip``, ``step``).

``run`` computes a case in elementary torch operations in 32 bits, rounded
once at the end; with ``own`` set it makes the library's calls instead.
``exact`` computes the same outputs in 64 bits from the definitions.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16}
LR, BETA1, BETA2, EPS = 6e-4, 0.9, 0.95, 1e-8
CLIP_EPS = 1e-6
FIRST_STEP = 11      # the step counter of the first timed step: moments with some history


def listed():
    return [
        # scoring a few positions (a short continuation, the last token of each of 16 sequences)
        {"name": "score_few", "op": "lm_loss", "N": 16, "V": 50257, "d": 768, "dtype": "bf16"},
        # evaluation of 4 sequences of 1024 tokens
        {"name": "score_batch", "op": "lm_loss", "N": 4096, "V": 50257, "d": 768, "dtype": "fp16"},
        # a toy model with a vocabulary of characters and pairs: latency
        {"name": "lm_tiny", "op": "lm_grad", "N": 129, "V": 1031, "d": 264, "dtype": "fp16"},
        # training, a micro-batch of 8 sequences of 1024 tokens at the GPT-2-small width
        {"name": "lm_gpt2_small", "op": "lm_grad", "N": 8192, "V": 50257, "d": 768, "dtype": "bf16"},
        # training at the GPT-2-1.5B width, packed sequences without their padding (an odd token count)
        {"name": "lm_gpt2_xl", "op": "lm_grad", "N": 4095, "V": 50257, "d": 1600, "dtype": "fp16"},
        # generating for 16 sequences: one token each
        {"name": "embed_few", "op": "embed", "N": 16, "V": 50257, "d": 768, "dtype": "bf16"},
        # a training batch of 32 sequences of 1024 tokens
        {"name": "embed_batch", "op": "embed", "N": 32768, "V": 50257, "d": 1600, "dtype": "fp16"},
        # the table's gradient of one micro-batch
        {"name": "embed_grad_batch", "op": "embed_grad", "N": 8192, "V": 50257, "d": 768, "dtype": "bf16",
         "add": False},
        # a tied table: added onto the gradient that the loss head has left there
        {"name": "embed_grad_tied", "op": "embed_grad", "N": 65535, "V": 50257, "d": 1600, "dtype": "fp16",
         "add": True},
        # the gradients as a backward pass leaves them: many tensors, biases and matrices, of 4 ranks
        {"name": "clip_tensors", "op": "clip", "tensors": 148, "n": 20_000_011, "W": 4, "dtype": "bf16"},
        # the clipped step of a small model: latency
        {"name": "step_small", "op": "step", "n": 1 << 20, "W": 8, "dtype": "fp16"},
        # the clipped step of the GPT-2-small vector
        {"name": "step_gpt2_small", "op": "step", "n": 124_439_808, "W": 8, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lm_loss", "lm_grad", "lm_grad", "embed", "embed_grad", "clip", "step"])
    case = {"op": op, "dtype": rng.choice(["fp16", "bf16"])}
    if op in ("lm_loss", "lm_grad"):
        case["N"] = _spread(rng, 1, 8192)
        case["V"] = _spread(rng, 512, 50304)
        case["d"] = 8 * _spread(rng, 8, 200)
        if case["N"] * case["V"] * case["d"] > 8192 * 50257 * 768:
            case["N"] = max(1, 8192 * 50257 * 768 // (case["V"] * case["d"]))
    elif op in ("embed", "embed_grad"):
        case["N"] = _spread(rng, 1, 60000)
        case["V"] = _spread(rng, 512, 50304)
        case["d"] = 8 * _spread(rng, 8, 200)
        if op == "embed_grad":
            case["add"] = rng.random() < 0.5
    elif op == "clip":
        case["tensors"] = _spread(rng, 1, 400)
        case["n"] = _spread(rng, 4096, 40_000_000)
        case["W"] = rng.choice([1, 1, 2, 3, 4, 8])
    else:
        case["n"] = _spread(rng, 1024, 60_000_000)
        case["W"] = rng.choice([1, 2, 3, 4, 8, 8, 16])
    return case


def _tensor_sizes(count, n):
    """`count` sizes that add up to n: a few large ones, many small and odd ones."""
    weight = [1.0 / (1 + (7 * k) % count) for k in range(count)]
    total = sum(weight)
    sizes = [max(1, int(n * w / total)) for w in weight]
    sizes[0] += max(0, n - sum(sizes))
    return sizes


def _tokens(gen, N, V):
    """Token ids as frequent as words are: the k-th about 1/k."""
    u = torch.rand(N, device="cuda", generator=gen, dtype=torch.float64)
    return (torch.exp(u * math.log(V + 1)).to(torch.int64) - 1).clamp_(0, V - 1)


def _normal(gen, shape, sigma, dtype):
    return (torch.randn(shape, device="cuda", generator=gen) * sigma).to(dtype)


def _grad_scale(case):
    """The factor of the loss's gradient: the mean over the tokens, and in fp16 a loss scale of 2^14."""
    return (16384.0 if case["dtype"] == "fp16" else 1.0) / case["N"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], DTYPE[case["dtype"]]
    s = {"case": case, "op": op}
    if op in ("lm_loss", "lm_grad"):
        N, V, d = case["N"], case["V"], case["d"]
        s["hidden"] = _normal(gen, (N, d), 1.0, dtype)
        s["table"] = _normal(gen, (V, d), 0.04, dtype)
        s["targets"] = _tokens(gen, N, V)
        # one position in 16 has no target (the ends of sequences, a prompt that is not trained on)
        s["targets"][torch.rand(N, device="cuda", generator=gen) < 1 / 16] = -100
        s["scale"] = _grad_scale(case)
    elif op in ("embed", "embed_grad"):
        N, V, d = case["N"], case["V"], case["d"]
        s["tokens"] = _tokens(gen, N, V)
        s["scale"] = math.sqrt(d)
        if op == "embed":
            s["table"] = _normal(gen, (V, d), 0.02, dtype)
        else:
            s["dout"] = _normal(gen, (N, d), 1e-3, dtype)
            s["add"] = case["add"]
            s["dtable"] = _normal(gen, (V, d), 1e-3, dtype) if case["add"] else torch.empty(
                (V, d), device="cuda", dtype=dtype)
    elif op == "clip":
        s["sizes"] = _tensor_sizes(case["tensors"], case["n"])
        s["grads"] = [[_normal(gen, (k,), 1e-3, dtype) for k in s["sizes"]] for _ in range(case["W"])]
        s["max_norm"] = 1.0
    else:
        n, W = case["n"], case["W"]
        n_pad = -(-n // W) * W
        s["t"] = FIRST_STEP - 1
        s["max_norm"] = 1.0
        s["flat"] = torch.zeros((W, -(-n_pad // 8) * 8), device="cuda", dtype=dtype)
        s["flat"][:, :n] = torch.randn((W, n), device="cuda", generator=gen).mul_(1e-3)
        s["grads"] = [row[:n_pad] for row in s["flat"]]
        master = torch.randn(n, device="cuda", generator=gen) * 0.02
        m = torch.randn(n, device="cuda", generator=gen) * 1e-4
        v = torch.rand(n, device="cuda", generator=gen) * 1e-7
        s["state"] = [torch.nn.functional.pad(x, (0, n_pad - n)) for x in (master, m, v)]
        s["n"], s["n_pad"] = n, n_pad
    if own:
        s["handle"] = _handle(s)
    return s


def _handle(s):
    """What a user's program keeps between calls: the owner of the workspace."""
    import zero_sharded_mixed_step_gb300 as zs
    case, op = s["case"], s["op"]
    if op in ("lm_loss", "lm_grad"):
        return zs.LmLoss(case["V"], case["d"], case["dtype"], max_tokens=case["N"])
    if op in ("embed", "embed_grad"):
        return zs.Embedding(case["V"], case["d"], case["dtype"], max_tokens=case["N"], scale=s["scale"])
    if op == "clip":
        return zs.GradClip(s["sizes"], case["W"], case["dtype"])
    step = zs.ZeroStep(zs.ZERO_SCHEME_Z2, case["W"], [s["n"]], case["dtype"])
    zs.zero_set_state(step.ctx, *s["state"], s["t"])
    return step


# ---- the plain forms -----------------------------------------------------------

def _plain_loss(s):
    logits = s["hidden"].float() @ s["table"].float().T
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    valid = (s["targets"] >= 0) & (s["targets"] < logits.shape[1])
    at = torch.where(valid, s["targets"], 0)[:, None]
    loss = torch.where(valid, (top + torch.log(total) - logits.gather(1, at))[:, 0], 0.0)
    return loss, e, total, valid, at


def _plain_lm_grad(s):
    loss, e, total, valid, at = _plain_loss(s)
    e /= total
    rows = torch.arange(e.shape[0], device=e.device)
    e[rows, at[:, 0]] -= 1.0
    e *= (valid * s["scale"])[:, None]
    dtype = s["hidden"].dtype
    return loss, (e @ s["table"].float()).to(dtype), (e.T @ s["hidden"].float()).to(dtype)


def _plain_embed_grad(s):
    table = s["dtable"]
    total = torch.zeros(table.shape, device=table.device)
    total.index_add_(0, s["tokens"], s["dout"].float())
    total *= s["scale"]
    if s["add"]:
        total += table.float()
    table.copy_(total)
    return table


def _plain_clip(s):
    count = len(s["sizes"])
    mean = torch.stack([torch.cat(g) for g in s["grads"]]).float().sum(0) / len(s["grads"])
    norm = mean.square().sum().sqrt()
    clipped = (mean * torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)).to(s["grads"][0][0].dtype)
    return norm.reshape(1), torch.cat(clipped.split(s["sizes"])) if count else clipped


def _plain_step(s):
    s["t"] += 1
    t = s["t"]
    master, m, v = s["state"]
    g = s["flat"][:, : s["n_pad"]].float().sum(0) / len(s["grads"])
    norm = g.square().sum().sqrt()
    g *= torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)
    m.mul_(BETA1).add_(g, alpha=1 - BETA1)
    v.mul_(BETA2).add_(g * g, alpha=1 - BETA2)
    den = v.sqrt().mul_(1.0 / math.sqrt(1.0 - BETA2 ** t)).add_(EPS)
    master.sub_((m / den).mul_(LR / (1.0 - BETA1 ** t)))
    return norm.reshape(1), master, m, v, master.to(s["flat"].dtype)


def _plain(s):
    op = s["op"]
    if op == "lm_loss":
        return _plain_loss(s)[0]
    if op == "lm_grad":
        return _plain_lm_grad(s)
    if op == "embed":
        rows = s["table"][s["tokens"]].float() * s["scale"]
        return rows.to(s["table"].dtype)
    if op == "embed_grad":
        return _plain_embed_grad(s)
    return _plain_clip(s) if op == "clip" else _plain_step(s)


# ---- the library's calls ---------------------------------------------------------

def _own(s):
    op, handle = s["op"], s["handle"]
    if op == "lm_loss":
        return handle.loss(s["hidden"], s["table"], s["targets"])[0]
    if op == "lm_grad":
        loss, lse = handle.loss(s["hidden"], s["table"], s["targets"])
        dhidden, dtable = handle.grad(s["hidden"], s["table"], s["targets"], lse, s["scale"])
        return loss, dhidden, dtable
    if op == "embed":
        return handle.forward(s["tokens"], s["table"])
    if op == "embed_grad":
        return handle.grad(s["tokens"], s["dout"], s["dtable"], accumulate=s["add"])
    if op == "clip":
        return handle.norm_and_clip(s["grads"], s["max_norm"])
    s["t"] += 1
    handle.step(s["grads"], LR, BETA1, BETA2, EPS, s["t"], max_norm=s["max_norm"])
    return handle.grad_norm, handle.master, handle.m, handle.v, handle.p16


def run(state):
    return _own(state) if own else _plain(state)


# ---- cost and definition ----------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("lm_loss", "lm_grad"):
        N, V, d = case["N"], case["V"], case["d"]
        once = 2 * (N + V) * d
        # read both matrices and the targets, write the losses; the gradients are as large as the inputs
        return {"bytes": once * (1 if op == "lm_loss" else 2) + 12 * N,
                "flops": 2.0 * N * V * d * (1 if op == "lm_loss" else 3)}
    if op in ("embed", "embed_grad"):
        N, V, d = case["N"], case["V"], case["d"]
        # N draws of a frequency of about 1/k meet this many different ids
        H = math.log(V + 1)
        met = sum(1.0 - math.exp(-N * math.log1p(1.0 / k) / H) for k in range(1, V + 1))
        if op == "embed":
            return {"bytes": 2 * d * (N + met) + 8 * N, "flops": float(N * d)}
        return {"bytes": 2 * d * (N + (2 * met if case["add"] else V)) + 8 * N, "flops": float(N * d)}
    n, W = case["n"], case["W"]
    if op == "clip":
        return {"bytes": 2.0 * n * (W + 1), "flops": float(n * (W + 3))}
    return {"bytes": n * (2.0 * W + 26), "flops": float(n * (W + 15))}


def exact(case, seed):
    if case["op"] in ("lm_loss", "lm_grad") and 6.0 * case["N"] * case["V"] * case["d"] > 5e12:
        return None
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    op = case["op"]
    if op in ("lm_loss", "lm_grad"):
        return _exact_lm(s, op == "lm_grad")
    if op == "embed":
        return torch.index_select(s["table"].double() * s["scale"], 0, s["tokens"])
    if op == "embed_grad":
        # the rows in the order of their tokens, running sums, differences at each token's last row
        order = torch.argsort(s["tokens"], stable=True)
        sums = torch.cumsum(s["dout"].double()[order] * s["scale"], 0)
        sums = torch.cat([torch.zeros_like(sums[:1]), sums])
        ends = torch.searchsorted(s["tokens"][order].contiguous(), torch.arange(case["V"], device="cuda"), right=True)
        starts = torch.cat([torch.zeros_like(ends[:1]), ends[:-1]])
        total = sums[ends] - sums[starts]
        return total + s["dtable"].double() if s["add"] else total
    W = case["W"]
    if op == "clip":
        mean = sum(torch.cat(g).double() for g in s["grads"]) / W
    else:
        mean = sum(g.double() for g in s["grads"]) / W
    norm = torch.linalg.vector_norm(mean)
    mean = mean * min(1.0, s["max_norm"] / (float(norm) + CLIP_EPS))
    if op == "clip":
        return norm.reshape(1), mean
    master, m, v = (x.double() for x in s["state"])
    m = BETA1 * m + (1.0 - BETA1) * mean
    v = BETA2 * v + (1.0 - BETA2) * mean ** 2
    m_hat, v_hat = m / (1.0 - BETA1 ** FIRST_STEP), v / (1.0 - BETA2 ** FIRST_STEP)
    master = master - LR * m_hat / (torch.sqrt(v_hat) + EPS)
    return norm.reshape(1), master, m, v, master


def _exact_lm(s, with_grad):
    table = s["table"].double()
    N = s["hidden"].shape[0]
    loss = torch.empty(N, device="cuda", dtype=torch.float64)
    dhidden = torch.empty(s["hidden"].shape, device="cuda", dtype=torch.float64)
    dtable = torch.zeros_like(table)
    for lo in range(0, N, 2048):
        h = s["hidden"][lo:lo + 2048].double()
        target = s["targets"][lo:lo + 2048]
        valid = (target >= 0).double()
        onehot = torch.nn.functional.one_hot(target.clamp(min=0), table.shape[0]).double()
        logp = torch.log_softmax(torch.matmul(h, table.t()), dim=1)
        loss[lo:lo + 2048] = -(logp * onehot).sum(1) * valid
        if with_grad:
            d = (logp.exp() - onehot) * (valid * s["scale"])[:, None]
            dhidden[lo:lo + 2048] = d @ table
            dtable += d.t() @ h
    return (loss, dhidden, dtable) if with_grad else loss
