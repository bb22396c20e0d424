"""What a language model's post-training takes beside the ZeRO step, as measured cases.

Four calls in two pairs.  The log probabilities of given tokens with the
entropy and the likeliest alternatives over a large vocabulary (``logprobs``),
and the gradients that a policy's loss sends back through them
(``logprobs_grad``).  The orthogonalised update of a matrix by Newton-Schulz
products (``orthogonalize``), and the optimizer step over many ranks'
gradients that takes its direction from it (``muon``).

``run`` computes a case in elementary torch operations in 32 bits, rounded
once at the end; with ``own`` set it makes the library's calls instead.
``exact`` computes the same outputs in 64 bits from the definitions.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
LR, MU, DECAY = 3e-4, 0.95, 0.1
COEFFICIENTS = ((3.4445, -4.7750, 2.0315),) * 5     # (a, b, c) of each step: X <- a X + b (X X^T) X + c (X X^T)^2 X

# the shapes of a transformer's matrices, as lists of (rows, cols, how many)
MATRICES = {
    # a small test model: a narrow one and a wide one of each
    "toy": ((136, 264, 2), (264, 136, 2), (136, 136, 2)),
    # 12 layers of the GPT-2-small width: queries, keys and values in one, and the projection
    "attention_768": ((768, 2304, 12), (768, 768, 12)),
    # one layer of the GPT-2-1.5B width
    "layer_1600": ((1600, 4800, 1), (1600, 1600, 1), (1600, 6400, 1), (6400, 1600, 1)),
}


def listed():
    return [
        # the alternatives of the next token while 16 sequences are generated
        {"name": "sampled_few", "op": "logprobs", "N": 16, "V": 50257, "d": 768, "top": 8, "scale": 1.25, "dtype": "bf16"},
        # the log probabilities under a reference model of 4 rollouts of 1024 tokens, nothing but them and the entropy
        {"name": "rollout", "op": "logprobs", "N": 4096, "V": 50257, "d": 768, "top": 0, "scale": 1.0, "dtype": "fp16"},
        # an evaluation that keeps the likeliest 16 words of every position, packed sequences (an odd token count)
        {"name": "top_words", "op": "logprobs", "N": 2047, "V": 32000, "d": 2048, "top": 16, "scale": 1.0, "dtype": "bf16"},
        # a toy policy over a vocabulary of characters and pairs: latency
        {"name": "policy_tiny", "op": "logprobs_grad", "N": 129, "V": 1031, "d": 264, "scale": 1.0, "dtype": "fp16"},
        # a policy's micro-batch of 8 rollouts of 1024 tokens at the GPT-2-small width
        {"name": "policy_small", "op": "logprobs_grad", "N": 8192, "V": 50257, "d": 768, "scale": 1.0, "dtype": "bf16"},
        # the GPT-2-1.5B width, rollouts without their padding (an odd token count), sampled at a temperature of 0.8
        {"name": "policy_xl", "op": "logprobs_grad", "N": 4095, "V": 50257, "d": 1600, "scale": 1.25, "dtype": "fp16"},
        # one small matrix: latency
        {"name": "orth_one", "op": "orthogonalize", "rows": 256, "cols": 256, "count": 1, "dtype": "bf16"},
        # the square matrices of a model of the GPT-2-small width
        {"name": "orth_768", "op": "orthogonalize", "rows": 768, "cols": 768, "count": 24, "dtype": "fp16"},
        # one large wide matrix
        {"name": "orth_wide", "op": "orthogonalize", "rows": 1600, "cols": 6400, "count": 1, "dtype": "bf16"},
        # the step of a small test model: latency
        {"name": "muon_toy", "op": "muon", "model": "toy", "W": 4, "dtype": "bf16"},
        # the attention's matrices of a model of the GPT-2-small width, 8 ranks
        {"name": "muon_768", "op": "muon", "model": "attention_768", "W": 8, "dtype": "bf16"},
        # one layer at the GPT-2-1.5B width, 4 ranks
        {"name": "muon_1600", "op": "muon", "model": "layer_1600", "W": 4, "dtype": "fp16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "orthogonalize", "muon"])
    case = {"op": op, "dtype": rng.choice(["fp16", "bf16"])}
    if op in ("logprobs", "logprobs_grad"):
        case["N"] = _spread(rng, 1, 8192)
        case["V"] = _spread(rng, 512, 50304)
        case["d"] = 8 * _spread(rng, 8, 200)
        case["scale"] = rng.choice([1.0, 1.0, 0.5, 1.25])
        if op == "logprobs":
            case["top"] = rng.choice([0, 0, 1, 4, 8, 16])
        most = 8192 * 50257 * 768 if op == "logprobs_grad" else 4096 * 50257 * 768
        case["N"] = max(1, min(case["N"], most // (case["V"] * case["d"])))
    elif op == "orthogonalize":
        case["rows"], case["cols"] = _spread(rng, 1, 2048), _spread(rng, 1, 2048)
        case["count"] = _spread(rng, 1, 24)
        case["dtype"] = rng.choice(["fp16", "bf16", "fp32"])
        small, large = sorted((case["rows"], case["cols"]))
        case["count"] = max(1, min(case["count"], 24 * 768 ** 3 // (small * small * large)))
    else:
        # a model of its own: two shapes, one or several of each
        wide, narrow = _spread(rng, 8, 1600), _spread(rng, 8, 1600)
        case["model"] = "%dx%dx%d %dx%dx%d" % (wide, narrow, rng.choice([1, 2, 5]), narrow, narrow, rng.choice([1, 3]))
        case["W"] = rng.choice([1, 2, 3, 4, 8])
    return case


def _shapes(case):
    """(rows, cols) of each matrix of a step."""
    kinds = MATRICES.get(case["model"]) or [tuple(map(int, part.split("x"))) for part in case["model"].split()]
    return [(r, c) for r, c, count in kinds for _ in range(count)]


def _starts(shapes):
    """Where each matrix starts in the flat vectors, on boundaries of 8 values, and their length."""
    at, starts = 0, []
    for r, c in shapes:
        starts.append(at)
        at += -(-r * c // 8) * 8
    return starts, at


def _tokens(gen, N, V):
    """Token ids as frequent as words are: the k-th about 1/k."""
    u = torch.rand(N, device="cuda", generator=gen, dtype=torch.float64)
    return (torch.exp(u * math.log(V + 1)).to(torch.int64) - 1).clamp_(0, V - 1)


def _normal(gen, shape, sigma, dtype):
    return (torch.randn(shape, device="cuda", generator=gen) * sigma).to(dtype)


def _grid(gen, shape, sigma, step, most, dtype):
    """Normal values on a grid of `step` up to `most`: every order of summing their products gives the same
    logits, so that the alternatives' ids can be compared; equal logits occur."""
    x = torch.randn(shape, device="cuda", generator=gen) * (sigma / step)
    return (x.round_().clamp_(-most / step, most / step) * step).to(dtype)


def _gradient(gen, rows, cols):
    """A gradient's matrix in fp32: a few directions that many tokens share, on top of noise."""
    few = min(32, rows, cols)
    weight = 0.3 / torch.arange(1, few + 1, device="cuda").sqrt()
    shared = (torch.randn(rows, few, device="cuda", generator=gen) * weight) @ torch.randn(few, cols, device="cuda",
                                                                                            generator=gen)
    return (shared + torch.randn(rows, cols, device="cuda", generator=gen)) * 1e-3


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], DTYPE[case["dtype"]]
    s = {"case": case, "op": op}
    if op in ("logprobs", "logprobs_grad"):
        N, V, d = case["N"], case["V"], case["d"]
        s["scale"] = case["scale"]
        s["targets"] = _tokens(gen, N, V)
        # one position in 16 is not scored (a prompt, padding)
        s["targets"][torch.rand(N, device="cuda", generator=gen) < 1 / 16] = -100
        if op == "logprobs":
            s["top"] = case["top"]
            s["hidden"] = _grid(gen, (N, d), 1.0, 2.0 ** -4, 4.0, dtype)
            s["table"] = _grid(gen, (V, d), 0.04, 2.0 ** -9, 0.25, dtype)
        else:
            s["hidden"] = _normal(gen, (N, d), 1.0, dtype)
            s["table"] = _normal(gen, (V, d), 0.04, dtype)
            # what the policy's loss sends back: an advantage for each token, some of them 0, and a bonus for entropy;
            # the mean over the tokens, in fp16 with a loss scale of 2^14
            mean = (16384.0 if case["dtype"] == "fp16" else 1.0) / N
            s["dlogp"] = torch.randn(N, device="cuda", generator=gen) * -mean
            s["dlogp"][torch.rand(N, device="cuda", generator=gen) < 1 / 8] = 0.0
            s["dentropy"] = torch.full((N,), -0.01 * mean, device="cuda")
    elif op == "orthogonalize":
        s["matrices"] = [_gradient(gen, case["rows"], case["cols"]).to(dtype) for _ in range(case["count"])]
    else:
        s["shapes"] = _shapes(case)
        s["starts"], n = _starts(s["shapes"])
        signal = torch.zeros(n, device="cuda")
        theta = torch.zeros(n, device="cuda")
        momentum = torch.zeros(n, device="cuda")
        for (r, c), at in zip(s["shapes"], s["starts"]):
            signal[at:at + r * c] = _gradient(gen, r, c).flatten()
            theta[at:at + r * c] = torch.randn(r * c, device="cuda", generator=gen) * 0.02
            momentum[at:at + r * c] = 10 * _gradient(gen, r, c).flatten()
        s["flat"] = [(signal + _normal(gen, (n,), 1e-3, torch.float32)).to(dtype) for _ in range(case["W"])]
        s["grads"] = [[g[at:at + r * c].view(r, c) for (r, c), at in zip(s["shapes"], s["starts"])] for g in s["flat"]]
        s["master"], s["momentum"] = theta, momentum
        s["scales"] = [0.2 * math.sqrt(max(r, c)) for r, c in s["shapes"]]
    if own:
        s["handle"] = _handle(s)
    return s


def _handle(s):
    """What a user's program keeps between calls: the owner of the workspace or of the state."""
    import zero_sharded_mixed_step_gb300 as zs
    case, op = s["case"], s["op"]
    if op in ("logprobs", "logprobs_grad"):
        return zs.LmLogprobs(case["V"], case["d"], case["dtype"], max_tokens=case["N"], scale=case["scale"],
                             top=case.get("top", 0), with_grad=op == "logprobs_grad")
    if op == "orthogonalize":
        return zs.Orthogonalize([(case["rows"], case["cols"])] * case["count"], case["dtype"],
                                coefficients=COEFFICIENTS)
    step = zs.MuonStep(s["shapes"], case["W"], case["dtype"], coefficients=COEFFICIENTS, scales=s["scales"])
    step.master.copy_(s["master"])
    step.momentum.copy_(s["momentum"])
    s["gaps"] = _gaps(s, step)
    return step


def _gaps(s, step):
    """What a call for the values between the matrices takes: the gradients' vectors go on there, and so does the
    momentum.  Each gap is a matrix of one row, whose step has a learning rate of 0; None without gaps."""
    import zero_sharded_mixed_step_gb300 as zs
    ends = s["starts"][1:] + [step.n]
    gaps = [(at + r * c, end) for (r, c), at, end in zip(s["shapes"], s["starts"], ends) if at + r * c < end]
    if not gaps:
        return None
    shapes = [(1, end - at) for at, end in gaps]
    states = [[x[at:] for at, _ in gaps] for x in (step.master, step.momentum, step.p16)]
    grads = [[g[at:] for at, _ in gaps] for g in s["flat"]]
    space = torch.zeros(zs.zero_muon_workspace_bytes(step.W, shapes), dtype=torch.uint8, device="cuda")
    return lambda: zs.zero_muon_step(step.W, shapes, step.dtype, step.wdt, grads, *states, LR, MU, True, DECAY,
                                     [0.0] * len(gaps), ((1.0, 0.0, 0.0),), 0, space, space.numel(),
                                     torch.cuda.current_stream())


# ---- the plain forms -----------------------------------------------------------

def _plain_softmax(s):
    """The scaled logits less their maximum, the exponentials' sums, the outputs of `logprobs` without alternatives."""
    raw = s["hidden"].float() @ s["table"].float().T
    x = raw * s["scale"]
    top = x.amax(1, keepdim=True)
    x -= top
    e = torch.exp(x)
    total = e.sum(1, keepdim=True)
    valid = (s["targets"] >= 0) & (s["targets"] < x.shape[1])
    at = torch.where(valid, s["targets"], 0)[:, None]
    lse = torch.log(total)
    logp = torch.where(valid, (x.gather(1, at) - lse)[:, 0], 0.0)
    entropy = lse - (e * x).sum(1, keepdim=True) / total
    return raw, x, e, total, lse, valid, at, logp, entropy, (top + lse)[:, 0]


def _plain_logprobs(s):
    raw, x, _, _, lse, _, _, logp, entropy, whole = _plain_softmax(s)
    if not s["top"]:
        return logp, entropy[:, 0], whole
    # the order of the floats as that of whole numbers, the lower of two equal logits' ids first
    bits = (raw + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64) << 32
    key += torch.arange(raw.shape[1] - 1, -1, -1, device=raw.device)
    ids = raw.shape[1] - 1 - (torch.topk(key, s["top"], dim=1).values & 0xFFFFFFFF)
    return logp, entropy[:, 0], whole, x.gather(1, ids) - lse, ids.to(torch.int32)


def _plain_logprobs_grad(s):
    _, x, e, total, lse, valid, at, logp, entropy, _ = _plain_softmax(s)
    g = torch.where(valid, s["dlogp"], 0.0)[:, None]
    h = torch.where(valid, s["dentropy"], 0.0)[:, None]
    # d logp / d l = onehot - p and d entropy / d l = -p (log p + entropy)
    d = e / total
    d *= -g - h * (x - lse + entropy)
    rows = torch.arange(d.shape[0], device=d.device)
    d[rows, at[:, 0]] += g[:, 0]
    d *= s["scale"]
    dtype = s["hidden"].dtype
    return logp, entropy[:, 0], (d @ s["table"].float()).to(dtype), (d.T @ s["hidden"].float()).to(dtype)


def _plain_orthogonal(g):
    """The Newton-Schulz steps on g over its norm, over the shorter side; a batch of matrices of one shape."""
    x = g.transpose(1, 2) if g.shape[1] > g.shape[2] else g
    x = x / x.square().sum((1, 2), keepdim=True).sqrt()
    for a, b, c in COEFFICIENTS:
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(1, 2) if g.shape[1] > g.shape[2] else x


def _plain_muon(s):
    g = sum(x.float() for x in s["flat"]) / len(s["flat"])
    m, master = s["momentum"], s["master"]
    m.mul_(MU).add_(g)
    update = g + MU * m
    master.mul_(1.0 - LR * DECAY)
    for r, c in dict.fromkeys(s["shapes"]):      # the matrices of one shape together
        here = [(at, scale) for shape, at, scale in zip(s["shapes"], s["starts"], s["scales"]) if shape == (r, c)]
        o = _plain_orthogonal(torch.stack([update[at:at + r * c].view(r, c) for at, _ in here]))
        for x, (at, scale) in zip(o, here):
            master[at:at + r * c] -= LR * scale * x.flatten()
    return master, m, master.to(s["flat"][0].dtype)


def _plain(s):
    op = s["op"]
    if op == "logprobs":
        return _plain_logprobs(s)
    if op == "logprobs_grad":
        return _plain_logprobs_grad(s)
    if op == "orthogonalize":
        g = torch.stack(s["matrices"])
        return list(_plain_orthogonal(g.float()).to(g.dtype))
    return _plain_muon(s)


# ---- the library's calls ---------------------------------------------------------

def _own(s):
    op, handle = s["op"], s["handle"]
    if op == "logprobs":
        return handle.logprobs(s["hidden"], s["table"], s["targets"])
    if op == "logprobs_grad":
        logp, entropy, lse = handle.logprobs(s["hidden"], s["table"], s["targets"])
        dhidden, dtable = handle.grad(s["hidden"], s["table"], s["targets"], lse, s["dlogp"], entropy, s["dentropy"])
        return logp, entropy, dhidden, dtable
    if op == "orthogonalize":
        return handle.forward(s["matrices"])
    handle.step(s["grads"], LR, MU, weight_decay=DECAY)
    if s["gaps"] is not None:
        s["gaps"]()
    return handle.master, handle.momentum, handle.p16


def run(state):
    return _own(state) if own else _plain(state)


# ---- cost and definition ----------------------------------------------------------

def _orthogonal_flops(rows, cols):
    """Operations of the steps: of the two symmetric products half, the third whole."""
    m, n = min(rows, cols), max(rows, cols)
    return len(COEFFICIENTS) * (m * m * n + m * m * m + 2.0 * m * m * n)


def work(case):
    op = case["op"]
    if op in ("logprobs", "logprobs_grad"):
        N, V, d = case["N"], case["V"], case["d"]
        once = 2 * (N + V) * d
        if op == "logprobs":
            return {"bytes": once + (20 + 8 * case["top"]) * N, "flops": 2.0 * N * V * d}
        return {"bytes": 2 * once + 24 * N, "flops": 6.0 * N * V * d}
    if op == "orthogonalize":
        item = 4 if case["dtype"] == "fp32" else 2
        r, c, count = case["rows"], case["cols"], case["count"]
        return {"bytes": 2.0 * item * r * c * count, "flops": count * _orthogonal_flops(r, c)}
    shapes, W = _shapes(case), case["W"]
    n = sum(r * c for r, c in shapes)
    # the gradients, master and momentum read, master, momentum and the working copy written
    return {"bytes": n * (2.0 * W + 18), "flops": n * (W + 8.0) + sum(_orthogonal_flops(r, c) for r, c in shapes)}


def exact(case, seed):
    op = case["op"]
    if op in ("logprobs", "logprobs_grad") and 6.0 * case["N"] * case["V"] * case["d"] > 5e12:
        return None
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    if op in ("logprobs", "logprobs_grad"):
        return _exact_lm(s, op)
    if op == "orthogonalize":
        return [_exact_orthogonal(g.double()) for g in s["matrices"]]
    master, momentum = s["master"].double(), s["momentum"].double()
    mean = torch.stack(s["flat"]).double().mean(0)
    momentum = momentum * MU + mean
    for (r, c), at, scale in zip(s["shapes"], s["starts"], s["scales"]):
        here = slice(at, at + r * c)
        o = _exact_orthogonal((mean[here] + momentum[here] * MU).reshape(r, c))
        master[here] = master[here] * (1.0 - LR * DECAY) - o.reshape(-1) * (LR * scale)
    return master, momentum, master


def _exact_orthogonal(g):
    """The same polynomial of the singular values, through the smaller side's eigenvectors: U p(S) V^T = Q r(L) Q^T G
    with G G^T = Q L Q^T and r = p(S) / S."""
    tall = g.shape[0] > g.shape[1]
    x = g.t() if tall else g
    x = x / torch.linalg.matrix_norm(x)
    lam, q = torch.linalg.eigh(torch.matmul(x, x.t()))
    lam = lam.clamp(min=0.0)
    ratio = torch.ones_like(lam)
    for a, b, c in COEFFICIENTS:
        now = lam * ratio ** 2
        ratio = ratio * (a + b * now + c * now ** 2)
    y = torch.matmul(q * ratio, torch.matmul(q.t(), x))
    return y.t() if tall else y


def _exact_lm(s, op):
    table, scale = s["table"].double(), s["scale"]
    V = table.shape[0]
    parts, dtable = [], torch.zeros_like(table) if op == "logprobs_grad" else None
    for lo in range(0, s["hidden"].shape[0], 2048):
        hidden, target = s["hidden"][lo:lo + 2048].double(), s["targets"][lo:lo + 2048]
        valid = (target >= 0).double()
        logits = torch.matmul(hidden, table.t())
        whole = torch.logsumexp(logits * scale, 1)
        logs = logits * scale - whole[:, None]
        p = logs.exp()
        entropy = -(p * logs).sum(1)
        logp = logs.gather(1, target.clamp(min=0)[:, None])[:, 0] * valid
        if op == "logprobs":
            out = [logp, entropy, whole]
            if s["top"]:
                # one sort that keeps the order of equal logits
                ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, : s["top"]]
                out += [logs.gather(1, ids), ids.to(torch.int32)]
        else:
            g, h = (s[k][lo:lo + 2048].double() * valid for k in ("dlogp", "dentropy"))
            onehot = torch.nn.functional.one_hot(target.clamp(min=0), V).double()
            d = scale * (g[:, None] * (onehot - p) - h[:, None] * p * (logs + entropy[:, None]))
            out = [logp, entropy, torch.matmul(d, table)]
            dtable += torch.matmul(d.t(), hidden)
        parts.append(out)
    whole = [torch.cat(x) for x in zip(*parts)]
    return whole + [dtable] if op == "logprobs_grad" else whole
