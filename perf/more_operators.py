"""Measured cases of the operators around the end of a language model's step.

* log-probabilities of given tokens from hidden states and the vocabulary's
  weights, without the logits: scoring (``score``), and a training step with
  both gradients (``step``);
* root-mean-square norm with the residual's addition (``norm``), with an
  output in 8 bits and its scales (``norm_quant``), and its backward pass
  (``norm_grad``);
* the balance loss of a router of experts with the experts' counts and its
  gradient (``balance``).

``run`` computes them in plain torch (``own`` false) or through the package's
entry points (``own`` true); ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_PRODUCT = 8192 * 4096 * 65536  # rows * dim * vocab of the largest step
_MATRIX = 1 << 27  # rows * len of the largest norm
_TOP = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token of an answer scored against a vocabulary: latency, the weights read once
        dict(name="score-1x2048x65536", op="score", rows=1, dim=2048, vocab=65536, dtype="bf16", scale=1.0,
             ignored=0.0, z=0.0),
        # a reference model's pass over packed answers: odd rows and vocabulary, prompts ignored, a temperature
        dict(name="score-2777x1024x50257", op="score", rows=2777, dim=1024, vocab=50257, dtype="f16", scale=0.8,
             ignored=0.25, z=0.0),
        # the smallest training step: a few tokens, the weights and their gradient are all there is to move
        dict(name="step-64x1024x32001", op="step", rows=64, dim=1024, vocab=32001, dtype="bf16", scale=1.0,
             ignored=0.0, z=0.0),
        # an ordinary micro-batch in half precision with a loss scale and a penalty on the normaliser
        dict(name="step-3001x2048x50257", op="step", rows=3001, dim=2048, vocab=50257, dtype="f16", scale=1.0,
             ignored=0.1, z=1e-4),
        # a full training step over packed sequences whose prompts are ignored
        dict(name="step-8192x4096x65536", op="step", rows=8192, dim=4096, vocab=65536, dtype="bf16", scale=1.0,
             ignored=0.25, z=0.0),
        # one token between two layers: latency
        dict(name="norm-1x4096", op="norm", rows=1, len=4096, pad=0, dtype="bf16", wtype="bf16", residual=True),
        # a prompt's activations for 8-bit products, a scale for each 128 values
        dict(name="norm-quant-4097x5120", op="norm_quant", rows=4097, len=5120, pad=0, dtype="bf16", wtype="bf16",
             residual=True, kind="e4m3", block=128),
        # a full batch in training
        dict(name="norm-16384x8192", op="norm", rows=16384, len=8192, pad=0, dtype="bf16", wtype="f32", residual=True),
        # backward of a norm over heads: many short rows, odd length, no residual
        dict(name="norm-grad-30001x127", op="norm_grad", rows=30001, len=127, pad=1, dtype="f32", wtype="f32",
             residual=False),
        # backward of a full batch
        dict(name="norm-grad-16384x4096", op="norm_grad", rows=16384, len=4096, pad=0, dtype="bf16", wtype="f32",
             residual=True),
        # a small batch's router
        dict(name="balance-257x64", op="balance", rows=257, len=64, k=6, dtype="f32", kind="softmax", ignored=0.1,
             z=1e-3),
        # a full batch's router
        dict(name="balance-65536x256", op="balance", rows=65536, len=256, k=8, dtype="f32", kind="sigmoid",
             ignored=0.05, z=0.0),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "step", "step", "norm", "norm_quant", "norm_grad", "balance"])
    if op in ("score", "step"):
        dim = 8 * _log_uniform(rng, 16, 1024)
        vocab = _log_uniform(rng, 257, min(131072, (1 << 28) // dim))
        return dict(op=op, rows=_log_uniform(rng, 1, min(16384, _PRODUCT // (dim * vocab))), dim=dim, vocab=vocab,
                    dtype=rng.choice(["bf16", "bf16", "f16"]), scale=rng.choice([0.7, 1.0, 1.0, 1.25]),
                    ignored=rng.choice([0.0, 0.1, 0.25, 0.4]), z=rng.choice([0.0, 1e-4]) if op == "step" else 0.0)
    if op == "balance":
        experts = _log_uniform(rng, 8, 512)
        return dict(op=op, rows=_log_uniform(rng, 1, min(131072, (1 << 24) // experts)), len=experts,
                    k=min(experts // 2, rng.choice([1, 2, 4, 6, 8])), dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                    kind=rng.choice(["softmax", "softmax", "sigmoid"]), ignored=rng.choice([0.0, 0.05, 0.3]),
                    z=rng.choice([0.0, 1e-3]))
    length = _log_uniform(rng, 64, 16384)
    if rng.random() < 0.7:
        length += -length % 64
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    case = dict(op=op, rows=_log_uniform(rng, 1, min(65536, _MATRIX // length)), len=length,
                pad=rng.choice([0, 0, 8, 64]), dtype=dtype, wtype=rng.choice([dtype, "f32"]),
                residual=rng.random() < 0.7)
    if op == "norm_quant":
        case.update(kind=rng.choice(["e4m3", "e4m3", "int8"]), block=rng.choice([0, 0, 64, 128]))
    return case


def _live(case):
    return case["rows"] - int(case["rows"] * case["ignored"])


def work(case):
    """Scoring: the weights and the live rows' hidden states once, one product.
    A step: both read once, both gradients written once, three products.  The
    norms: each matrix once.  The balance loss: the live rows' logits and ids
    once, the gradient once."""
    op, rows = case["op"], case["rows"]
    size = _BYTES[case["dtype"]]
    if op in ("score", "step"):
        dim, vocab, live = case["dim"], case["vocab"], _live(case)
        read = (vocab + live) * dim * size + 16 * rows
        if op == "score":
            return {"bytes": read, "flops": 2 * live * dim * vocab}
        return {"bytes": read + (vocab + rows) * dim * size, "flops": 6 * live * dim * vocab}
    n = rows * case["len"]
    if op == "norm":
        return {"bytes": n * size * (4 if case["residual"] else 2) + 4 * rows, "flops": 6 * n}
    if op == "norm_quant":
        block = case["block"] or case["len"]
        scales = rows * -(-case["len"] // block)
        return {"bytes": n * size * (3 if case["residual"] else 1) + n + 4 * rows + 4 * scales, "flops": 9 * n}
    if op == "norm_grad":
        return {"bytes": n * size * (4 if case["residual"] else 3) + 4 * rows, "flops": 10 * n}
    live = _live(case)
    return {"bytes": (live + rows) * case["len"] * size + 8 * live * case["k"] + rows, "flops": 10 * live * case["len"]}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype, rows, op = _DTYPES[case["dtype"]], case["rows"], case["op"]
    state = dict(case=case)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def out_of(n):
        """n of the rows, at random."""
        return torch.randperm(rows, generator=gen, device=dev)[:n]

    if op in ("score", "step"):
        dim, vocab = case["dim"], case["vocab"]
        # logits are a bell of width 1.5 and, at most positions, the target's is well above it
        weight = (randn(vocab, dim) * (1.5 / math.sqrt(dim))).to(dtype)
        target = torch.randint(0, vocab, (rows,), generator=gen, device=dev)
        lift = torch.rand((rows, 1), generator=gen, device=dev) * 6.0
        hidden = (randn(rows, dim) + weight[target].float() * lift).to(dtype)
        out = out_of(rows - _live(case))
        target[out] = -100
        state.update(hidden=hidden, weight=weight, target=target)
        if op == "step":
            # the mean over the live rows; half precision trains with a loss scale
            state["unit"] = (65536.0 if case["dtype"] == "f16" else 1.0) / max(1, _live(case))
            state["dlogp"] = torch.full((rows,), -state["unit"], device=dev)
    elif op == "balance":
        x = randn(rows, case["len"]) * 1.5 + randn(case["len"]) * 0.5
        state["x"] = x.to(dtype)
        state["ids"] = torch.topk(state["x"].float(), case["k"], 1).indices
        state["live"] = torch.ones(rows, dtype=torch.bool, device=dev)
        state["live"][out_of(rows - _live(case))] = False
        state["grad_scale"] = 65536.0 if case["dtype"] == "f16" else 1.0
    else:
        length, pad = case["len"], case["pad"]

        def matrix(width=1.0):
            whole = torch.full((rows, length + pad), float("nan"), dtype=dtype, device=dev)
            whole[:, :length] = randn(rows, length) * width
            return whole[:, :length]

        state["x"] = matrix()
        # the residual stream holds a few channels of large values
        state["residual"] = None
        if op != "norm_grad" and case["residual"]:
            state["residual"] = matrix(2.0)
            state["residual"][:, ::97] *= 12.0
        state["weight"] = (1.0 + 0.2 * randn(length)).to(_DTYPES[case["wtype"]])
        if op == "norm_grad":
            state["x"][:, ::97] *= 12.0
            state["rstd"] = torch.rsqrt(state["x"].float().square().mean(1) + 1e-6)
            state["dy"] = matrix()
            state["dtotal"] = matrix() if case["residual"] else None
    return state


# ----------------------------------------------------------- the operators

def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_score(s):
    import int_tensor_reductions_gb300 as itr
    return itr.red_linear_logprob(s["hidden"], s["weight"], s["target"], scale=s["case"]["scale"])


def _own_step(s):
    import int_tensor_reductions_gb300 as itr
    scale, z = s["case"]["scale"], s["case"]["z"]
    logp, lse = itr.red_linear_logprob(s["hidden"], s["weight"], s["target"], scale=scale)
    dlse = lse * (2.0 * z * s["unit"]) if z else None
    dhidden, dweight = itr.red_linear_logprob_grad(s["hidden"], s["weight"], s["target"], lse, s["dlogp"], dlse=dlse,
                                                   scale=scale)
    return logp, lse, dhidden, dweight


def _own_norm(s):
    import int_tensor_reductions_gb300 as itr
    return itr.red_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=1e-6)


def _own_norm_quant(s):
    import int_tensor_reductions_gb300 as itr
    c = s["case"]
    q, scales, total, rstd = itr.red_rmsnorm_quant(s["x"], s["weight"], residual=s["residual"], eps=1e-6,
                                                   kind=c["kind"], block=c["block"])
    return q.bfloat16(), scales, total, rstd  # what the 8 bits stand for, exactly


def _own_norm_grad(s):
    import int_tensor_reductions_gb300 as itr
    return itr.red_rmsnorm_grad(s["dy"], s["x"], s["rstd"], s["weight"], dtotal=s["dtotal"])


def _own_balance(s):
    import int_tensor_reductions_gb300 as itr
    c = s["case"]
    return itr.red_balance(s["x"], s["ids"], live=s["live"], coef=0.01, z_coef=_z(c), kind=c["kind"],
                           grad_scale=s["grad_scale"])


_OWN = {"score": _own_score, "step": _own_step, "norm": _own_norm, "norm_quant": _own_norm_quant,
        "norm_grad": _own_norm_grad, "balance": _own_balance}


def _z(case):
    return case["z"] if case["kind"] == "softmax" else 0.0


def _plain_logits(s):
    """(live rows, hidden states, weights, scaled logits, log-sum-exp, targets, log-probabilities) in 32 bits."""
    target = s["target"]
    rows = (target >= 0).nonzero()[:, 0]
    h, w = s["hidden"][rows].float(), s["weight"].float()
    z = (h @ w.t()) * s["case"]["scale"]
    top = z.max(1, keepdim=True).values
    lse = top + (z - top).exp().sum(1, keepdim=True).log()
    at = target[rows][:, None]
    return rows, h, w, z, lse, at, z.gather(1, at) - lse


def _plain_vectors(s, rows, logp, lse):
    zero = torch.zeros(s["target"].shape[0], device=logp.device)
    return zero.index_copy(0, rows, logp[:, 0]), zero.index_copy(0, rows, lse[:, 0])


def _plain_score(s):
    rows, _, _, _, lse, _, logp = _plain_logits(s)
    return _plain_vectors(s, rows, logp, lse)


def _plain_step(s):
    rows, h, w, z, lse, at, logp = _plain_logits(s)
    scale, zc = s["case"]["scale"], s["case"]["z"]
    d = s["dlogp"][rows][:, None]
    g = (z - lse).exp() * (lse * (2.0 * zc * s["unit"]) - d)
    g.scatter_add_(1, at, d)
    g = g * scale
    dhidden = torch.zeros_like(s["hidden"])
    dhidden[rows] = (g @ w).to(dhidden.dtype)
    dweight = (g.t() @ h).to(s["weight"].dtype)
    return *_plain_vectors(s, rows, logp, lse), dhidden, dweight


def _plain_normalised(s):
    """(x + residual, 1 / root mean square, normalised and weighted) in 32 bits."""
    t = s["x"].float()
    if s["residual"] is not None:
        t = t + s["residual"].float()
    rstd = torch.rsqrt((t * t).mean(1) + 1e-6)
    return t, rstd, t * rstd[:, None] * s["weight"].float()


def _plain_total(s, t):
    return t.to(s["x"].dtype) if s["residual"] is not None else None


def _plain_norm(s):
    t, rstd, y = _plain_normalised(s)
    return y.to(s["x"].dtype), _plain_total(s, t), rstd


def _blocks(y, block):
    """y in blocks of the last axis, filled up with zeros."""
    block = block or y.shape[1]
    return torch.nn.functional.pad(y, (0, -y.shape[1] % block)).view(y.shape[0], -1, block)


def _plain_norm_quant(s):
    c = s["case"]
    t, rstd, y = _plain_normalised(s)
    parts = _blocks(y, c["block"])
    top = parts.abs().amax(2)
    scales = torch.where(top > 0, top / _TOP[c["kind"]], torch.ones_like(top))
    q = (parts / scales[:, :, None]).clamp(-_TOP[c["kind"]], _TOP[c["kind"]])
    q = q.to(torch.float8_e4m3fn).float() if c["kind"] == "e4m3" else q.round()
    return q.reshape(y.shape[0], -1)[:, :y.shape[1]].bfloat16(), scales, _plain_total(s, t), rstd


def _plain_norm_grad(s):
    rstd = s["rstd"][:, None]
    xhat = s["x"].float() * rstd
    dy = s["dy"].float()
    g = dy * s["weight"].float()
    dx = (g - xhat * (g * xhat).mean(1, keepdim=True)) * rstd
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"].float()
    return dx.to(s["x"].dtype), (dy * xhat).sum(0).to(s["weight"].dtype)


def _plain_balance(s):
    c, x, ids = s["case"], s["x"].float(), s["ids"]
    experts, live = c["len"], s["live"][:, None]
    counts = torch.zeros(experts, dtype=torch.int64, device=x.device)
    counts = counts.index_add(0, ids.reshape(-1), live.expand_as(ids).reshape(-1).long())
    n = live.sum().clamp(min=1).float()
    top = x.max(1, keepdim=True).values
    e = (x - top).exp()
    total = e.sum(1, keepdim=True)
    lse = top + total.log()
    if c["kind"] == "softmax":
        p = e / total
        slope = p
    else:
        sig = 1.0 / (1.0 + (-x).exp())
        p = sig / sig.sum(1, keepdim=True)
        slope = p / (1.0 + x.exp())
    zero = torch.zeros_like(x)
    prob = torch.where(live, p, zero).sum(0) / n
    share = counts.float() / (n * c["k"])
    balance = experts * (share * prob).sum()
    z = torch.where(live, lse * lse, torch.zeros_like(lse)).sum() / n if c["kind"] == "softmax" else torch.zeros_like(n)
    zc = _z(c)
    loss = 0.01 * balance + zc * z
    by_p = 0.01 * experts * share / n
    g = slope * (by_p - (p * by_p).sum(1, keepdim=True)) + (2.0 * zc / n) * lse * p
    g = torch.where(live, g * s["grad_scale"], zero)
    return counts, prob, torch.stack([loss, balance, z, live.sum().float()]), g.to(s["x"].dtype)


_PLAIN = {"score": _plain_score, "step": _plain_step, "norm": _plain_norm, "norm_quant": _plain_norm_quant,
          "norm_grad": _plain_norm_grad, "balance": _plain_balance}


# ------------------------------------------------------ 64-bit definitions

def exact(case, seed):
    """The definitions in 64 bits, gradients by automatic differentiation."""
    s = prepare(case, seed)
    return {"score": _exact_linear, "step": _exact_linear, "norm": _exact_norm, "norm_quant": _exact_norm,
            "norm_grad": _exact_norm_grad, "balance": _exact_balance}[case["op"]](s)


def _exact_linear(s):
    case, target = s["case"], s["target"]
    step = case["op"] == "step"
    logp = torch.zeros(target.shape[0], dtype=torch.float64, device=target.device)
    lse = torch.zeros_like(logp)
    weight = s["weight"].double().requires_grad_(step)
    dhidden = torch.zeros(s["hidden"].shape, dtype=torch.float64, device=target.device) if step else None
    live = torch.nonzero(target >= 0).flatten()
    for rows in live.split(max(1, (1 << 26) // case["vocab"])):
        hidden = s["hidden"][rows].double().requires_grad_(step)
        z = torch.nn.functional.linear(hidden, weight) * case["scale"]
        norm = torch.logsumexp(z, 1)
        taken = z[torch.arange(rows.numel(), device=rows.device), target[rows]] - norm
        if step:
            # the mean of -logp + z_coef * lse^2
            loss = (taken * s["dlogp"][rows].double()).sum() + case["z"] * s["unit"] * norm.square().sum()
            loss.backward()
            dhidden[rows] = hidden.grad
        logp[rows], lse[rows] = taken.detach(), norm.detach()
    if not step:
        return logp, lse
    if weight.grad is None:
        weight.grad = torch.zeros_like(weight)
    return logp, lse, dhidden, weight.grad


def _exact_norm(s):
    case = s["case"]
    total = s["x"].double()
    if s["residual"] is not None:
        total = total + s["residual"].double()
    rstd = (total.square().sum(1) / case["len"] + 1e-6) ** -0.5
    y = torch.einsum("rc,r,c->rc", total, rstd, s["weight"].double())
    kept = total if s["residual"] is not None else None
    if case["op"] == "norm":
        return y, kept, rstd
    block = case["block"] or case["len"]
    top = torch.stack([part.abs().max(1).values for part in y.split(block, 1)], 1)
    scales = torch.where(top == 0, 1.0, top / _TOP[case["kind"]])
    # the 8 bits are the nearest to y / scales in 32 bits: between two of them there is no nearer one
    return None, scales, kept, rstd


def _exact_norm_grad(s):
    x = s["x"].double().requires_grad_()
    weight = s["weight"].double().requires_grad_()
    # 1 / rms as given: it is the norm's own, a function of x
    mean = x.square().mean(1, keepdim=True)
    y = x / torch.sqrt(mean + 1e-6) * weight
    out = (y * s["dy"].double()).sum()
    if s["dtotal"] is not None:
        out = out + (x * s["dtotal"].double()).sum()
    out.backward()
    return x.grad, weight.grad


def _exact_balance(s):
    case = s["case"]
    rows = torch.nonzero(s["live"]).flatten()
    leaf = s["x"].double().requires_grad_()
    x = leaf[rows]
    counts = torch.bincount(s["ids"][rows].flatten(), minlength=case["len"])
    n = max(1, rows.numel())
    if case["kind"] == "softmax":
        p, z = torch.softmax(x, 1), torch.logsumexp(x, 1).square().sum() / n
    else:
        p = torch.sigmoid(x)
        p, z = p / p.sum(1, keepdim=True), x.sum() * 0.0
    prob = p.sum(0) / n
    balance = case["len"] * torch.dot(counts.double() / (n * case["k"]), prob)
    loss = 0.01 * balance + _z(case) * z
    (loss * s["grad_scale"]).backward()
    stats = torch.stack([loss.detach(), balance.detach(), z.detach(), torch.full_like(loss.detach(), rows.numel())])
    return counts, prob.detach(), stats, leaf.grad
