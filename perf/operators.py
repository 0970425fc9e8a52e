"""Measured cases of the losses over rows of logits.

Four operators, each a reduction over the vocabulary of every row of a
(rows, vocab) matrix of logits, with its gradient:

* log-probabilities of given tokens, forward (``logprob``) and backward
  (``logprob_grad``);
* distillation from a teacher's top logits, loss and gradient (``distill``);
* the clipped policy loss with a KL term, loss and gradient (``policy``);
* the preference loss of pairs of packed sequences, loss and gradient
  (``preference``).

``run`` computes them in plain torch (``own`` false) or through the package's
entry points (``own`` true); ``exact`` computes them in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_MAX_ELEMS = 1 << 29  # rows * vocab of the largest case


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token scored in an answering loop: latency
        dict(name="score-1x65536", op="logprob", rows=1, vocab=65536, pad=0, dtype="bf16", scale=1.0,
             ignored=0.0, masked=0),
        # a reference model's pass over a batch of packed answers: an odd vocabulary in rows padded to 64
        dict(name="score-4096x50257", op="logprob", rows=4096, vocab=50257, pad=47, dtype="f16", scale=1.0,
             ignored=0.25, masked=0),
        # scoring with a small vocabulary (bytes or a codebook): many short rows
        dict(name="score-65536x1024", op="logprob", rows=65536, vocab=1024, pad=0, dtype="f32", scale=0.7,
             ignored=0.1, masked=0),
        # backward of the log-probabilities in a training step, odd rows without padding
        dict(name="score-grad-3001x32001", op="logprob_grad", rows=3001, vocab=32001, pad=0, dtype="bf16",
             scale=1.0, ignored=0.2, masked=0),
        # a small distillation micro-batch, odd vocabulary, stored top-20 logits with the teacher's normaliser
        dict(name="distill-257x32001", op="distill", rows=257, vocab=32001, pad=0, dtype="f16", scale=0.5,
             ignored=0.1, masked=0, k=20, teacher="f16", normalised=True),
        # a full distillation step: long vocabulary, top-64 renormalised
        dict(name="distill-4096x65536", op="distill", rows=4096, vocab=65536, pad=0, dtype="bf16", scale=1.0,
             ignored=0.05, masked=64, k=64, teacher="bf16", normalised=False),
        # one short group of sampled tokens: the smallest update
        dict(name="policy-64x65536", op="policy", rows=64, vocab=65536, pad=0, dtype="bf16", scale=1.0,
             ignored=0.0, masked=64, kl=0.05),
        # logits kept in 32 bits, sampled at a temperature
        dict(name="policy-1000x32001", op="policy", rows=1000, vocab=32001, pad=0, dtype="f32", scale=1.25,
             ignored=0.2, masked=0, kl=0.04),
        # a full policy step over packed answers whose prompts are masked out, without the KL term
        dict(name="policy-8192x65536", op="policy", rows=8192, vocab=65536, pad=0, dtype="bf16", scale=1.0,
             ignored=0.25, masked=0, kl=0.0),
        # two short pairs: the smallest preference step
        dict(name="preference-2x190x16384", op="preference", rows=190, vocab=16384, pad=0, dtype="f32", scale=1.0,
             ignored=0.3, masked=0, pairs=2, kind="sigmoid", average=False, reference=True),
        # an ordinary micro-batch of pairs, odd vocabulary in padded rows, length-averaged without a reference
        dict(name="preference-8x2777x50257", op="preference", rows=2777, vocab=50257, pad=47, dtype="f16",
             scale=1.0, ignored=0.2, masked=0, pairs=8, kind="sigmoid", average=True, reference=False),
        # a full preference step
        dict(name="preference-16x8192x65536", op="preference", rows=8192, vocab=65536, pad=0, dtype="bf16",
             scale=1.0, ignored=0.3, masked=0, pairs=16, kind="sigmoid", average=False, reference=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprob", "logprob_grad", "distill", "policy", "preference"])
    vocab = _log_uniform(rng, 257, 131072)
    if rng.random() < 0.5:
        vocab += 32 - vocab % 64  # rows of whole 64-byte blocks
    rows = _log_uniform(rng, 1, min(65536, _MAX_ELEMS // vocab))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    case = dict(op=op, rows=rows, vocab=vocab, pad=(-vocab) % 64 if rng.random() < 0.4 else 0, dtype=dtype,
                scale=rng.choice([0.5, 0.7, 1.0, 1.0, 1.25]), ignored=rng.choice([0.0, 0.1, 0.25, 0.4]),
                masked=rng.choice([0, 0, 64]))
    if op == "distill":
        case.update(k=_log_uniform(rng, 1, 128), teacher=rng.choice(["f32", "bf16", "f16"]),
                    normalised=rng.random() < 0.5)
    elif op == "policy":
        case.update(kl=rng.choice([0.0, 0.01, 0.05]))
    elif op == "preference":
        rows = case["rows"] = max(2, rows)
        case.update(pairs=min(_log_uniform(rng, 1, 64), rows // 2), kind=rng.choice(["sigmoid", "hinge", "squared"]),
                    average=rng.random() < 0.4, reference=rng.random() < 0.7)
    return case


def work(case):
    """Bytes: the logits of the rows that take part once, the gradient of all
    rows once, and the per-row vectors.  Flops: about 4 per element and
    direction (scale, subtract, exponential, sum or product)."""
    rows, vocab = case["rows"], case["vocab"]
    size = _BYTES[case["dtype"]]
    live = rows - int(rows * case["ignored"])
    logits, grad = live * vocab * size, rows * vocab * size
    elems = live * vocab
    op = case["op"]
    if op == "logprob":
        return {"bytes": logits + 16 * rows, "flops": 4 * elems}
    if op == "logprob_grad":
        return {"bytes": logits + grad + 16 * rows, "flops": 4 * elems}
    if op == "distill":
        teacher = rows * case["k"] * (8 + _BYTES[case["teacher"]])
        return {"bytes": logits + grad + teacher + 12 * rows, "flops": 8 * elems}
    if op == "policy":
        return {"bytes": logits + grad + 32 * rows, "flops": 8 * elems}
    return {"bytes": logits + grad + 8 * rows + 40 * case["pairs"], "flops": 8 * elems}


# ------------------------------------------------------------------ inputs

def _chunks(rows, vocab, elems=1 << 26):
    step = max(1, elems // vocab)
    for lo in range(0, rows, step):
        yield slice(lo, min(rows, lo + step))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    rows, vocab, pad = case["rows"], case["vocab"], case["pad"]
    dtype, scale = _DTYPES[case["dtype"]], case["scale"]

    # logits: a bell of width 2.5 and, at most positions, one token well above it; padding columns hold garbage
    whole = torch.full((rows, vocab + pad), float("nan"), dtype=dtype, device=dev)
    x = whole[:, :vocab]
    usable = vocab - case["masked"]
    target = torch.randint(0, usable, (rows,), generator=gen, device=dev)
    lift = torch.rand(rows, generator=gen, device=dev) * 14.0
    logp = torch.empty(rows, device=dev)
    for part in _chunks(rows, vocab):
        z = torch.randn((part.stop - part.start, vocab), generator=gen, device=dev) * 2.5
        at = torch.arange(z.shape[0], device=dev)
        z[at, target[part]] += lift[part]
        if case["masked"]:
            z[:, usable:] = -math.inf  # entries that pad the vocabulary
        x[part] = z.to(dtype)
        z = x[part].float() * scale
        logp[part] = z[at, target[part]] - torch.logsumexp(z, 1)

    n_out = int(rows * case["ignored"])
    out = torch.randperm(rows, generator=gen, device=dev)[:n_out]
    live = torch.ones(rows, device=dev)
    live[out] = 0.0
    state = dict(case=case, x=x, target=target)
    size = 1.0 / max(1, rows - n_out)
    # f16 gradients are trained with a loss scale: the mean over rows would underflow
    state["grad_scale"] = 1.0
    if case["dtype"] == "f16":
        state["grad_scale"] = 1024.0 if case["op"] == "preference" else min(65536.0, 1024.0 * (rows - n_out))
    if pad and case["op"] != "logprob":
        # a program with padded rows keeps the gradient in such rows too
        state["grad"] = torch.empty_like(whole)[:, :vocab]

    op = case["op"]
    if op in ("logprob", "logprob_grad"):
        target[out] = -100
        if op == "logprob_grad":
            state["dlogp"] = torch.randn(rows, generator=gen, device=dev)
            lse = torch.zeros(rows, device=dev)
            for part in _chunks(rows, vocab):
                lse[part] = torch.logsumexp(x[part].float() * scale, 1)
            state["lse"] = torch.where(live > 0, lse, torch.zeros_like(lse))
    elif op == "distill":
        k = case["k"]
        ids = torch.empty((rows, k), dtype=torch.int64, device=dev)
        vals = torch.empty((rows, k), dtype=_DTYPES[case["teacher"]], device=dev)
        lse = torch.empty(rows, device=dev)
        for part in _chunks(rows, vocab):
            # the teacher disagrees with the student by noise of width 1
            z = x[part].float()
            z = z + torch.randn(z.shape, generator=gen, device=dev)
            top = torch.topk(z, k, 1)
            ids[part], vals[part] = top.indices, top.values.to(vals.dtype)
            lse[part] = torch.logsumexp(z * scale, 1)
        # some rows hold fewer than k tokens
        short = torch.rand((rows, 1), generator=gen, device=dev) < 0.1
        ids[short & (torch.arange(k, device=dev) >= (k + 1) // 2)] = -1
        state.update(ids=ids, vals=vals, lse=lse if case["normalised"] else None, weight=live * size)
        del state["target"]
    elif op == "policy":
        target[out] = -100  # prompt tokens
        # the sampling policy and the reference are near the present one
        state["old"] = logp + torch.randn(rows, generator=gen, device=dev) * 0.2
        state["ref"] = logp + torch.randn(rows, generator=gen, device=dev) * 0.3 if case["kl"] else None
        state["adv"] = torch.randn(rows, generator=gen, device=dev)
        state["weight"] = torch.full((rows,), size, device=dev)
    else:
        pairs = case["pairs"]
        # 2 * pairs sequences of random lengths, none empty, that fill the rows
        cuts = torch.randperm(rows - 1, generator=cpu)[:2 * pairs - 1].sort().values + 1
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.full((1,), rows, dtype=torch.int64)])
        start, length = offsets[:-1], offsets[1:] - offsets[:-1]
        prompt = (length.double() * case["ignored"]).long()
        seq = torch.repeat_interleave(torch.arange(2 * pairs), length)
        target[(torch.arange(rows) - start[seq] < prompt[seq]).to(dev)] = -100
        state["offsets"] = offsets.to(dev)
        count = (length - prompt).to(dev).float()
        taken = torch.where(target >= 0, logp, torch.zeros_like(logp)).double().cpu().numpy()
        sums = torch.from_numpy(np.add.reduceat(taken, offsets[:-1].numpy())).float().to(dev)
        # the reference model's sums differ by a few nats (per token where lengths are averaged)
        sums = sums + torch.randn(2 * pairs, generator=gen, device=dev) * 0.5 * count.sqrt()
        if case["average"]:
            sums = sums / count
        state["ref"] = sums if case["reference"] else None
        state["beta"] = 2.0 if case["average"] else 0.1
        state["margin"] = 0.5 if case["average"] else 0.0
        state["weight"] = torch.full((pairs,), 1.0 / pairs, device=dev)
    return state


# ----------------------------------------------------------- the operators

def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_logprob(s):
    import int_tensor_reductions_gb300 as itr
    return itr.red_logprob(s["x"], s["target"], scale=s["case"]["scale"])


def _own_logprob_grad(s):
    import int_tensor_reductions_gb300 as itr
    return itr.red_logprob_grad(s["x"], s["target"], s["lse"], s["dlogp"], scale=s["case"]["scale"],
                                out=s.get("grad"))


def _own_distill(s):
    import int_tensor_reductions_gb300 as itr
    return itr.red_distill(s["x"], s["ids"], s["vals"], lse=s["lse"], weight=s["weight"], scale=s["case"]["scale"],
                           grad_scale=s["grad_scale"], grad=s.get("grad"))


def _own_policy(s):
    import int_tensor_reductions_gb300 as itr
    return itr.red_policy(s["x"], s["target"], s["old"], s["adv"], ref_logp=s["ref"], weight=s["weight"],
                          clip_low=0.2, clip_high=0.28, kl_coef=s["case"]["kl"], scale=s["case"]["scale"],
                          grad_scale=s["grad_scale"], grad=s.get("grad"))


def _own_preference(s):
    import int_tensor_reductions_gb300 as itr
    c = s["case"]
    return itr.red_preference(s["x"], s["target"], s["offsets"], ref_logp=s["ref"], weight=s["weight"],
                              kind=c["kind"], beta=s["beta"], margin=s["margin"], smoothing=0.1 * (c["kind"] == "sigmoid"),
                              average=c["average"], scale=c["scale"], grad_scale=s["grad_scale"],
                              grad=s.get("grad"))


_OWN = {"logprob": _own_logprob, "logprob_grad": _own_logprob_grad, "distill": _own_distill,
        "policy": _own_policy, "preference": _own_preference}


def _softmax(x, scale):
    """(scaled logits minus the row's maximum, exponentials, their sum, maximum) in 32 bits."""
    z = x.float() * scale
    top = z.max(1, keepdim=True).values
    z = z - top
    e = z.exp()
    return z, e, e.sum(1, keepdim=True), top


def _plain_logprob(s):
    x, target = s["x"], s["target"]
    live = (target >= 0) & (target < x.shape[1])
    at = torch.where(live, target, torch.zeros_like(target))[:, None]
    z, _, total, top = _softmax(x, s["case"]["scale"])
    zero = torch.zeros_like(total)
    logp = torch.where(live[:, None], z.gather(1, at) - total.log(), zero)
    lse = torch.where(live[:, None], top + total.log(), zero)
    return logp[:, 0], lse[:, 0]


def _plain_logprob_grad(s):
    x, target, scale = s["x"], s["target"], s["case"]["scale"]
    live = (target >= 0) & (target < x.shape[1])
    p = (x.float() * scale - s["lse"][:, None]).exp()
    c = torch.where(live, s["dlogp"] * scale, torch.zeros_like(s["dlogp"]))
    g = torch.where(live[:, None], p * -c[:, None], torch.zeros_like(p))
    at = torch.where(live, target, torch.zeros_like(target))
    rows = torch.arange(x.shape[0], device=x.device)
    g[rows, at] += c
    return g.to(x.dtype)


def _plain_distill(s):
    x, ids, scale = s["x"], s["ids"], s["case"]["scale"]
    z, e, total, _ = _softmax(x, scale)
    kept = (ids >= 0) & (ids < x.shape[1])
    at = torch.where(kept, ids, torch.zeros_like(ids))
    v = s["vals"].float() * scale
    v = torch.where(kept, v, torch.full_like(v, -math.inf))
    if s["lse"] is None:
        v = v - v.max(1, keepdim=True).values
        logq = v - v.exp().sum(1, keepdim=True).log()
    else:
        logq = v - s["lse"][:, None]
    q = logq.exp()
    logp = z.gather(1, at) - total.log()
    terms = torch.where(q > 0, q * (logq - logp), torch.zeros_like(q))
    w = s["weight"]
    loss = terms.sum(1) * w
    g = e / total * q.sum(1, keepdim=True)
    g.scatter_add_(1, at, -q)
    g = torch.where(w[:, None] != 0, g * (w * (s["grad_scale"] * scale))[:, None], torch.zeros_like(g))
    return loss, torch.stack([loss.sum(), w.sum()]), g.to(x.dtype)


def _plain_policy(s):
    x, target, scale, kl = s["x"], s["target"], s["case"]["scale"], s["case"]["kl"]
    z, e, total, _ = _softmax(x, scale)
    live = (target >= 0) & (target < x.shape[1])
    at = torch.where(live, target, torch.zeros_like(target))
    zero = torch.zeros_like(s["adv"])
    logp = torch.where(live, (z.gather(1, at[:, None]) - total.log())[:, 0], zero)
    w = torch.where(live, s["weight"], zero)
    adv = s["adv"]
    ratio = (logp - s["old"]).exp()
    one, two = ratio * adv, ratio.clamp(1.0 - 0.2, 1.0 + 0.28) * adv
    clipped = one > two
    loss, c = -torch.where(clipped, two, one), torch.where(clipped, zero, -one)
    drift = zero
    if kl:
        d = s["ref"] - logp
        drift = d.exp() - d - 1.0
        loss, c = loss + kl * drift, c + kl * (1.0 - d.exp())
    loss = loss * w
    stats = torch.stack([loss.sum(), (drift * w).sum(), (clipped * w).sum(), w.sum()])
    c = c * w * (s["grad_scale"] * scale)
    g = e / total * -c[:, None]
    g[torch.arange(x.shape[0], device=x.device), at] += c
    return loss, logp, stats, torch.where(live[:, None], g, torch.zeros_like(g)).to(x.dtype)


def _plain_preference(s):
    x, target, scale, case = s["x"], s["target"], s["case"]["scale"], s["case"]
    pairs, beta = case["pairs"], s["beta"]
    z, e, total, _ = _softmax(x, scale)
    live = (target >= 0) & (target < x.shape[1])
    at = torch.where(live, target, torch.zeros_like(target))
    logp = (z.gather(1, at[:, None]) - total.log())[:, 0]
    rows = torch.arange(x.shape[0], device=x.device)
    seq = torch.bucketize(rows, s["offsets"][1:], right=True)
    member = (seq[None, :] == torch.arange(2 * pairs, device=x.device)[:, None]) & live[None, :]
    sums = torch.where(member, logp[None, :], torch.zeros_like(logp)[None, :]).sum(1)
    count = member.sum(1).float().clamp(min=1.0) if case["average"] else torch.ones_like(sums)
    sums = sums / count
    gain = sums if s["ref"] is None else sums - s["ref"]
    u = beta * (gain[:pairs] - gain[pairs:]) - s["margin"]
    if case["kind"] == "sigmoid":
        eps = 0.1
        soft = (1.0 + (-u.abs()).exp()).log()
        loss = (1.0 - eps) * (soft + (-u).clamp(min=0.0)) + eps * (soft + u.clamp(min=0.0))
        du = eps - 1.0 / (1.0 + u.exp())
    elif case["kind"] == "hinge":
        loss, du = (1.0 - u).clamp(min=0.0), torch.where(u < 1.0, -torch.ones_like(u), torch.zeros_like(u))
    else:
        off = (u - 0.5) / beta
        loss, du = off * off, 2.0 * off / beta
    w = s["weight"]
    loss = loss * w
    stats = torch.stack([loss.sum(), (u * w).sum(), ((u > 0) * w).sum(), w.sum()])
    c = torch.cat([du * w, -du * w]) * (beta * s["grad_scale"] * scale) / count
    c = torch.where(live, c[seq], torch.zeros_like(logp))
    g = e / total * -c[:, None]
    g[rows, at] += c
    return loss, sums, stats, torch.where(live[:, None], g, torch.zeros_like(g)).to(x.dtype)


_PLAIN = {"logprob": _plain_logprob, "logprob_grad": _plain_logprob_grad, "distill": _plain_distill,
          "policy": _plain_policy, "preference": _plain_preference}


# ------------------------------------------------------ 64-bit definitions

def exact(case, seed):
    """The definitions in 64 bits, gradients by automatic differentiation, a block of rows at a time."""
    s = prepare(case, seed)
    return {"logprob": _exact_logprob, "logprob_grad": _exact_logprob_grad, "distill": _exact_distill,
            "policy": _exact_policy, "preference": _exact_preference}[case["op"]](s)


def _exact_rows(s, rows):
    """log-softmax of some rows, with the leaf that its gradient goes to."""
    leaf = s["x"][rows].double().requires_grad_()
    return leaf, torch.log_softmax(leaf * s["case"]["scale"], 1)


def _exact_logprob(s):
    x, target = s["x"], s["target"]
    logp = torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    lse = torch.zeros_like(logp)
    for part in _chunks(*x.shape):
        rows = torch.arange(part.start, part.stop, device=x.device)[target[part] >= 0]
        z = x[rows].double() * s["case"]["scale"]
        lse[rows] = torch.logsumexp(z, 1)
        logp[rows] = z.gather(1, target[rows, None])[:, 0] - lse[rows]
    return logp, lse


def _exact_backward(s, dlogp, scale=1.0):
    """sum_t dlogp_t * logp_t, differentiated by the logits, times scale."""
    x, target = s["x"], s["target"]
    grad = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for part in _chunks(*x.shape):
        rows = torch.arange(part.start, part.stop, device=x.device)[target[part] >= 0]
        leaf, logp = _exact_rows(s, rows)
        (logp.gather(1, target[rows, None])[:, 0] * dlogp[rows]).sum().backward()
        grad[rows] = leaf.grad * scale
    return grad


def _exact_logprob_grad(s):
    return _exact_backward(s, s["dlogp"].double())


def _exact_distill(s):
    x, scale = s["x"], s["case"]["scale"]
    w = s["weight"].double()
    loss = torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    grad = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for part in _chunks(*x.shape):
        rows = torch.arange(part.start, part.stop, device=x.device)[s["weight"][part] != 0]
        leaf, logp = _exact_rows(s, rows)
        kept = s["ids"][rows] >= 0
        v = (s["vals"][rows].double() * scale).masked_fill(~kept, -math.inf)
        norm = torch.logsumexp(v, 1) if s["lse"] is None else s["lse"][rows].double()
        logq = v - norm[:, None]
        gap = logq.masked_fill(~kept, 0.0) - logp.gather(1, s["ids"][rows].clamp(min=0))
        each = (logq.exp() * torch.where(kept, gap, torch.zeros_like(gap))).sum(1) * w[rows]
        each.sum().backward()
        loss[rows], grad[rows] = each.detach(), leaf.grad * s["grad_scale"]
    return loss, torch.stack([loss.sum(), w.sum()]), grad


def _exact_policy(s):
    kl, target = s["case"]["kl"], s["target"]
    taken, _ = _exact_logprob(s)
    live = target >= 0
    w = s["weight"].double() * live
    logp = taken.clone().requires_grad_()
    ratio = torch.exp(logp - s["old"].double())
    adv = s["adv"].double()
    bound = torch.clamp(ratio, 1.0 - 0.2, 1.0 + 0.28)
    gain = torch.minimum(ratio * adv, bound * adv)
    drift = torch.zeros_like(taken)
    if kl:
        d = s["ref"].double() - logp
        drift = torch.expm1(d) - d
    loss = (kl * drift - gain) * w
    loss.sum().backward()
    clipped = (ratio * adv > bound * adv).double()
    loss = loss.detach()
    stats = torch.stack([loss.sum(), (drift * w).sum().detach(), (clipped * w).sum(), w.sum()])
    return loss, taken, stats, _exact_backward(s, logp.grad, s["grad_scale"])


def _exact_preference(s):
    case, target = s["case"], s["target"]
    pairs, beta = case["pairs"], s["beta"]
    logp, _ = _exact_logprob(s)
    logp.requires_grad_()
    bounds = s["offsets"].tolist()
    sums = []
    for lo, hi in zip(bounds[:-1], bounds[1:]):
        n = max(1, int((target[lo:hi] >= 0).sum())) if case["average"] else 1
        sums.append(logp[lo:hi].sum() / n)
    sums = torch.stack(sums)
    gain = sums if s["ref"] is None else sums - s["ref"].double()
    u = beta * (gain[:pairs] - gain[pairs:]) - s["margin"]
    if case["kind"] == "sigmoid":
        loss = -0.9 * torch.nn.functional.logsigmoid(u) - 0.1 * torch.nn.functional.logsigmoid(-u)
    elif case["kind"] == "hinge":
        loss = torch.relu(1.0 - u)
    else:
        loss = ((u - 0.5) / beta) ** 2
    w = s["weight"].double()
    loss = loss * w
    loss.sum().backward()
    loss, u, sums = loss.detach(), u.detach(), sums.detach()
    stats = torch.stack([loss.sum(), (u * w).sum(), ((u > 0) * w).sum(), w.sum()])
    return loss, sums, stats, _exact_backward(s, logp.grad, s["grad_scale"])
