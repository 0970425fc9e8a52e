"""64-bit definitions of the losses over rows of logits, and the tolerances
of their fp32 kernels.

Tolerances, from the arithmetic (u = 2**-24):
  * an exponential's argument (x - m) * scale * log2(e) carries three
    roundings, so a term at distance d from the maximum is off by 3u*d
    relative, plus 2 ulp of the exponential itself; weighted by the terms, d
    averages at most ln(len) < 21;  sums add at most 64 roundings in a
    row per thread, and a tree.  The sum l is then off by less than
    (63 + 64 + 8)u = 8e-6 relative, ln l by 8e-6 absolute.
  * logp adds 3u |scale * (x_y - m)| <= 3u (|logp| + ln len) on top, lse one
    rounding.
  * a probability is off by 8e-6 + 4u*d relative: 3e-5 up to d = 88, beyond
    which it is below 1e-38.
  * gradients round once to the element type: half an ulp, or half the
    smallest subnormal.
"""
import math

import torch

LOGP_ABS, LOGP_REL = 8e-6 + 4e-6, 4e-7
PROB_REL = 3e-5
ROUND = {torch.float32: 2.0 ** -23, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-37}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def log_softmax(x, scale):
    """(log p, lse) in 64 bits on the host; rows of -inf: lse = log p = -inf."""
    z = x.detach().cpu().double() * scale
    top = z.max(1, keepdim=True).values
    ref = torch.where(torch.isinf(top) & (top < 0), torch.zeros_like(top), top)
    log_sum = (z - ref).exp().sum(1, keepdim=True).log()
    lse = ref + log_sum
    # from the maximum first: at the type's lowest value lse has no digits left for the log count
    logp = torch.where(torch.isinf(lse) & (lse < 0), torch.full_like(z, -math.inf), z - ref - log_sum)
    return logp, lse[:, 0]


def taken(logp, target):
    live = (target >= 0) & (target < logp.shape[1])
    at = torch.where(live, target, torch.zeros_like(target))
    return torch.where(live, logp.gather(1, at[:, None])[:, 0], torch.zeros(logp.shape[0], dtype=torch.float64)), live


def target_grad(logp, lse, target, live, c):
    """c * ([j == y] - p_j), zero for rows out of the loss or of -inf only."""
    g = -c[:, None] * logp.exp()
    rows = torch.arange(logp.shape[0])
    at = torch.where(live, target, torch.zeros_like(target))
    g[rows, at] += c
    live = live & (c != 0) & ~(torch.isinf(lse) & (lse < 0))
    return torch.where(live[:, None], g, torch.zeros_like(g))


def assert_logp(got, want, what=""):
    got, want = got.cpu().double(), want.cpu().double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~same & ~((got - want).abs() <= LOGP_ABS + LOGP_REL * want.abs())
    assert not bad.any(), f"{what}: {int(bad.sum())} off, first {got[bad][0]} for {want[bad][0]}"


def assert_grad(got, want, p, c, target=None, extra=0.0, what=""):
    """``c``: per row, the size of the terms of the coefficient; ``extra``:
    relative error of the coefficient itself."""
    dt = got.dtype
    got, want = got.detach().cpu().double(), want.cpu().double()
    c = c.abs()[:, None]
    # rows that take no part may hold NaN: nothing but zeros is right there
    tol = c * p.nan_to_num(nan=0.0) * (PROB_REL + extra) + ROUND[dt] * want.abs() + TINY[dt]
    if target is not None:
        rows = torch.arange(got.shape[0])
        at = target.clamp(0, got.shape[1] - 1)
        tol[rows, at] += c[:, 0] * (1e-6 + extra)
    bad = ~((got - want).abs() <= tol) & ~(got.isnan() & want.isnan())
    assert not bad.any(), (f"{what}: {int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {tol[bad][0]}")


def policy(logp, old, ref, adv, w, low, high, kl):
    """(loss, dlogp, drift, clipped) per token in 64 bits, before any mask."""
    ratio = (logp - old).exp()
    a, b = ratio * adv, ratio.clamp(1.0 - low, 1.0 + high) * adv
    clipped = a > b
    loss, c = -torch.where(clipped, b, a), torch.where(clipped, torch.zeros_like(a), -a)
    drift = torch.zeros_like(a)
    if kl:
        d = ref - logp
        drift = torch.expm1(d) - d
        loss, c = loss + kl * drift, c - kl * torch.expm1(d)
    return loss * w, c * w, drift, clipped


def pair_loss(u, kind, beta, eps):
    if kind == "sigmoid":
        loss = -(1 - eps) * torch.nn.functional.logsigmoid(u) - eps * torch.nn.functional.logsigmoid(-u)
        return loss, eps - torch.sigmoid(-u)
    if kind == "hinge":
        return torch.relu(1 - u), -(u < 1).double()
    off = (u - 0.5) / beta
    return off * off, 2 * off / beta
