"""Losses over rows of logits where they are easily wrong: many rows without a
gradient, logits far from zero, waits that run out, NaN and infinities in each
input, memory of other streams."""
import math

import pytest
import torch

import int_tensor_reductions_gb300 as itr
import loss_reference as ref
from gpu_util import lib_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def device_gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def distill_loss(x, ids, vals):
    """(loss, size of its terms) per row in 64 bits, q = softmax(vals), no scale."""
    logp = torch.log_softmax(x.double(), 1).gather(1, ids)
    logq = torch.log_softmax(vals.double(), 1)
    q = logq.exp()
    return (q * (logq - logp)).sum(1), (q * (logq.abs() + logp.abs() + 30)).sum(1)


# Several rows per CTA, of one batch of the kernel's ring to many: each row's
# loss from its own statistics, though the next rows' are formed meanwhile.
@pytest.mark.parametrize("dtype,length,rows", [(torch.float32, 2100, 6000), (torch.float32, 5000, 4000),
                                               (torch.bfloat16, 13001, 3000), (torch.float16, 30000, 1500),
                                               (torch.float32, 40000, 800)])
def test_distill_loss_alone_over_many_rows(dtype, length, rows):
    g = device_gen(length)
    width = torch.rand((rows, 1), generator=g, device=DEV) * 4 + 0.1    # rows of very different statistics
    x = (torch.randn((rows, length), generator=g, device=DEV) * width).to(dtype)
    ids = torch.randint(0, length, (rows, 5), generator=g, device=DEV)
    vals = torch.randn((rows, 5), generator=g, device=DEV)
    loss, stats, grad = itr.red_distill(x, ids, vals, grad=False)
    assert grad is None and stats[1].item() == rows
    for part in torch.arange(rows, device=DEV).split(200):
        want, size = distill_loss(x[part], ids[part], vals[part])
        assert bool(((loss[part].double() - want).abs() <= 4e-5 * size + 1e-9).all())


def log_softmax(x, scale=1.0):
    """ref.log_softmax, computed on the device: (log p, lse) on the host."""
    z = x.double() * scale
    top = z.max(1, keepdim=True).values
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    norm = (z - base).exp().sum(1, keepdim=True).log()
    logp = torch.where(top == -math.inf, torch.full_like(z, -math.inf), z - base - norm)
    return logp.cpu(), (base + norm)[:, 0].cpu()


# Rows by groups of lanes, by two warps, by clusters and by the row kernel's
# CTAs.  1.163e7 is where s2 * x passes 2^24: maxima on both sides of it.
ROWS = [(5, 900), (300, 3500), (6, 9001), (6, 40000), (300, 9001), (300, 30000)]
FARAWAY = [(torch.float32, 1e3, 1.0), (torch.float32, -1e4, 0.7), (torch.float32, 1e6, 1.0), (torch.float32, 1.163e7, 1.0),
           (torch.float32, -1.163e7, 1.0), (torch.float32, 300.0, 30.0), (torch.float16, 1e4, 1.0),
           (torch.float16, 300.0, 30.0), (torch.bfloat16, -1e4, 1.25), (torch.bfloat16, 300.0, 30.0)]


@pytest.mark.parametrize("rows,length", ROWS)
@pytest.mark.parametrize("dtype,offset,scale", FARAWAY)
def test_logits_far_from_zero(rows, length, dtype, offset, scale):
    """A constant added to a row changes no probability: what a row's parts of
    different maxima add up to is as near as at zero."""
    g = device_gen(length + rows)
    width = 3.0 / scale if scale > 1 else 3.0
    x = (torch.randn((rows, length), generator=g, device=DEV) * width + offset).to(dtype)
    t = torch.randint(0, length, (rows,), generator=g, device=DEV)
    lp, lse = log_softmax(x, scale)
    want, live = ref.taken(lp, t.cpu())
    p = lp.exp()
    got, norm = itr.red_logprob(x, t, scale=scale)
    ref.assert_logp(got, want, "logp")
    ref.assert_logp(norm, lse, "lse")
    old = want.float().to(DEV)
    down = torch.full((rows,), -1.0, device=DEV)
    _, got, _, grad = itr.red_policy(x, t, old, down, scale=scale)
    ref.assert_logp(got, want, "policy")
    # the ratio is 1 up to the rounding of old and the error of logp
    c = torch.full((rows,), scale, dtype=torch.float64)
    extra = 3e-5 + 2.0 ** -23 * float(want.abs().max())
    ref.assert_grad(grad, ref.target_grad(lp, lse, t.cpu(), live, c), p, c, t.cpu(), extra=extra, what="policy")
    ids = torch.randint(0, length, (rows, 3), generator=g, device=DEV)
    vals = torch.zeros((rows, 3), device=DEV)
    loss, _, grad = itr.red_distill(x, ids, vals, scale=scale)
    at = lp.gather(1, ids.cpu())
    size = math.log(3.0) + at.abs().mean(1)
    assert bool(((loss.cpu().double() - (-math.log(3.0) - at.mean(1))).abs() <= 1.2e-5 + 1e-6 * size).all())
    mass = torch.zeros_like(p).scatter_add_(1, ids.cpu(), torch.full((rows, 3), 1 / 3, dtype=torch.float64))
    ref.assert_grad(grad, (p - mass) * scale, p + mass, c, extra=3e-5, what="distill")
