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
