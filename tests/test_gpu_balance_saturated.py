"""Balance loss of sigmoids that are all but 1: the gradient's factor 1 - s, against 64 bits.

Tolerance (u = 2**-24): the slope p (1 - s) is two exponentials, a quotient and the row's sum: 3e-5 of it, and the
argument's rounding, |x| * 2u; the other factor, c - sum p c, is off by 3e-5 of both; each result is rounded once more.
"""
import pytest
import torch

import int_tensor_reductions_gb300 as itr
from gpu_util import lib_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-37}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("rows,experts,k", [(60, 16, 2), (900, 8, 2), (6000, 64, 4), (30000, 201, 8), (90, 1000, 8)])
def test_saturated_sigmoids(rows, experts, k, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows)
    x = torch.randn((rows, experts), generator=g, device=DEV) * 2
    x[:, ::3] += torch.rand((rows, 1), generator=g, device=DEV) * 40  # 0 to 40, some of each
    x[1] = 30.0
    x[2, 0] = 87.0
    x = x.to(dtype)
    ids = torch.topk(x.float(), k, 1).indices
    scale = 1024.0 * rows
    counts, prob, stats, grad = itr.red_balance(x, ids, coef=0.5, kind="sigmoid", grad_scale=scale)
    z = x.double()
    s = torch.sigmoid(z)
    p = s / s.sum(1, keepdim=True)
    slope = p * torch.sigmoid(-z)
    c = 0.5 * experts * counts.double() / (rows * k) / rows * scale
    d = (p * c).sum(1, keepdim=True)
    want = slope * (c - d)
    off = slope * ((3e-5 + z.abs() * 2.0 ** -23) * (c - d).abs() + 3e-5 * (c.abs() + d.abs()))
    tol = off + HALF[dtype] * (want.abs() + off) + TINY[dtype]
    bad = ~((grad.double() - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}: {grad[bad][0]} for {want[bad][0]}"
    assert bool(((prob.double() - p.mean(0)).abs() <= (3e-5 + (rows + 64) * 2.0 ** -24) * p.mean(0)).all())
