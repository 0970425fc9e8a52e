"""Long sums of one sign: what the tensor cores' rounding toward zero leaves of a logit.

Products are positive and of about one size, so that a partial sum grows by an even share with each step: n steps in
a row are off by less than an ulp each, 2u of the partial sum (u = 2**-24), in all by (n + 1)u of the whole, and the
additions of m such sums to nearest by (m + 1) / 2 u.  dim is 1024, 16 blocks of 64: of up to 32 rows eight sums of 8
steps (9u + 4.5u), up to 64 rows four of 16 (17u + 2.5u), up to 128 two times two of 16 (the same), beyond one of 64
(65u + u).  lse is a mean of logits that are off by that, beside 1.2e-5 and its own rounding (2u).
"""
import pytest
import torch

import int_tensor_reductions_gb300 as itr
from gpu_util import lib_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@pytest.mark.parametrize("size", [1.0, 1e4, 1e6])
@pytest.mark.parametrize("rows,steps", [(1, 13.5), (16, 13.5), (20, 13.5), (50, 19.5), (100, 19.5), (300, 66.0)])
@pytest.mark.parametrize("dim", [1000, 1024])
def test_logits_of_one_sign(dim, rows, steps, size):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows)
    hidden = ((0.9 + 0.2 * torch.rand((rows, dim), generator=g, device=DEV)) * size).bfloat16()
    weight = (0.7 + 0.2 * torch.rand((3001, dim), generator=g, device=DEV)).bfloat16()
    target = torch.randint(0, 3001, (rows,), generator=g, device=DEV)
    z = hidden.double() @ weight.double().t()
    _, lse = itr.red_linear_logprob(hidden, weight, target)
    want = torch.logsumexp(z, 1)
    off = (lse.double() - want).abs()
    tol = z.amax(1) * (steps + 2) * U + 1.2e-5
    assert bool((off <= tol).all()), (float((off / z.amax(1)).max()) / U, steps + 2)
