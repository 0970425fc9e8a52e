"""Long sums of one sign: what the tensor cores' rounding toward zero leaves of a logit.

Products are positive and of about one size, so that a partial sum grows by an even share with each step: n steps in
a row are off by less than an ulp each, 2u of the partial sum (u = 2**-24), in all by (n + 1)u of the whole, and the
additions of m such sums to nearest by (m + 1) / 2 u.  dim is 1024, 16 blocks of 64: of up to 32 rows eight sums of 8
steps (9u + 4.5u), up to 64 rows four of 16 (17u + 2.5u), up to 128 two times two of 16 (the same), beyond two of 32
(33u + 1.5u).  lse is a mean of logits that are off by that, beside 1.2e-5 and its own rounding (2u).
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
@pytest.mark.parametrize("rows,steps", [(1, 13.5), (16, 13.5), (20, 13.5), (50, 19.5), (100, 19.5), (300, 34.5)])
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


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(262144, 300), (600, 200000)])
def test_gradients_of_one_sign(rows, vocab, dtype):
    """Sums over many rows (dw) and over a long vocabulary (dh) of terms of one sign: their mean error.

    The roundings of g and of the results, half a step each, have no sign: the mean of n of them is below 4 / sqrt(n) of
    that.  n is not the number of results, for many of them are alike and are rounded alike: dw along dim is a sum of
    rows of the same mean (262144 of them spread it by 0.29 / 512, 0.06%, less than a step of 0.1 to 0.8%), so n is 300
    at least, the tokens; dh along its rows is a mean of weights under nearly even probabilities, so n is dim.
    p is off by 3e-5, the rounding of lse (2**-24 of it) and 2e-7 of it (its mean error).  256 steps toward zero in
    a row, of partial sums that grow evenly, take (256 + 1) / 2 ulps of 2**-23 of a sum.
    """
    dim = 64
    g = torch.Generator(device=DEV)
    g.manual_seed(vocab)
    hidden = (0.5 + torch.rand((rows, dim), generator=g, device=DEV)).to(dtype)
    weight = (0.02 + 0.03 * torch.rand((vocab, dim), generator=g, device=DEV)).to(dtype)
    target = torch.randint(0, 10, (rows,), generator=g, device=DEV)
    dlse = torch.full((rows,), 0.75, device=DEV)
    dlogp = torch.zeros(rows, device=DEV)
    _, lse = itr.red_linear_logprob(hidden, weight, target)
    gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, dlse=dlse)
    want_h = torch.zeros((rows, dim), dtype=torch.float64, device=DEV)
    want_w = torch.zeros((vocab, dim), dtype=torch.float64, device=DEV)
    for part in torch.arange(rows, device=DEV).split(max(1, (1 << 26) // vocab)):
        h = hidden[part].double()
        p = torch.softmax(h @ weight.double().t(), 1) * 0.75
        want_h[part] = p @ weight.double()
        want_w += p.t() @ h
    half = torch.finfo(dtype).eps / 2
    for got, want, n in ((gh, want_h, dim), (gw, want_w, 300)):
        tol = 2 * 4 * half / n ** 0.5 + 3e-5 + float(lse.max()) * 3e-7 + 257 * U
        off = float((got.double() / want - 1).mean())
        print(off, tol)
        assert abs(off) <= tol, (off, tol)
