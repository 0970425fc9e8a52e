"""Gradients of red_linear_logprob where a CTA writes several tiles of them, against the 64-bit definition."""
import math

import pytest
import torch

import int_tensor_reductions_gb300 as itr
from gpu_util import lib_ready
from linear_reference import Reference
from test_gpu_linear import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


# rows of the weights that end off 16 bytes, in the first and in the second 64 of 128 columns
@pytest.mark.parametrize("rows,dim,vocab", [(64, 1030, 32001), (40, 2150, 20000), (9, 331, 60000), (3000, 331, 40000),
                                            (2500, 300, 40000)])
def test_ends_of_rows_in_many_tiles(rows, dim, vocab):
    hidden, weight, target, dlogp, _ = inputs(rows, dim, vocab, torch.bfloat16)
    ref = Reference(hidden, weight, target)
    _, lse = itr.red_linear_logprob(hidden, weight, target)
    gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
    ref.check_gradients(gh, gw, dlogp)
    for _ in range(5):
        again = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
        assert torch.equal(again[0], gh) and torch.equal(again[1], gw)


@pytest.mark.parametrize("rows", [1, 3, 16, 20, 64, 100, 128, 192, 250, 256, 300])
def test_weights_gradient_with_a_token_ruled_out(rows):
    """A token of weights -inf has probability 0 in every row, and a gradient of 0, whatever number of rows a tile holds."""
    hidden, weight, target, dlogp, dlse = inputs(rows, 64, 900, torch.bfloat16, 0.0)
    hidden[:, 7] = 1.0
    weight[5, 7] = -math.inf
    target[:] = target.where(target != 5, 6)
    _, lse = itr.red_linear_logprob(hidden, weight, target)
    _, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, dlse=dlse, grad_hidden=False)
    assert bool((gw[5] == 0).all())
    # without the token
    rest = torch.arange(900, device=DEV) != 5
    moved = target - (target > 5).long()
    ref = Reference(hidden, weight[rest], moved)
    _, clean = itr.red_linear_logprob(hidden, weight[rest], moved)
    ref.check_gradients(None, gw[rest], dlogp, dlse)
    assert float((lse - clean).abs().max()) <= 2.4e-5  # (the same logits, a softmax in fp32 each)


def test_pieces_of_many_rows():
    """Pieces of 4096 columns at most where g of them takes more than 256 MiB."""
    hidden, weight, target, dlogp, _ = inputs(70000, 16, 9000, torch.bfloat16)
    ref = Reference(hidden, weight, target)
    logp, lse = itr.red_linear_logprob(hidden, weight, target)
    ref.check_forward(logp, lse)
    ref.check_gradients(*itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp), dlogp)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [40, 300])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_coefficient_that_is_no_number(bad, rows, dtype):
    """An infinite dlogp is its row's matter: the others' hidden gradients are what they are without that row."""
    hidden, weight, target, dlogp, dlse = inputs(rows, 72, 3000, dtype, 0.0)
    dlogp, dlse = dlogp * 1e-5, dlse * 1e-5
    _, lse = itr.red_linear_logprob(hidden, weight, target)
    dlogp[1] = dlse[1] = 0.0
    want, _ = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, dlse=dlse)
    dlogp[1] = bad
    got, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, dlse=dlse)
    rest = torch.arange(rows, device=DEV) != 1
    assert torch.equal(got[rest], want[rest])
    assert not bool(got[1].isfinite().any()) and not bool(gw.isfinite().any())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,taken", [(1, 1), (2, 2), (5, 5), (8, 8), (9, 9), (13, 12), (16, 16), (16, 3), (20, 16), (40, 32),
                                        (64, 1), (64, 31), (128, 64), (100, 50), (128, 2)])
def test_gradients_of_few_rows(rows, taken, dtype):
    """Up to 16 rows, and up to half of the next power of two from 32 on: g is kept in two parts of 16 bits, and its
    rounding is not to be seen beside the results'.

    g is off by half = eps / 2 of what a first part leaves, half**2 of it, beside p's error (as in linear_reference, of
    p's share alone); sums and results as there.
    """
    half, u = torch.finfo(dtype).eps / 2, 2.0 ** -24
    for dim, vocab, scale in ((136, 3000, 1.0), (1040, 5001, 0.7), (2600, 729, 1.25)):
        hidden, weight, target, dlogp, dlse = inputs(rows, dim, vocab, dtype, 0.0, pad=8)
        target[torch.arange(rows, device=DEV) * taken % rows >= taken] = -100  # all but `taken` rows, spread out
        assert int((target >= 0).sum()) == taken
        dlogp[:] = dlogp.sign() * (1.0 + torch.arange(rows, device=DEV) * 0.37)
        ref = Reference(hidden, weight, target, scale)
        _, lse = itr.red_linear_logprob(hidden, weight, target, scale=scale)
        gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, dlse=dlse, scale=scale)
        ref.gradients(dlogp, dlse)
        by_p = ((dlse.double() - dlogp.double()).abs() * scale)[:, None] * ref.p
        dg = by_p * (2 * ref.dz + 3e-5 + 4 * u * ref.lse.abs())[:, None] + half * half * ref.g.abs() + 1e-9
        dg = torch.where(ref.live[:, None], dg, 0.0)
        for got, want, tol in ((gh, ref.g @ ref.w, dg @ ref.w.abs() + (ref.g.abs() @ ref.w.abs()) * (vocab / 16 + 16) * 2 * u),
                               (gw, ref.g.t() @ ref.h, dg.t() @ ref.h.abs() + (ref.g.abs().t() @ ref.h.abs()) * 50 * u)):
            off = (got.double() - want).abs()
            tol = tol + half * (want.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
            assert bool((off <= tol).all()), float((off - tol).max())


@pytest.mark.parametrize("rows", [5, 100])
def test_few_rows_of_a_long_vocabulary(rows):
    """dh of few rows in shares of more than 16384 columns: its sums move to fp32 registers on the way."""
    hidden, weight, target, dlogp, _ = inputs(rows, 4104, 70000, torch.float16, 0.0)
    ref = Reference(hidden, weight, target)
    _, lse = itr.red_linear_logprob(hidden, weight, target)
    gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
    ref.check_gradients(gh, gw, dlogp)
    again = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
    assert torch.equal(again[0], gh) and torch.equal(again[1], gw)
