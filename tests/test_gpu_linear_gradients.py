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
