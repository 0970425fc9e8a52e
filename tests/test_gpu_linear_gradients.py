"""Gradients of red_linear_logprob where a CTA writes several tiles of them, against the 64-bit definition."""
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
