"""Norms and their gradients over their inputs, rows off the 16-byte blocks."""
import pytest
import torch

import int_tensor_reductions_gb300 as itr
from gpu_util import lib_ready
from test_gpu_rmsnorm import randn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("length,pad,shift", [(100, 3, 1), (4095, 2, 3), (8200, 1, 1), (12001, 0, 1), (16383, 0, 3), (16384, 0, 0)])
def test_in_place_off_the_blocks(length, pad, shift, dtype):
    """The longest rows of 32 bits do not fit the ring and are read twice; results over each input, bit for bit."""
    rows = 700
    x, res, dy, dt = (randn(rows, length, dtype, i, pad, shift) for i in range(4))
    w = randn(1, length, torch.float32, 5)[0] + 1.0

    def over(t):
        buf = torch.empty(shift + rows * (length + pad), dtype=dtype, device=DEV)
        v = buf[shift:].view(rows, length + pad)[:, :length]
        v.copy_(t)
        return v

    y, total, rstd = itr.red_rmsnorm(x, w, residual=res)
    for y_over, total_over in (("x", "res"), ("res", "x")):
        t = dict(x=over(x), res=over(res))
        got = itr.red_rmsnorm(t["x"], w, residual=t["res"], out=t[y_over], total=t[total_over])
        assert torch.equal(got[0], y) and torch.equal(got[1], total) and torch.equal(got[2], rstd)
    dx, dw = itr.red_rmsnorm_grad(dy, total, rstd, w, dtotal=dt)
    for which in range(3):
        t = [over(dy), over(total), over(dt)]
        got = itr.red_rmsnorm_grad(t[0], t[1], rstd, w, dtotal=t[2], grad=t[which])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
