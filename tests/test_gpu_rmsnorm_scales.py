"""Scales of red_rmsnorm_quant near fp32's smallest numbers."""
import pytest
import torch

import int_tensor_reductions_gb300 as itr
from gpu_util import lib_ready
from test_gpu_rmsnorm import definition, near, randn

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
LEAST = 2.0 ** -149  # a step of fp32 below 2^-126


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("length,block,pad", [(384, 32, 0), (1000, 64, 3), (5120, 128, 0), (200, 0, 0)])
def test_small_scales(length, block, pad, dtype, kind):
    """y down to 1e-45: scales end at 2^-126, and q is y / scale all the same (y is off by a step of fp32 at most)."""
    top = 448.0 if kind == "e4m3" else 127.0
    x = randn(7, length, dtype, 1, pad)
    width = block or length
    power = torch.linspace(-28, -44, -(-length // width), device=DEV, dtype=torch.float64) if block else \
        torch.full((1,), -39.0, device=DEV, dtype=torch.float64)
    w = (10.0 ** power).repeat_interleave(width)[:length].float()
    q, scales, _, _ = itr.red_rmsnorm_quant(x, w, eps=1e-6, kind=kind, block=block)
    _, _, want = definition(x, w, None, float(torch.tensor(1e-6)))
    amax = torch.nn.functional.pad(want, (0, -length % width)).view(7, -1, width).abs().amax(2)
    exact = (amax / top).clamp(min=2.0 ** -126)
    near(scales, exact, 32 * U * exact, "scales")
    wide = scales.double().repeat_interleave(width, 1)[:, :length]
    value = want / wide
    step = 2.0 ** -4 * value.abs() + 2.0 ** -10 if kind == "e4m3" else torch.full_like(value, 0.5)
    near(q.float(), value, step + 36 * U * value.abs() + LEAST / wide, "q")
    assert float(q.float().abs().max()) <= top
