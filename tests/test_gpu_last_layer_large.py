"""Norms, balance loss and log-probabilities from hidden states over matrices of more than 2**31 elements: offsets
past 32 bits, by row strides and by rows."""
import math

import pytest
import torch

import int_tensor_reductions_gb300 as itr
from gpu_util import lib_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def far_apart(x):
    """x's rows 1.5 * 2**30 elements apart: the third starts past 2**31."""
    rows, cols = x.shape
    ld = 3 * 2 ** 29
    whole = torch.empty((rows - 1) * ld + cols, dtype=x.dtype, device=DEV)
    v = whole.as_strided((rows, cols), (ld, 1))
    v.copy_(x)
    return v


def test_rows_far_apart():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    for cols in (512, 1001):
        x, r, d = (torch.randn((4, cols), generator=g, device=DEV).bfloat16() for _ in range(3))
        y, total, rstd = itr.red_rmsnorm(x, residual=r)
        dx, _ = itr.red_rmsnorm_grad(d, total, rstd)
        q, scales, *_ = itr.red_rmsnorm_quant(x, residual=r, block=32)
        far = far_apart(x)
        out = far_apart(torch.zeros_like(x))
        got = itr.red_rmsnorm(far, residual=r, out=out)
        assert got[0] is out and torch.equal(out, y) and torch.equal(got[1], total) and torch.equal(got[2], rstd)
        got = itr.red_rmsnorm_quant(far, residual=r, block=32)
        assert torch.equal(got[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(got[1], scales)
        out.copy_(d)
        assert itr.red_rmsnorm_grad(out, total, rstd, grad=out)[0] is out and torch.equal(out, dx)
        ids = torch.topk(x.float(), 2, 1).indices
        want = itr.red_balance(x, ids)
        got = itr.red_balance(far, ids, grad=out)
        assert got[3] is out and all(torch.equal(a, b) for a, b in zip(got, want))


def test_many_rows():
    rows, cols = 300000, 8192
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    part = torch.randn((1000, cols), device=DEV).bfloat16()
    for i in range(0, rows, 1000):
        x[i:i + 1000] = part
    y, _, rstd = itr.red_rmsnorm(x)
    want = itr.red_rmsnorm(part)[0]
    for i in (0, 150000, rows - 1000):
        assert torch.equal(y[i:i + 1000], want)
    itr.red_rmsnorm_grad(y, x, rstd, grad=x)
    want = itr.red_rmsnorm_grad(want, part, rstd[:1000].contiguous())[0]
    for i in (0, 150000, rows - 1000):
        assert torch.equal(x[i:i + 1000], want)


@pytest.mark.parametrize("rows", [3, 200])
def test_vocabulary_past_2_to_the_31(rows):
    """600000 x 4096 weights.  Logits of 4096 products of magnitude 1/64 each are off by less than
    (96 + 8) * 2**-23 * 64 = 8e-4 (the tests of smaller sizes hold them to their own sizes); p by that and 3e-5;
    g and dw are rounded to bf16, 2**-8 each."""
    vocab, dim = 600000, 4096
    g = torch.Generator(device=DEV)
    g.manual_seed(rows)
    weight = torch.empty((vocab, dim), dtype=torch.bfloat16, device=DEV)
    for i in range(0, vocab, 100000):
        weight[i:i + 100000] = torch.randn((100000, dim), generator=g, device=DEV) / 64
    hidden = torch.randn((rows, dim), generator=g, device=DEV).bfloat16()
    target = torch.randint(vocab - 50000, vocab, (rows,), generator=g, device=DEV)
    target[0] = vocab - 1
    z = torch.cat([(hidden.double() @ weight[i:i + 100000].double().t()) for i in range(0, vocab, 100000)], 1)
    norm = torch.logsumexp(z, 1)
    logp, lse = itr.red_linear_logprob(hidden, weight, target)
    assert float((lse - norm).abs().max()) < 1e-3
    assert float((logp - (z.gather(1, target[:, None])[:, 0] - norm)).abs().max()) < 2e-3
    dlogp = torch.rand(rows, generator=g, device=DEV) + 0.5
    gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
    p = (z - norm[:, None]).exp() * -dlogp.double()[:, None]
    p[torch.arange(rows, device=DEV), target] += dlogp.double()
    for i in (0, vocab // 2, vocab - 2000):
        c = p[:, i:i + 2000]
        want = c.t() @ hidden.double()
        size = c.abs().t() @ hidden.double().abs()
        assert bool(((gw[i:i + 2000].double() - want).abs() <= size * (2.0 ** -8 + 2e-3) + want.abs() * 2.0 ** -8).all())
    want = sum(p[:, i:i + 100000] @ weight[i:i + 100000].double() for i in range(0, vocab, 100000))
    size = sum(p[:, i:i + 100000].abs() @ weight[i:i + 100000].double().abs() for i in range(0, vocab, 100000))
    assert bool(((gh.double() - want).abs() <= size * (2.0 ** -8 + 2e-3) + want.abs() * 2.0 ** -8).all())
    assert math.isfinite(float(gh.float().abs().max()))
