"""Root-mean-square norm, its 8-bit output and its backward against 64-bit
definitions.

Tolerances (u = 2**-24; v = half an eps of the type): a sum of squares is up to 32
multiply-adds in a row per thread and a tree of at most 10 additions, so it is off by
less than 43u, relative, beside 2u of each square; rstd by half of that and a
rounding: 25u.  y = t * rstd * weight adds a rounding of t and two products: 30u,
then v.  mean(g * h) is off by 60u of the mean of its terms' magnitudes.  A sum over
rows is off by at most (rows + 64)u of its terms' magnitudes, in any order.
"""
import math

import pytest
import torch

import int_tensor_reductions_gb300 as itr
from gpu_util import lib_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-44, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-40}
GUARD = 7.25


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def matrix(rows, cols, dtype, pad=0, shift=0, fill=GUARD):
    buf = torch.full((shift + rows * (cols + pad),), fill, device=DEV).to(dtype)
    return buf[shift:].view(rows, cols + pad)[:, :cols]


def guard_intact(t, fill=GUARD):
    whole = t.as_strided((t.shape[0], t.stride(0)), t.stride(), t.storage_offset())
    assert bool((whole[:, t.shape[1]:].float() == fill).all()), "write behind the rows"


def randn(rows, cols, dtype, seed, pad=0, shift=0, width=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    m = matrix(rows, cols, dtype, pad, shift, math.nan)
    m.copy_(torch.randn((rows, cols), generator=g, device=DEV) * width)
    return m


def near(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}: {got[bad][0]} for "
                           f"{want[bad][0]} +- {tol.expand_as(want)[bad][0]}")


def definition(x, weight, residual, eps):
    t = x.double() if residual is None else x.double() + residual.double()
    rstd = (t.square().mean(1) + eps).rsqrt()
    w = 1.0 if weight is None else weight.double()
    return t, rstd, t * rstd[:, None] * w


LENGTHS = [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 200, 256, 257, 512, 515, 1000, 1024, 1032, 2048, 2049, 4095, 4096, 5120,
           8192, 8200, 16384]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("length", LENGTHS)
def test_norm(length, dtype):
    for rows, pad, shift, with_residual, wtype in ((1, 0, 0, True, dtype), (37, 8, 0, False, torch.float32),
                                                   (5, 3, 1, True, torch.float32), (300, 0, 0, True, None)):
        x = randn(rows, length, dtype, length, pad, shift)
        res = randn(rows, length, dtype, length + 1, 2 * pad, shift, 2.0) if with_residual else None
        w = None if wtype is None else (randn(1, length, torch.float32, 3)[0] + 1.0).to(wtype)
        out = matrix(rows, length, dtype, pad, shift)
        y, total, rstd = itr.red_rmsnorm(x, w, residual=res, eps=1e-5, out=out)
        assert y is out
        guard_intact(out)
        t, want_rstd, want = definition(x, w, res, float(torch.tensor(1e-5)))
        near(rstd, want_rstd, 26 * U * want_rstd, "rstd")
        near(y, want, 30 * U * want.abs() + HALF[dtype] * want.abs() * (1 + 30 * U) + TINY[dtype], "y")
        if with_residual:
            near(total, t, (HALF[dtype] + 2 * U) * t.abs() + TINY[dtype], "total")
        else:
            assert total is None


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("length", [1, 7, 33, 64, 100, 127, 128, 257, 640, 1000, 2056, 4096, 5000, 8192, 16384])
def test_quantised(length, dtype, kind):
    top = 448.0 if kind == "e4m3" else 127.0
    for rows, pad, shift, block in ((1, 0, 0, 0), (37, 0, 0, 128), (5, 3, 1, 64), (70, 8, 0, 32), (3, 8, 0, 128)):
        x = randn(rows, length, dtype, length, pad, shift)
        res = randn(rows, length, dtype, length + 1, pad, shift, 2.0)
        if rows == 70:
            x[3] = 0.0
            res[3] = 0.0
        w = randn(1, length, torch.float32, 3)[0] + 1.0
        q, scales, total, rstd = itr.red_rmsnorm_quant(x, w, residual=res, eps=1e-6, kind=kind, block=block)
        assert q.dtype == (torch.float8_e4m3fn if kind == "e4m3" else torch.int8)
        t, want_rstd, want = definition(x, w, res, float(torch.tensor(1e-6)))
        near(rstd, want_rstd, 26 * U * want_rstd, "rstd")
        near(total, t, (HALF[dtype] + 2 * U) * t.abs() + TINY[dtype], "total")
        width = block or length
        parts = torch.nn.functional.pad(want, (0, -length % width)).view(rows, -1, width)
        amax = parts.abs().amax(2)
        want_scale = torch.where(amax == 0, 1.0, amax / top)
        assert scales.shape == want_scale.shape
        near(scales, want_scale, 32 * U * want_scale, "scales")
        # against the scale that came back: a step of the type, and the error of y in it
        value = want / scales.double().repeat_interleave(width, 1)[:, :length]
        step = 2.0 ** -4 * value.abs() + 2.0 ** -10 if kind == "e4m3" else torch.full_like(value, 0.5)
        near(q.float(), value, step + 36 * U * value.abs(), "q")
        assert float(q.float().abs().max()) <= top
        if rows == 70:
            assert bool((scales[3] == 1).all() and (q[3].float() == 0).all())


def test_ties_to_even():
    """Values on the border of two: rows of a single magnitude, whose norm is 1."""
    x = torch.ones((1, 64), device=DEV)
    w = torch.arange(64, device=DEV) + 0.5
    w[63] = 127.0
    q, scales, _, _ = itr.red_rmsnorm_quant(x, w, eps=0.0, kind="int8")
    assert float(scales) == 1.0
    assert q[0, :63].tolist() == [int(v) for v in torch.round(w[:63]).tolist()]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("length", LENGTHS)
def test_gradient(length, dtype):
    for rows, pad, shift, with_total, wtype in ((1, 0, 0, True, dtype), (37, 8, 0, False, torch.float32),
                                                (5, 3, 1, True, torch.float32), (1500, 0, 0, True, None)):
        if rows * length > 1 << 23:
            rows = 400
        x = randn(rows, length, dtype, length, pad, shift)
        dy = randn(rows, length, dtype, length + 1, 2 * pad, shift)
        dt = randn(rows, length, dtype, length + 2, pad, shift) if with_total else None
        w = None if wtype is None else (randn(1, length, torch.float32, 3)[0] + 1.0).to(wtype)
        rstd = (x.double().square().mean(1) + 1e-6).rsqrt().float()
        out = matrix(rows, length, dtype, pad, shift)
        dx, dw = itr.red_rmsnorm_grad(dy, x, rstd, w, dtotal=dt, grad=out)
        assert dx is out
        guard_intact(out)
        r = rstd.double()[:, None]
        h = x.double() * r
        g = dy.double() * (1.0 if w is None else w.double())
        c = (g * h).mean(1, keepdim=True)
        want = r * (g - h * c)
        tol = r * (4 * U * (g.abs() + h.abs() * c.abs()) + h.abs() * 64 * U * (g * h).abs().mean(1, keepdim=True))
        if dt is not None:
            want = want + dt.double()
        tol = tol + 2 * U * want.abs()
        near(dx, want, tol + HALF[dtype] * (want.abs() + tol) + TINY[dtype], "dx")
        if w is None:
            assert dw is None
            continue
        terms = dy.double() * h
        tol = terms.abs().sum(0) * (rows + 64) * U
        assert dw.dtype == w.dtype
        near(dw, terms.sum(0), tol + HALF[w.dtype] * (terms.sum(0).abs() + tol) + TINY[w.dtype], "dw")


def test_gradient_by_differences():
    """The forward on both sides, in fp32: its rounding is 1e-6 of the values, a step 1e-2."""
    x = randn(6, 96, torch.float32, 1)
    w = randn(1, 96, torch.float32, 2)[0]
    dy = randn(6, 96, torch.float32, 3)
    y, _, rstd = itr.red_rmsnorm(x, w)
    dx, dw = itr.red_rmsnorm_grad(dy, x, rstd, w)
    u, uw = randn(6, 96, torch.float32, 4), randn(1, 96, torch.float32, 5)[0]
    h = 1e-2

    def loss(x, w):
        return float((itr.red_rmsnorm(x, w)[0].double() * dy.double()).sum())

    size = float((y.abs() * dy.abs()).sum())
    for a, b, slope in ((loss(x + h * u, w), loss(x - h * u, w), float((dx.double() * u).sum())),
                        (loss(x, w + h * uw), loss(x, w - h * uw), float((dw.double() * uw).sum()))):
        # third order in h: the norm's third derivative is below 20 |u|^3 / |x|^3 of its values
        assert abs((a - b) / (2 * h) - slope) <= size * (20 * h * h + 2e-6 / h)


@pytest.mark.parametrize("length", [100, 1024, 5000])
def test_in_place(length):
    dtype = torch.bfloat16
    x, res = randn(20, length, dtype, 1), randn(20, length, dtype, 2)
    w = randn(1, length, dtype, 3)[0]
    y, total, rstd = itr.red_rmsnorm(x, w, residual=res)
    for y_over, total_over in (("x", "res"), ("res", "x"), (None, "res"), ("x", None)):
        t = dict(x=x.clone(), res=res.clone())
        got = itr.red_rmsnorm(t["x"], w, residual=t["res"], out=t.get(y_over), total=t.get(total_over))
        assert torch.equal(got[0], y) and torch.equal(got[1], total) and torch.equal(got[2], rstd)
    one = x.clone()
    want = itr.red_rmsnorm(x, w)[0]
    assert itr.red_rmsnorm(one, w, out=one)[0] is one and torch.equal(one, want)
    q = itr.red_rmsnorm_quant(x, w, residual=res)[0]
    t = res.clone()
    got = itr.red_rmsnorm_quant(x, w, residual=t, total=t)
    assert torch.equal(got[0].view(torch.int8), q.view(torch.int8)) and torch.equal(t, total)
    dy, dt = randn(20, length, dtype, 4), randn(20, length, dtype, 5)
    dx, dw = itr.red_rmsnorm_grad(dy, total, rstd, w, dtotal=dt)
    for over in range(3):
        t = [dy.clone(), total.clone(), dt.clone()]
        got = itr.red_rmsnorm_grad(t[0], t[1], rstd, w, dtotal=t[2], grad=t[over])
        assert got[0] is t[over] and torch.equal(got[0], dx) and torch.equal(got[1], dw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("length", [64, 1000, 4096])
def test_nan_and_infinity_stay_in_their_row(length, dtype):
    x = randn(9, length, dtype, 1)
    w = torch.ones(length, device=DEV)
    clean = itr.red_rmsnorm(x, w)[0]
    x[2, 5] = math.nan
    x[4, length - 1] = math.inf
    x[6] = 0.0
    y, _, rstd = itr.red_rmsnorm(x, w)
    keep = torch.tensor([0, 1, 3, 5, 7, 8], device=DEV)
    assert torch.equal(y[keep], clean[keep])
    assert bool(y[2].isnan().all() and y[4, length - 1].isnan() and (y[4, :length - 1] == 0).all() and (y[6] == 0).all())
    q, scales, _, _ = itr.red_rmsnorm_quant(x, w, block=32)
    assert bool(scales[2].isnan().all() and q[2].float().isnan().all() and not scales[keep].isnan().any())
    spoilt = w.clone()
    spoilt[3] = math.nan  # one column: its block of each row
    q, scales, _, _ = itr.red_rmsnorm_quant(x[:2], spoilt, block=32)
    assert bool(scales[:, 0].isnan().all() and not scales[:, 1:].isnan().any() and q[:, :32].float().isnan().all())
    assert bool(q[:, 32:].float().isfinite().all())
    dy = randn(9, length, dtype, 2)
    good = torch.where(rstd.isfinite() & (rstd > 0), rstd, 1.0)
    want = itr.red_rmsnorm_grad(dy, torch.where(x.isfinite(), x, 0.0), good, w)[0]
    dx, dw = itr.red_rmsnorm_grad(dy, x, rstd, w)
    assert torch.equal(dx[keep], want[keep]) and bool(dx[2].isnan().all())
    assert bool(dw.isnan().any())


def test_nothing_and_one():
    w = torch.ones(64, device=DEV)
    x = torch.empty((0, 64), device=DEV)
    y, total, rstd = itr.red_rmsnorm(x, w, residual=x)
    assert y.shape == total.shape == (0, 64) and rstd.numel() == 0
    q, scales, _, _ = itr.red_rmsnorm_quant(x, w, block=32)
    assert q.shape == (0, 64) and scales.shape == (0, 2)
    dx, dw = itr.red_rmsnorm_grad(x, x, rstd, w)
    assert dx.shape == (0, 64) and bool((dw == 0).all())
    got = itr.red_rmsnorm_grad(randn(3, 64, torch.float32, 1), randn(3, 64, torch.float32, 2), torch.ones(3, device=DEV), w,
                               grad_weight=False)
    assert got[1] is None


def test_repeatable_streams_and_graphs():
    x, res, dy = (randn(3000, 640, torch.bfloat16, i) for i in range(3))
    w = randn(1, 640, torch.float32, 5)[0]

    def step():
        y, total, rstd = itr.red_rmsnorm(x, w, residual=res)
        q, scales, _, _ = itr.red_rmsnorm_quant(x, w, residual=res, block=128)
        dx, dw = itr.red_rmsnorm_grad(dy, total, rstd, w, dtotal=dy)
        return y, total, rstd, q.view(torch.int8), scales, dx, dw

    want = step()
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
    stream = torch.cuda.Stream()
    y, total, _ = itr.red_rmsnorm(x, w, residual=res, stream=stream)
    stream.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(total, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for shift in (0.0, 1.0):
        x.add_(shift)
        graph.replay()
        torch.cuda.synchronize()
        fresh = step()
        assert all(torch.equal(a, b) for a, b in zip(got, fresh))


def test_refusals():
    x = randn(4, 64, torch.bfloat16, 1)
    w = torch.ones(64, device=DEV)
    rstd = torch.ones(4, device=DEV)
    for call in (lambda: itr.red_rmsnorm(x.int(), w), lambda: itr.red_rmsnorm(x, w[:63]),
                 lambda: itr.red_rmsnorm(x, w, residual=x.float()), lambda: itr.red_rmsnorm(x, w, total=x),
                 lambda: itr.red_rmsnorm(x.t(), w), lambda: itr.red_rmsnorm(x, w, out=x[:3]),
                 lambda: itr.red_rmsnorm_quant(x, w, kind="e5m2"), lambda: itr.red_rmsnorm_quant(x, w, out=x),
                 lambda: itr.red_rmsnorm_grad(x, x, rstd[:3], w), lambda: itr.red_rmsnorm_grad(x.float(), x, rstd, w),
                 lambda: itr.red_rmsnorm_grad(x, x, rstd, w, grad_weight=w.half())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: itr.red_rmsnorm(x, w.half()), lambda: itr.red_rmsnorm(x, w, eps=-1.0),
                 lambda: itr.red_rmsnorm(torch.empty((2, 16385), device=DEV)),
                 lambda: itr.red_rmsnorm_quant(x, w, block=48), lambda: itr.red_rmsnorm_quant(x, w, block=-32)):
        with pytest.raises(itr.RedError):
            call()
