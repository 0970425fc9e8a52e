"""Balance loss of a router against its 64-bit definition.

Tolerances (u = 2**-24): a probability is off by 3e-5 relative (its exponential's
argument carries three roundings, the sum 64 additions and a tree); a mean over
tokens by that and (tokens + 64)u; lse by 1.2e-5 + 4e-7 of itself.  A gradient is
p * (c - sum p c): off by 1e-4 of p times the size of the two, with its coefficients'
few roundings, and v, half an eps of the type.
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


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def inputs(rows, experts, k, dtype, out=0.2, pad=0, shift=0, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows + 31 * experts + k + seed)
    buf = torch.full((shift + rows * (experts + pad),), math.nan, dtype=dtype, device=DEV)
    x = buf[shift:].view(rows, experts + pad)[:, :experts]
    x.copy_(torch.randn((rows, experts), generator=g, device=DEV) * 2 + torch.randn(experts, generator=g, device=DEV))
    ids = torch.topk(x.float(), k, 1).indices
    live = torch.rand(rows, generator=g, device=DEV) >= out
    return x, ids, live


def check(x, ids, live, got, kind, coef, z_coef, gs):
    rows, experts = x.shape
    k = ids.shape[1]
    counts, prob, stats, grad = got
    keep = torch.ones(rows, dtype=torch.bool, device=DEV) if live is None else live.bool()
    z = torch.where(keep[:, None], x.double(), 0.0)
    empty = torch.isinf(z).all(1) & (z < 0).all(1)
    n = int(keep.sum())
    named = ids[keep]
    named = named[(named >= 0) & (named < experts)]
    want_counts = torch.bincount(named.flatten(), minlength=experts)
    assert counts.dtype == torch.int64 and torch.equal(counts, want_counts)
    if kind == "softmax":
        lse = torch.where(empty, 0.0, torch.logsumexp(z, 1))
        # from the maximum: a row of the type's lowest value leaves no digits for its lse's logarithm
        p = torch.where(empty[:, None], 0.0, torch.softmax(z, 1))
        slope = p
    else:
        lse = torch.zeros(rows, dtype=torch.float64, device=DEV)
        s = torch.sigmoid(z)
        p = torch.where(empty[:, None], 0.0, s / s.sum(1, keepdim=True).clamp(min=1e-300))
        slope = p * torch.sigmoid(-z)
    p, slope = (torch.where(keep[:, None], v, 0.0) for v in (p, slope))
    lse = torch.where(keep, lse, 0.0)
    m = max(1, n)
    rel = 3e-5 + (rows + 64) * U
    want_prob = p.sum(0) / m
    assert bool(((prob.double() - want_prob).abs() <= rel * want_prob + 1e-37).all())
    share = want_counts.double() / (m * k)
    balance = experts * float((share * want_prob).sum())
    zz = float(lse.square().sum()) / m
    dz = float((2 * lse.abs() * (1.2e-5 + 4e-7 * lse.abs())).sum()) / m + (rows + 64) * U * zz
    want = [coef * balance + z_coef * zz, balance, zz, float(n)]
    tol = [abs(coef) * balance * 2 * rel + abs(z_coef) * dz + 1e-6 * (abs(coef) * balance + abs(z_coef) * zz),
           balance * 2 * rel, dz + 1e-6 * zz, 0.0]
    if want[2] > torch.finfo(torch.float32).max:  # beyond fp32: infinity is its rounding
        assert float(stats[2]) == math.inf
        want[2] = tol[2] = 0.0
        stats = stats.clone()
        stats[2] = 0.0
    for i in range(4):
        assert abs(float(stats[i]) - want[i]) <= tol[i], (i, float(stats[i]), want[i], tol[i])
    if grad is None:
        return
    c = coef * experts * share / m
    d = (p * c).sum(1, keepdim=True)
    g = slope * (c - d) + (2 * z_coef / m) * lse[:, None] * p
    off = p * 1e-4 * (c.abs() + d.abs()) + 2 * abs(z_coef) / m * p * (1.2e-5 + 4e-5 * lse.abs()[:, None])
    tol = abs(gs) * off + HALF[x.dtype] * abs(gs) * (g.abs() + off) + TINY[x.dtype]
    tol = torch.where(keep[:, None], tol, 0.0)
    bad = ~((grad.double() - gs * g).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}: {grad[bad][0]} for {(gs * g)[bad][0]}"


SHAPES = [(1, 1, 1), (1, 8, 2), (5, 3, 2), (9, 64, 6), (257, 64, 6), (300, 60, 4), (1000, 100, 1), (5000, 16, 2),
          (4099, 128, 8), (2000, 256, 8), (700, 300, 5), (300, 512, 8), (200, 1000, 3), (70, 1500, 16), (40, 4096, 10)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,experts,k", SHAPES)
def test_balance(rows, experts, k, dtype):
    for pad, shift, kind, z_coef, gs in ((0, 0, "softmax", 1e-2, 1.0), (8, 0, "sigmoid", 0.0, 64.0),
                                         (3, 1, "softmax", 0.0, 1024.0)):
        x, ids, live = inputs(rows, experts, k, dtype, 0.2 if pad else 0.0, pad, shift)
        live = live if pad else None
        got = itr.red_balance(x, ids, live=live, coef=0.5, z_coef=z_coef, kind=kind, grad_scale=gs)
        assert got[3].dtype == dtype and got[3].shape == x.shape
        check(x, ids, live, got, kind, 0.5, z_coef, gs)
        again = itr.red_balance(x, ids, live=live, coef=0.5, z_coef=z_coef, kind=kind, grad_scale=gs, grad=False)
        assert again[3] is None and all(torch.equal(a, b) for a, b in zip(again[:3], got[:3]))


@pytest.mark.parametrize("rows,experts", [(60, 16), (6000, 64), (90, 1000)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_masks_and_odd_ids(rows, experts, kind):
    """Tokens that are out hold NaN; experts ruled out by -inf, in one token all of them; ids outside, and twice."""
    for dtype in DTYPES:
        x, ids, live = inputs(rows, experts, 4, dtype)
        live[:6] = True
        x[0, ::2] = -math.inf
        x[1] = -math.inf
        x[2, 1:] = -math.inf
        x[3] = torch.finfo(dtype).min
        ids[4] = ids[4, 0]
        ids[5, 1:] = torch.tensor([-1, experts, 2 ** 40], device=DEV)
        x[~live] = math.nan
        for mask in (live, live.to(torch.uint8) * 3):
            got = itr.red_balance(x, ids, live=mask, coef=0.1, z_coef=0.0, kind=kind)
            check(x, ids, live, got, kind, 0.1, 0.0, 1.0)
        assert bool((got[3][1] == 0).all())


@pytest.mark.parametrize("rows,experts", [(60, 16), (900, 8), (6000, 64), (90, 1000)])
def test_sigmoids_near_zero(rows, experts):
    """Tokens whose sigmoids are below fp32's smallest have probabilities all the same."""
    for dtype in DTYPES:
        x, ids, live = inputs(rows, experts, 4, dtype)
        x[::3] -= 100.0
        x[1::7] -= 60.0
        x[5, 1:] = torch.finfo(dtype).min
        x[8] -= 600.0
        got = itr.red_balance(x, ids, live=live, coef=0.1, kind="sigmoid")
        check(x, ids, live, got, "sigmoid", 0.1, 0.0, 1.0)


def test_results_of_rows_out_of_a_larger_tensor():
    """Results do not take the row stride of what x was cut from."""
    whole = torch.randn((20, 50, 64), device=DEV)
    x = whole[:, -1]
    ids = torch.topk(x, 2, 1).indices
    grad = itr.red_balance(x, ids)[3]
    assert grad.stride(0) == 64 and torch.equal(grad, itr.red_balance(x.contiguous(), ids)[3])
    y, _, rstd = itr.red_rmsnorm(x)
    assert y.stride(0) == 64 and torch.equal(y, itr.red_rmsnorm(x.contiguous())[0])
    dx, _ = itr.red_rmsnorm_grad(y, x, rstd)
    assert dx.stride(0) == 64 and torch.equal(dx, itr.red_rmsnorm_grad(y, x.contiguous(), rstd)[0])


@pytest.mark.parametrize("rows,experts", [(60, 16), (6000, 64)])
def test_nobody_takes_part(rows, experts):
    x, ids, live = inputs(rows, experts, 2, torch.float32)
    x[:] = math.nan
    counts, prob, stats, grad = itr.red_balance(x, ids, live=torch.zeros_like(live), z_coef=1.0)
    assert all(bool((t == 0).all()) for t in (counts, prob, stats, grad))
    counts, prob, stats, grad = itr.red_balance(x[:0], ids[:0])
    assert all(bool((t == 0).all()) for t in (counts, prob, stats)) and grad.shape == (0, experts)


def test_nan_in_a_token_that_takes_part():
    for rows in (60, 6000):
        x, ids, _ = inputs(rows, 64, 2, torch.float32)
        want = itr.red_balance(x, ids, coef=0.5)
        x[3, 7] = math.nan
        counts, prob, stats, grad = itr.red_balance(x, ids, coef=0.5)
        assert torch.equal(counts, want[0]) and bool(prob.isnan().all()) and bool(stats[:2].isnan().all())
        keep = torch.arange(rows, device=DEV) != 3
        assert bool(grad[3].isnan().all()) and torch.equal(grad[keep], want[3][keep])


def test_gradient_by_differences():
    """loss(x + h u) - loss(x - h u) with the ids, hence the counts, held."""
    for kind, z_coef in (("softmax", 0.05), ("sigmoid", 0.0)):
        x, ids, live = inputs(50, 24, 3, torch.float32)
        u = inputs(50, 24, 3, torch.float32, seed=9)[0]
        grad = itr.red_balance(x, ids, live=live, coef=1.0, z_coef=z_coef, kind=kind)[3]
        h = 1e-2

        def loss(v):
            return float(itr.red_balance(v, ids, live=live, coef=1.0, z_coef=z_coef, kind=kind)[2][0])

        slope = float((grad.double() * u.double()).sum())
        size = abs(loss(x))
        assert abs((loss(x + h * u) - loss(x - h * u)) / (2 * h) - slope) <= size * (50 * h * h + 2e-6 / h)


def test_in_place_streams_and_graphs():
    for rows, experts in ((100, 32), (9000, 128)):
        x, ids, live = inputs(rows, experts, 4, torch.bfloat16)
        want = itr.red_balance(x, ids, live=live, z_coef=1e-3)
        over = x.clone()
        got = itr.red_balance(over, ids, live=live, z_coef=1e-3, grad=over)
        assert got[3] is over and all(torch.equal(a, b) for a, b in zip(got, want))
        stream = torch.cuda.Stream()
        got = itr.red_balance(x, ids, live=live, z_coef=1e-3, stream=stream)
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = itr.red_balance(x, ids, live=live, z_coef=1e-3)
        for seed in (1, 2):
            y, i, m = inputs(rows, experts, 4, torch.bfloat16, 0.3 * seed, seed=seed)
            x.copy_(y), ids.copy_(i), live.copy_(m)
            graph.replay()
            torch.cuda.synchronize()
            check(x, ids, live, got, "softmax", 1.0, 1e-3, 1.0)


def test_refusals():
    x, ids, live = inputs(10, 16, 2, torch.float32)
    for call in (lambda: itr.red_balance(x.double(), ids), lambda: itr.red_balance(x, ids.int()),
                 lambda: itr.red_balance(x, ids[:9]), lambda: itr.red_balance(x, ids, live=live[:9]),
                 lambda: itr.red_balance(x, ids, live=live.float()), lambda: itr.red_balance(x, ids, kind="tanh"),
                 lambda: itr.red_balance(x, ids[:, 0]), lambda: itr.red_balance(x, ids, grad=x.half())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: itr.red_balance(x, ids, coef=math.nan), lambda: itr.red_balance(x, ids[:, :0]),
                 lambda: itr.red_balance(x, ids, kind="sigmoid", z_coef=0.1),
                 lambda: itr.red_balance(x, torch.zeros((10, 17), dtype=torch.int64, device=DEV))):
        with pytest.raises(itr.RedError):
            call()
