"""Log-probabilities from hidden states and weights, and their gradients,
against the 64-bit definition: types, odd sizes and strides, ignored rows,
extreme values, streams, graphs and repeatability."""
import math

import pytest
import torch

import int_tensor_reductions_gb300 as itr
from gpu_util import lib_ready
from linear_reference import Reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def matrix(rows, cols, dtype, pad=0, fill=math.nan):
    """A (rows, cols) view of row stride up(cols, 8) + pad, `fill` in between."""
    ld = (cols + 7) // 8 * 8 + pad
    return torch.full((rows, ld), fill, dtype=dtype, device=DEV)[:, :cols]


def inputs(rows, dim, vocab, dtype, ignore=0.25, pad=0, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows + 3 * dim + 7 * vocab + seed)
    weight = matrix(vocab, dim, dtype, pad)
    weight.copy_(torch.randn((vocab, dim), generator=g, device=DEV) * (1.5 / math.sqrt(dim)))
    target = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    hidden = matrix(rows, dim, dtype, 2 * pad)
    lift = torch.rand((rows, 1), generator=g, device=DEV) * 5
    hidden.copy_(torch.randn((rows, dim), generator=g, device=DEV) + weight[target].float() * lift)
    drop = torch.rand(rows, generator=g, device=DEV) < ignore
    outside = torch.tensor([-100, -1, vocab, 2 ** 40], device=DEV)
    target[drop] = outside[torch.randint(0, 4, (rows,), generator=g, device=DEV)][drop]
    dlogp = torch.randn(rows, generator=g, device=DEV)
    dlse = torch.randn(rows, generator=g, device=DEV) * 0.1
    return hidden, weight, target, dlogp, dlse


SHAPES = [(1, 8, 1), (1, 1, 5), (2, 64, 256), (3, 70, 257), (5, 100, 1000), (16, 1040, 777), (17, 200, 5000), (33, 136, 130), (64, 512, 2049), (100, 2056, 20000), (128, 72, 255),
          (129, 576, 513), (255, 64, 4097), (256, 1000, 300), (257, 1032, 1111), (300, 24, 9000), (1000, 520, 3001),
          (4100, 40, 700)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,dim,vocab", SHAPES)
def test_forward_and_gradients(rows, dim, vocab, dtype):
    for pad, scale, ignore, with_lse in ((0, 1.0, 0.25, False), (8, 0.7, 0.0, True), (0, 1.25, 0.6, True)):
        hidden, weight, target, dlogp, dlse = inputs(rows, dim, vocab, dtype, ignore, pad)
        dlse = dlse if with_lse else None
        ref = Reference(hidden, weight, target, scale)
        logp, lse = itr.red_linear_logprob(hidden, weight, target, scale=scale)
        ref.check_forward(logp, lse)
        gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, dlse=dlse, scale=scale)
        assert gh.dtype == dtype and gh.shape == hidden.shape and gw.shape == weight.shape
        ref.check_gradients(gh, gw, dlogp, dlse)


def test_pieces_of_a_long_vocabulary():
    """More rows and columns than one piece of the vocabulary holds."""
    hidden, weight, target, dlogp, _ = inputs(9000, 32, 20000, torch.bfloat16)
    ref = Reference(hidden, weight, target)
    logp, lse = itr.red_linear_logprob(hidden, weight, target)
    ref.check_forward(logp, lse)
    ref.check_gradients(*itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp), dlogp)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_out_of_the_loss_reach_nothing(dtype):
    """NaN and infinities in ignored rows, rows of no coefficient, and columns between dim and the stride."""
    for rows in (7, 300):
        hidden, weight, target, dlogp, dlse = inputs(rows, 72, 600, dtype, 0.5, pad=8)
        target[0] = 3
        dlogp[::3] = 0.0
        dlse[::3] = 0.0
        dlogp[1::3] = 0.0  # the normaliser alone
        clean = hidden.clone()
        ref = Reference(clean, weight, target)
        hidden[~ref.live] = math.nan
        hidden[~ref.live, 1] = math.inf
        logp, lse = itr.red_linear_logprob(hidden, weight, target)
        ref.check_forward(logp, lse)
        hidden[(dlogp == 0) & (dlse == 0)] = math.nan
        for got in ((itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, dlse=dlse)),):
            ref.check_gradients(*got, dlogp, dlse)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 40, 400])
def test_nothing_takes_part(rows, dtype):
    hidden, weight, target, dlogp, _ = inputs(rows, 64, 300, dtype)
    hidden[:] = math.nan
    target[:] = -100
    logp, lse = itr.red_linear_logprob(hidden, weight, target)
    assert bool((logp == 0).all() and (lse == 0).all())
    gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
    assert bool((gh == 0).all() and (gw == 0).all())


def test_no_rows():
    hidden, weight, target, dlogp, _ = inputs(4, 64, 300, torch.bfloat16)
    logp, lse = itr.red_linear_logprob(hidden[:0], weight, target[:0])
    assert logp.numel() == lse.numel() == 0
    gh, gw = itr.red_linear_logprob_grad(hidden[:0], weight, target[:0], lse, dlogp[:0])
    assert gh.shape == (0, 64) and bool((gw == 0).all())


@pytest.mark.parametrize("rows", [5, 300])
def test_results_to_write(rows):
    """Given results, one of the two alone, the gradient over the hidden states; what lies between their rows stays."""
    dtype = torch.bfloat16
    hidden, weight, target, dlogp, _ = inputs(rows, 100, 700, dtype)
    _, lse = itr.red_linear_logprob(hidden, weight, target)
    gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
    oh, ow = matrix(rows, 100, dtype, 16, 7.25), matrix(700, 100, dtype, 24, 7.25)
    got = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, grad_hidden=oh, grad_weight=ow)
    assert got[0] is oh and got[1] is ow and torch.equal(oh, gh) and torch.equal(ow, gw)
    for t in (oh, ow):
        whole = t.as_strided((t.shape[0], t.stride(0)), t.stride())
        assert bool((whole[:, 100:] == 7.25).all())
    a, none = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, grad_weight=False)
    assert none is None and torch.equal(a, gh)
    none, a = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, grad_hidden=False)
    assert none is None and torch.equal(a, gw)
    got = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, grad_hidden=hidden)
    assert got[0] is hidden and torch.equal(hidden, gh) and torch.equal(got[1], gw)


@pytest.mark.parametrize("rows", [3, 290])
def test_extreme_logits(rows):
    """Logits of thousands, one entry that has all the weight, a target of none."""
    hidden, weight, target, dlogp, _ = inputs(rows, 64, 900, torch.bfloat16, 0.0)
    hidden *= 300.0
    ref = Reference(hidden, weight, target)
    logp, lse = itr.red_linear_logprob(hidden, weight, target)
    ref.check_forward(logp, lse)
    # lse in 32 bits shifts every p by its rounding
    ref.check_gradients(*itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp), dlogp)


@pytest.mark.parametrize("rows", [3, 290])
def test_nan_and_infinity_stay_in_their_row(rows):
    hidden, weight, target, dlogp, _ = inputs(rows, 64, 900, torch.bfloat16, 0.0)
    ref = Reference(hidden, weight, target)
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    bad[1] = bad[2] = True
    hidden[1, 3] = math.nan
    hidden[2, 5] = math.inf
    logp, lse = itr.red_linear_logprob(hidden, weight, target)
    assert bool(logp[bad].isnan().all() and lse[bad].isnan().all())
    assert bool(logp[~bad].isfinite().all()) and float((lse - ref.lse)[~bad].abs().max()) < 1e-3
    gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
    assert bool(gh[bad].isnan().all()) and bool(gh[~bad].isfinite().all())
    assert bool(gw.isnan().all())


def test_half_precision_coefficients():
    """A mean over many rows, without a loss scale: coefficients far below f16's smallest."""
    hidden, weight, target, dlogp, dlse = inputs(300, 64, 1000, torch.float16, 0.0)
    hidden *= 4.0
    _, lse = itr.red_linear_logprob(hidden, weight, target)
    ref = Reference(hidden, weight, target)
    for size in (1e-4, 1e-2, 30.0):
        got = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp * size, dlse=dlse * size)
        ref.check_gradients(*got, dlogp * size, dlse * size)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [2, 200])
def test_even_choice_of_many(rows, dtype):
    """Probabilities of 4e-6 keep their digits in the 16-bit gradient by the logits: hidden states of one value,
    and weights of 0 but for a constant, make every p = 1 / vocab."""
    vocab, dim = 2 ** 18, 32
    hidden = torch.full((rows, dim), 0.5, dtype=dtype, device=DEV)
    weight = torch.full((vocab, dim), 0.25, dtype=dtype, device=DEV)
    target = torch.arange(rows, device=DEV) * 1000
    dlogp = torch.linspace(-300.0, -100.0, rows, device=DEV)
    logp, lse = itr.red_linear_logprob(hidden, weight, target)
    gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
    want = -0.5 * float(dlogp.double().sum()) / vocab  # of every token that is no target
    rest = torch.ones(vocab, dtype=torch.bool, device=DEV)
    rest[target] = False
    # g and the result are rounded once each, p is off by the rounding of lse = 16.5 (2e-6) and its own 3e-5
    half = torch.finfo(dtype).eps / 2
    assert float((gw[rest].double() / want - 1).abs().max()) <= 2 * half + half * half + 4e-5


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [3, 290])
def test_almost_certain(rows, dtype):
    """log p of about -1e-4, relative to itself: what the others' logits and the target's are off by, the sum of their
    exponentials (3e-5), and the rounding of the arguments."""
    hidden, weight, target, _, _ = inputs(rows, 64, 900, dtype, 0.0)
    hidden.copy_(9.0 * weight[target].float())
    ref = Reference(hidden, weight, target)
    logp, _ = itr.red_linear_logprob(hidden, weight, target)
    assert float(ref.logp.median()) > -1e-2
    z = ref.lse.abs() + ref.logp.abs()
    off = (logp.double() - ref.logp).abs() / ref.logp.abs()
    assert bool((off <= 2 * ref.dz + 3e-5 + z * 4 * 2.0 ** -24).all())


@pytest.mark.parametrize("rows", [3, 290])
def test_token_ruled_out(rows):
    """Weights of -inf where all hidden states are above 0: a token without a probability, target or not."""
    hidden, weight, target, _, _ = inputs(rows, 64, 900, torch.bfloat16, 0.0)
    hidden[:, 7] = 1.0
    weight[5, 7] = -math.inf
    target[:] = target.where(target != 5, 6)
    target[1] = 5
    z = hidden.double() @ weight.double().t()
    logp, lse = itr.red_linear_logprob(hidden, weight, target)
    want = torch.logsumexp(z, 1)
    tol = 1e-3  # (logits of some tens: the finite ones are held to more elsewhere)
    assert float((lse.double() - want).abs().max()) < tol
    assert float(logp[1]) == -math.inf
    rest = torch.arange(rows, device=DEV) != 1
    want = z.gather(1, target[:, None])[:, 0] - want
    assert float((logp.double() - want)[rest].abs().max()) < tol


def test_gradient_by_differences():
    """The forward pass at both sides, along directions of 16-bit steps."""
    rows, dim, vocab = 20, 64, 500
    hidden, weight, target, dlogp, dlse = inputs(rows, dim, vocab, torch.float16, 0.1)
    hidden.copy_((hidden.float() * 16).round() / 16)
    weight.copy_((weight.float() * 256).round() / 256)
    _, lse = itr.red_linear_logprob(hidden, weight, target)
    gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, dlse=dlse)

    def loss(h, w):
        logp, lse = itr.red_linear_logprob(h, w, target)
        return float((logp.double() * dlogp).sum() + (lse.double() * dlse).sum())

    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    for which, grad, step in (("h", gh, 2.0 ** -4), ("w", gw, 2.0 ** -8)):
        base = hidden if which == "h" else weight
        sign = torch.randint(0, 2, base.shape, generator=g, device=DEV) * 2 - 1
        u = (sign * step).to(torch.float16)
        up, down = (loss(base + u, weight), loss(base - u, weight)) if which == "h" else \
            (loss(hidden, base + u), loss(hidden, base - u))
        slope = float((grad.double() * u.double()).sum())
        # logits move by e = |u . w| (or |h . u|): the third order is below e^3 / 10 a row, and each loss is off by
        # the forward's tolerance
        move = float((u.double() @ weight.double().t()).abs().max() if which == "h" else
                     (hidden.double() @ u.double().t()).abs().max())
        size = float((dlogp.abs() + dlse.abs()).sum())
        noise = size * 3e-5 + float((grad.double() * u.double()).abs().sum()) * 2.0 ** -11
        # g's rounding, relative to the logits' moves that it weighs
        noise += size * 2 * move * 2.0 ** -11
        assert abs((up - down) / 2 - slope) <= size * move ** 3 / 10 + noise


def test_same_targets_and_repeatability():
    """One token everywhere; the same bits from call to call."""
    hidden, weight, target, dlogp, _ = inputs(700, 264, 3000, torch.bfloat16, 0.0)
    target[:] = 1234
    ref = Reference(hidden, weight, target)
    logp, lse = itr.red_linear_logprob(hidden, weight, target)
    ref.check_forward(logp, lse)
    gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
    ref.check_gradients(gh, gw, dlogp)
    for _ in range(3):
        again = itr.red_linear_logprob(hidden, weight, target)
        assert torch.equal(again[0], logp) and torch.equal(again[1], lse)
        again = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
        assert torch.equal(again[0], gh) and torch.equal(again[1], gw)


def test_streams_side_by_side():
    """Two calls at once, each on its own stream with its own scratch."""
    sets = [inputs(200 + 150 * i, 136, 5000, torch.bfloat16, seed=i) for i in range(2)]
    want = []
    for hidden, weight, target, dlogp, _ in sets:
        logp, lse = itr.red_linear_logprob(hidden, weight, target)
        want.append((logp, lse, *itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, (hidden, weight, target, dlogp, _) in zip(streams, sets):
            logp, lse = itr.red_linear_logprob(hidden, weight, target, stream=s)
            got.append((logp, lse, *itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, stream=s)))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("rows", [9, 600])
def test_graph(rows):
    """Captured once, replayed on other inputs of the same buffers."""
    hidden, weight, target, dlogp, _ = inputs(rows, 128, 1500, torch.bfloat16)
    itr.red_linear_logprob(hidden, weight, target)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        logp, lse = itr.red_linear_logprob(hidden, weight, target)
        gh, gw = itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp)
    for seed in (1, 2):
        h, w, t, d, _ = inputs(rows, 128, 1500, torch.bfloat16, 0.1 * seed, seed=seed)
        hidden.copy_(h), weight.copy_(w), target.copy_(t), dlogp.copy_(d)
        graph.replay()
        torch.cuda.synchronize()
        ref = Reference(h, w, t)
        ref.check_forward(logp, lse)
        ref.check_gradients(gh, gw, d)


def test_refusals():
    hidden, weight, target, dlogp, _ = inputs(4, 64, 300, torch.bfloat16)
    lse = dlogp.clone()
    with pytest.raises(ValueError):
        itr.red_linear_logprob(hidden.float(), weight.float(), target)
    with pytest.raises(ValueError):
        itr.red_linear_logprob(hidden, weight.half(), target)
    with pytest.raises(ValueError):
        itr.red_linear_logprob(hidden, weight[:, :60], target)
    with pytest.raises(ValueError):
        itr.red_linear_logprob(hidden, weight, target.int())
    with pytest.raises(ValueError):
        itr.red_linear_logprob(hidden.t(), weight, target)
    with pytest.raises(itr.RedError):
        itr.red_linear_logprob(hidden[:, 1:], weight[:, :63], target)  # not on a 16-byte boundary
    odd = torch.zeros((4, 63), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(itr.RedError):
        itr.red_linear_logprob(odd, weight[:, :63], target)  # rows of 126 bytes
    with pytest.raises(itr.RedError):
        itr.red_linear_logprob(hidden, weight, target, scale=0.0)
    with pytest.raises(itr.RedError):
        itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, grad_hidden=False, grad_weight=False)
    with pytest.raises(itr.RedError):
        itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, grad_weight=weight)
    with pytest.raises(ValueError):
        itr.red_linear_logprob_grad(hidden, weight, target, lse, dlogp, grad_hidden=weight)
    with pytest.raises(ValueError):
        itr.red_linear_logprob_grad(hidden, weight, target, lse[:3], dlogp)
