"""Losses over rows of logits where they are easily wrong: many rows without a
gradient, logits far from zero, waits that run out, NaN and infinities in each
input, memory of other streams."""
import math

import pytest
import torch

import int_tensor_reductions_gb300 as itr
import loss_reference as ref
from gpu_util import lib_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def device_gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def distill_loss(x, ids, vals):
    """(loss, size of its terms) per row in 64 bits, q = softmax(vals), no scale."""
    logp = torch.log_softmax(x.double(), 1).gather(1, ids)
    logq = torch.log_softmax(vals.double(), 1)
    q = logq.exp()
    return (q * (logq - logp)).sum(1), (q * (logq.abs() + logp.abs() + 30)).sum(1)


# Several rows per CTA, of one batch of the kernel's ring to many: each row's
# loss from its own statistics, though the next rows' are formed meanwhile.
@pytest.mark.parametrize("dtype,length,rows", [(torch.float32, 2100, 6000), (torch.float32, 5000, 4000),
                                               (torch.bfloat16, 13001, 3000), (torch.float16, 30000, 1500),
                                               (torch.float32, 40000, 800)])
def test_distill_loss_alone_over_many_rows(dtype, length, rows):
    g = device_gen(length)
    width = torch.rand((rows, 1), generator=g, device=DEV) * 4 + 0.1    # rows of very different statistics
    x = (torch.randn((rows, length), generator=g, device=DEV) * width).to(dtype)
    ids = torch.randint(0, length, (rows, 5), generator=g, device=DEV)
    vals = torch.randn((rows, 5), generator=g, device=DEV)
    loss, stats, grad = itr.red_distill(x, ids, vals, grad=False)
    assert grad is None and stats[1].item() == rows
    for part in torch.arange(rows, device=DEV).split(200):
        want, size = distill_loss(x[part], ids[part], vals[part])
        assert bool(((loss[part].double() - want).abs() <= 4e-5 * size + 1e-9).all())


def log_softmax(x, scale=1.0):
    """ref.log_softmax, computed on the device: (log p, lse) on the host."""
    z = x.double() * scale
    top = z.max(1, keepdim=True).values
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    norm = (z - base).exp().sum(1, keepdim=True).log()
    logp = torch.where(top == -math.inf, torch.full_like(z, -math.inf), z - base - norm)
    return logp.cpu(), (base + norm)[:, 0].cpu()


# Rows by groups of lanes, by two warps, by clusters and by the row kernel's
# CTAs.  1.163e7 is where s2 * x passes 2^24: maxima on both sides of it.
ROWS = [(5, 900), (300, 3500), (6, 9001), (6, 40000), (300, 9001), (300, 30000)]
FARAWAY = [(torch.float32, 1e3, 1.0), (torch.float32, -1e4, 0.7), (torch.float32, 1e6, 1.0), (torch.float32, 1.163e7, 1.0),
           (torch.float32, -1.163e7, 1.0), (torch.float32, 300.0, 30.0), (torch.float16, 1e4, 1.0),
           (torch.float16, 300.0, 30.0), (torch.bfloat16, -1e4, 1.25), (torch.bfloat16, 300.0, 30.0)]


@pytest.mark.parametrize("rows,length", ROWS)
@pytest.mark.parametrize("dtype,offset,scale", FARAWAY)
def test_logits_far_from_zero(rows, length, dtype, offset, scale):
    """A constant added to a row changes no probability: what a row's parts of
    different maxima add up to is as near as at zero."""
    g = device_gen(length + rows)
    width = 3.0 / scale if scale > 1 else 3.0
    x = (torch.randn((rows, length), generator=g, device=DEV) * width + offset).to(dtype)
    t = torch.randint(0, length, (rows,), generator=g, device=DEV)
    lp, lse = log_softmax(x, scale)
    want, live = ref.taken(lp, t.cpu())
    p = lp.exp()
    got, norm = itr.red_logprob(x, t, scale=scale)
    ref.assert_logp(got, want, "logp")
    ref.assert_logp(norm, lse, "lse")
    old = want.float().to(DEV)
    down = torch.full((rows,), -1.0, device=DEV)
    _, got, _, grad = itr.red_policy(x, t, old, down, scale=scale)
    ref.assert_logp(got, want, "policy")
    # the ratio is 1 up to the rounding of old and the error of logp
    c = torch.full((rows,), scale, dtype=torch.float64)
    extra = 3e-5 + 2.0 ** -23 * float(want.abs().max())
    ref.assert_grad(grad, ref.target_grad(lp, lse, t.cpu(), live, c), p, c, t.cpu(), extra=extra, what="policy")
    ids = torch.randint(0, length, (rows, 3), generator=g, device=DEV)
    vals = torch.zeros((rows, 3), device=DEV)
    loss, _, grad = itr.red_distill(x, ids, vals, scale=scale)
    at = lp.gather(1, ids.cpu())
    size = math.log(3.0) + at.abs().mean(1)
    assert bool(((loss.cpu().double() - (-math.log(3.0) - at.mean(1))).abs() <= 1.2e-5 + 1e-6 * size).all())
    mass = torch.zeros_like(p).scatter_add_(1, ids.cpu(), torch.full((rows, 3), 1 / 3, dtype=torch.float64))
    ref.assert_grad(grad, (p - mass) * scale, p + mass, c, extra=3e-5, what="distill")


def check_preference(x, t, offsets, w=None, kind="sigmoid", beta=0.5, margin=0.0, eps=0.0, average=False, scale=1.0,
                     gs=1.0, rf=None, only=None):
    """red_preference against 64 bits, each row's gradient by the tolerance of
    its own pair; ``only``: the rows whose gradient is compared."""
    rows, pairs = x.shape[0], offsets.numel() // 2
    w = torch.ones(pairs) if w is None else w
    rf = torch.zeros(2 * pairs) if rf is None else rf
    loss, seq, stats, grad = itr.red_preference(
        x, t, offsets.to(DEV), ref_logp=rf.to(DEV), weight=w.to(DEV), kind=kind, beta=beta, margin=margin, smoothing=eps,
        average=average, scale=scale, grad_scale=gs)
    lp, lse = log_softmax(x, scale)
    tc = t.cpu()
    logp, live = ref.taken(lp, tc)
    live = live & (lse != -math.inf)
    of = torch.bucketize(torch.arange(rows), offsets[1:], right=True)
    inside = (torch.arange(rows) >= offsets[0]) & (of < 2 * pairs)
    live, of = live & inside, of.clamp(max=2 * pairs - 1)
    zero = torch.zeros(2 * pairs, dtype=torch.float64)
    count = zero.index_add(0, of, live.double()).clamp(min=1.0) if average else zero + 1.0
    sums = zero.index_add(0, of[live], logp[live]) / count
    # the sums' errors: 1.2e-5 and 4e-7 |logp| per token
    slack = zero.index_add(0, of[live], 1.2e-5 + 4e-7 * logp[live].abs()) / count
    assert bool(((seq.cpu().double() - sums).abs() <= slack + 2e-7 * sums.abs()).all())
    gain = sums - rf.double()
    u = beta * (gain[:pairs] - gain[pairs:]) - margin
    want, du = ref.pair_loss(u, kind, beta, eps)
    du_u = beta * (slack[:pairs] + slack[pairs:]) + 2e-7 * (u.abs() + beta * gain.abs().max()) + 1e-7
    curve = {"sigmoid": 0.25, "hinge": 0.0, "squared": 2.0 / beta ** 2}[kind] * du_u
    if kind == "hinge":
        curve = ((u - 1).abs() <= du_u).double()     # either side of the kink
    wd = w.double()
    assert bool(((loss.cpu().double() - want * wd).abs() <= wd * (du_u * (du.abs() + curve) + 2e-6 * want.abs() + 1e-7)).all())
    f = wd * beta * gs * scale
    c, dc = torch.cat([du * f, -du * f]) / count, torch.cat([curve * f, curve * f]) / count + 0.0
    c, dc = c[of], dc[of] + 2e-6 * c[of].abs()
    c, dc = torch.where(live, c, torch.zeros_like(c)), torch.where(live, dc, torch.zeros_like(dc))
    only = torch.arange(rows) if only is None else only
    p = lp[only].exp()
    g = ref.target_grad(lp[only], lse[only], tc[only], live[only], c[only])
    got = grad[only.to(DEV)].cpu().double()
    tol = p.nan_to_num(nan=0.0) * (c[only].abs() * ref.PROB_REL + dc[only])[:, None]
    tol += ref.ROUND[x.dtype] * g.abs() + ref.TINY[x.dtype]
    at = tc[only].clamp(0, x.shape[1] - 1)
    tol[torch.arange(only.numel()), at] += 1e-6 * c[only].abs() + dc[only]
    bad = ~((got - g).abs() <= tol)
    assert not bad.any(), (f"{int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}: {got[bad][0]} for {g[bad][0]} "
                           f"+- {tol[bad][0]}")
    return loss, seq, stats, grad


@pytest.mark.parametrize("rows,length", ROWS)
@pytest.mark.parametrize("dtype,offset,scale", FARAWAY)
def test_preference_far_from_zero(rows, length, dtype, offset, scale):
    """The gradient's probabilities do not suffer from the size of the row's
    log-sum-exp."""
    g = device_gen(length + rows)
    width = 3.0 / scale if scale > 1 else 3.0
    x = (torch.randn((rows, length), generator=g, device=DEV) * width + offset).to(dtype)
    t = torch.randint(0, length, (rows,), generator=g, device=DEV)
    pairs = min(rows // 2, 40)      # the few-row kernel's last CTA does few pairs, a kernel of their own more
    off = torch.linspace(0, rows, 2 * pairs + 1).round().long()
    # the squared loss pulls even where the policy has decided
    check_preference(x, t, off, kind="squared", average=True, scale=scale)


@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("copies,length", [(1, 700), (60, 700), (1, 9000), (60, 9000), (1, 40000), (32, 40000)])
def test_preference_of_extreme_rows(copies, length, dtype):
    """Rows whose masks leave little or nothing, and rows of nothing but the
    type's lowest or highest value, which are uniform."""
    low = torch.finfo(dtype).min
    rows = 10 * copies
    g = device_gen(length)
    x = (torch.randn((rows, length), generator=g, device=DEV) * 3).to(dtype)
    t = torch.full((rows,), 1)
    k = torch.arange(rows) % 10
    x[k == 0, length // 2:] = -math.inf
    x[k == 1, :length - 2] = -math.inf
    t[k == 1] = length - 1
    x[k == 2] = -math.inf               # nothing left
    x[k == 3] = low                     # uniform
    x[k == 4, 2:] = low
    x[k == 5, :length - 2] = low        # a prefix far below the rest
    t[k == 5] = length - 2
    x[k == 6] = -low                    # uniform at the other end
    t[k == 7] = -100
    x[k == 7] = math.nan
    pairs = rows // 5
    off = torch.linspace(0, rows, 2 * pairs + 1).round().long()
    check_preference(x, t.to(DEV), off, kind="squared", average=True, scale=1.0, gs=2.0)


@pytest.mark.parametrize("kind,average", [("sigmoid", False), ("sigmoid", True), ("hinge", False), ("squared", True)])
@pytest.mark.parametrize("rows,length,pairs", [(64, 4099, 8), (900, 257, 200), (600, 9001, 50)])
def test_preference_by_its_own_pair(rows, length, pairs, kind, average):
    """Each pair's rows within the tolerance of that pair, saturated ones among
    them."""
    g = device_gen(rows)
    x = (torch.randn((rows, length), generator=g, device=DEV) * 3).to(torch.float32)
    t = torch.randint(0, length, (rows,), generator=g, device=DEV)
    t[torch.rand(rows, generator=g, device=DEV) < 0.3] = -100
    off = torch.randint(0, rows + 1, (2 * pairs + 1,), generator=g, device=DEV).cpu().sort().values
    w = torch.rand(pairs) + 0.05
    w[::7] = 0.0
    rf = torch.randn(2 * pairs) * 4
    rf[0] += 60.0       # a pair of no doubt
    check_preference(x, t, off, w=w, kind=kind, beta=0.6, margin=0.1, eps=0.1 if kind == "sigmoid" else 0.0,
                     average=average, scale=0.9, gs=3.0, rf=rf)


def test_preference_of_many_rows():
    """More rows than the workspace has room for their statistics, at an offset."""
    rows, length = (1 << 21) + 1003, 6
    g = device_gen(3)
    x = torch.randn((rows, length), generator=g, device=DEV) * 2 + 3e4
    t = torch.randint(0, length, (rows,), generator=g, device=DEV)
    off = torch.tensor([5, 1000000, rows - 3])
    only = torch.cat([torch.arange(2000), torch.arange((1 << 21) - 700, rows)])
    check_preference(x, t, off, kind="hinge", average=True, only=only)


@pytest.mark.parametrize("dtype,length,rows", [(torch.float32, 9001, 400), (torch.bfloat16, 30001, 300),
                                               (torch.float32, 70001, 300)])
def test_wait_that_runs_out(dtype, length, rows):
    """A wait that gives up at its first try in vain: rows whose copies it did
    not wait for are NaN, in every output, and none holds anything else that is
    wrong.  The calls after it are as before."""
    g = device_gen(rows)
    x = (torch.randn((rows, length), generator=g, device=DEV) * 3).to(dtype)
    t = torch.randint(0, length, (rows,), generator=g, device=DEV)
    t[::5] = -100
    live = t >= 0
    f = torch.randn(rows, generator=g, device=DEV)
    ids = torch.randint(0, length, (rows, 5), generator=g, device=DEV)
    vals = torch.randn((rows, 5), generator=g, device=DEV)
    w = live.float()
    off = torch.linspace(0, rows, 2 * 20 + 1).round().long().to(DEV)
    lse = itr.red_logprob(x, t)[1]
    calls = [lambda: itr.red_logprob(x, t),
             lambda: (itr.red_logprob_grad(x, t, lse, f),),
             lambda: itr.red_policy(x, t, f - 9, f),
             lambda: itr.red_distill(x, ids, vals, weight=w),
             lambda: itr.red_distill(x, ids, vals, weight=w, grad=False)[:1],
             lambda: itr.red_preference(x, t, off)]
    good = [call() for call in calls]
    itr.red_set_knob(itr.RED_KNOB_LOSS_TRIES, 1)
    try:
        bad = [call() for call in calls]
        torch.cuda.synchronize()
    finally:
        itr.red_set_knob(itr.RED_KNOB_LOSS_TRIES, 0)
    for a, b in zip(good, bad):
        for u, v in zip(a, b):
            nan = v.isnan()
            assert bool(nan.any())
            if u.shape[0] == rows:      # results of rows: NaN or what they are; those out of the loss 0
                assert bool((nan | (u == v)).all()) and bool((v[~live] == 0).all())
    for call, a in zip(calls, good):
        for u, v in zip(a, call()):
            assert torch.equal(u, v)


def test_hinge_of_nan():
    """NaN in a token makes its pair's loss and gradient NaN, and no other's."""
    for length in (60, 9000):
        x = torch.randn((8, length), generator=device_gen(1), device=DEV)
        t = torch.full((8,), 3, device=DEV)
        x[1, 5] = math.nan
        for kind in ("hinge", "sigmoid", "squared"):
            loss, _, _, grad = itr.red_preference(x, t, torch.tensor([0, 2, 4, 6, 8], device=DEV), kind=kind)
            assert math.isnan(loss[0].item()) and math.isfinite(loss[1].item())
            assert bool(grad[[0, 1, 4, 5]].isnan().all()) and bool(grad[[2, 3, 6, 7]].isfinite().all())


def test_policy_nan_without_advantage():
    """No advantage does not hide a NaN, and makes nothing of an infinite ratio
    or of a token that neither policy gives."""
    for length in (60, 9000):
        x = torch.randn((5, length), generator=device_gen(1), device=DEV)
        t = torch.full((5,), 3, device=DEV)
        old, adv = torch.full((5,), -5.0, device=DEV), torch.zeros(5, device=DEV)
        x[0, 7] = math.nan
        old[1] = -1000.0
        x[2, 3] = -math.inf
        old[2] = -math.inf
        old[3] = math.nan
        loss, logp, _, grad = itr.red_policy(x, t, old, adv)
        for r in (0, 3):
            assert math.isnan(loss[r].item()) and bool(grad[r].isnan().all())
        for r in (1, 2, 4):
            assert loss[r].item() == 0.0 and bool((grad[r] == 0).all())
        assert math.isnan(logp[0].item()) and logp[2].item() == -math.inf


def test_policy_drift_of_a_token_ruled_out():
    """A token that the reference gives and the policy does not: e^d - d - 1 is
    infinite, not NaN; likewise one that the reference alone rules out."""
    for length in (60, 9000):
        x = torch.randn((3, length), generator=device_gen(1), device=DEV)
        t = torch.full((3,), 3, device=DEV)
        x[0, 3] = -math.inf
        old, adv = torch.full((3,), -5.0, device=DEV), torch.ones(3, device=DEV)
        rf = torch.tensor([-4.0, -math.inf, -5.0], device=DEV)
        loss, _, stats, _ = itr.red_policy(x, t, old, adv, ref_logp=rf, kl_coef=0.1)
        assert loss[0].item() == loss[1].item() == math.inf and math.isfinite(loss[2].item())
        assert stats[0].item() == math.inf


@pytest.mark.parametrize("normalised", [False, True])
@pytest.mark.parametrize("offset,scale", [(0.0, 1.0), (1e4, 0.7), (-1e5, 1.25), (300.0, 30.0)])
@pytest.mark.parametrize("rows,length", [(40, 500), (5, 9001), (300, 9001)])
def test_teacher_logits_far_from_zero(rows, length, offset, scale, normalised):
    """A constant in all of a teacher's logits changes no q."""
    k = 12
    g = device_gen(rows)
    x = torch.randn((rows, length), generator=g, device=DEV) / scale
    ids = torch.stack([torch.randperm(length, generator=g, device=DEV)[:k] for _ in range(rows)])
    vals = torch.randn((rows, k), generator=g, device=DEV) * 2 / scale + offset
    scale = float(torch.tensor(scale, dtype=torch.float32))     # as the call has it: 1.7e-8 of 7000 is not nothing
    lse = torch.logsumexp(vals.double() * scale, 1).float() + 0.5 if normalised else None
    loss, _, grad = itr.red_distill(x, ids, vals, lse=lse, scale=scale)
    v = vals.double() * scale
    logq = v - (lse.double()[:, None] if normalised else torch.logsumexp(v, 1, keepdim=True))
    q = logq.exp()
    lp = log_softmax(x, scale)[0]
    at = lp.gather(1, ids.cpu())
    logq, q = logq.cpu(), q.cpu()
    want = (q * (logq - at)).sum(1)
    # log q is off by a few roundings of its size (at most 20), q by as much relative
    assert bool(((loss.cpu().double() - want).abs() <= 4e-5 * (q * (logq.abs() + at.abs() + 1)).sum(1)).all())
    p = lp.exp() * q.sum(1, keepdim=True)
    mass = torch.zeros_like(p).scatter_add_(1, ids.cpu(), q)
    c = torch.full((rows,), scale, dtype=torch.float64)
    ref.assert_grad(grad, (p - mass) * scale, p + mass, c, extra=3e-5)


def test_teacher_of_lowest_values():
    """A teacher's list of nothing but the lowest value is uniform, at any scale."""
    x = torch.randn((3, 500), generator=device_gen(2), device=DEV)
    ids = torch.tensor([[1, 5, 9, 200]] * 3, device=DEV)
    vals = torch.full((3, 4), torch.finfo(torch.float32).min, device=DEV)
    flat = itr.red_distill(x, ids, torch.zeros_like(vals), scale=1.25)
    for a, b in zip(itr.red_distill(x, ids, vals, scale=1.25), flat):
        assert torch.equal(a, b)


def test_results_are_memory_of_the_calls_stream():
    """A block that the current stream's program gave back may be in use there
    still: a call on another stream does not get it."""
    rows, length = 400_000, 8
    x = torch.randn((rows, length), generator=device_gen(1), device=DEV)
    t = torch.randint(0, length, (rows,), generator=device_gen(2), device=DEV)
    f = torch.randn(rows, generator=device_gen(3), device=DEV)
    ids, vals = t[:, None].expand(rows, 2).contiguous(), torch.zeros((rows, 2), device=DEV)
    off = torch.linspace(0, rows, 2 * 30000 + 1).round().long().to(DEV)
    lse = itr.red_logprob(x, t)[1]
    calls = [lambda s: itr.red_logprob(x, t, stream=s),
             lambda s: (itr.red_logprob_grad(x, t, lse, f, stream=s),),
             lambda s: itr.red_policy(x, t, f - 2, f, stream=s),
             lambda s: itr.red_distill(x, ids, vals, stream=s),
             lambda s: itr.red_preference(x, t, off, stream=s)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        for call in calls:
            want = call(None)
            torch.cuda.synchronize()
            sizes = [v.untyped_storage().nbytes() for v in want]
            blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
            spans = [(b.data_ptr(), b.data_ptr() + b.numel()) for b in blocks]
            del blocks
            got = call(stream)
            for u, v in zip(want, got):
                assert not any(lo <= v.data_ptr() < hi for lo, hi in spans)
            side.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(want, got))
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
            del want, got


def test_kind_is_not_cut_to_32_bits():
    x = torch.zeros((2, 5), device=DEV)
    t = torch.zeros(2, dtype=torch.int64, device=DEV)
    off = torch.arange(3, device=DEV)
    for kind in (1 << 32, -(1 << 32), (1 << 32) + 1):
        with pytest.raises(ValueError):
            itr.red_preference(x, t, off, kind=kind)
    for kind in (3, -1):
        with pytest.raises(itr.RedError):
            itr.red_preference(x, t, off, kind=kind)
