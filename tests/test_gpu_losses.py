"""Losses over rows of logits against their 64-bit definitions: types, row
lengths and strides, ignored and fully masked rows, extreme logits, gradients
by formula and by differences, streams, graphs and repeatability."""
import math

import pytest
import torch

import int_tensor_reductions_gb300 as itr
import loss_reference as ref
from gpu_util import lib_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = 7.25  # what columns beyond a row hold


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def logits(rows, length, dtype, seed, pad=0, shift=0, width=3.0):
    """(x, buffer): x a (rows, length) view of row stride length + pad that
    starts `shift` elements into its buffer; the rest holds NaN."""
    ld = length + pad
    buf = torch.full((shift + rows * ld,), math.nan, dtype=dtype, device=DEV)
    x = buf[shift:].view(rows, ld)[:, :length]
    x.copy_(torch.randn((rows, length), generator=gen(seed)) * width)
    return x, buf


def targets(rows, length, seed, ignore=0.2):
    g = gen(seed + 1000)
    t = torch.randint(0, length, (rows,), generator=g)
    drop = torch.rand(rows, generator=g) < ignore
    t[drop] = torch.tensor([-100, -1, length, 2 ** 40])[torch.randint(0, 4, (int(drop.sum()),), generator=g)]
    return t


def out_like(x, pad=0, shift=0):
    rows, length = x.shape
    buf = torch.full((shift + rows * (length + pad),), GUARD, dtype=x.dtype, device=DEV)
    return buf[shift:].view(rows, length + pad)[:, :length], buf


def guard_intact(buf, view):
    probe = buf.clone()
    probe.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(GUARD)
    assert bool((probe == GUARD).all()), "write outside the gradient"


SHAPES = [(1, 1), (3, 2), (5, 7), (4, 31), (33, 32), (2, 33), (70, 257), (9, 1000), (300, 1024), (5, 4099),
          (150, 8192), (3, 16385), (2, 32001), (1, 65536), (1, 131073), (400, 4100), (170, 20001)]


@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("rows,length", SHAPES)
def test_logprob(rows, length, dtype):
    for pad, shift, scale in ((0, 0, 1.0), (3, 1, 0.7), (64, 0, 1.25)):
        x, _ = logits(rows, length, dtype, rows + length, pad, shift)
        t = targets(rows, length, rows)
        logp, lse = itr.red_logprob(x, t.to(DEV), scale=scale)
        lp, norm = ref.log_softmax(x, scale)
        want, live = ref.taken(lp, t)
        ref.assert_logp(logp, want, "logp")
        ref.assert_logp(lse, torch.where(live, norm, torch.zeros_like(norm)), "lse")


@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("rows,length", SHAPES)
def test_logprob_grad(rows, length, dtype):
    g = gen(3 * rows + length)
    for pad, shift, opad, oshift, scale in ((0, 0, 0, 0, 1.0), (3, 1, 3, 1, 0.7), (64, 0, 5, 3, 1.25)):
        x, _ = logits(rows, length, dtype, rows + length, pad, shift)
        t = targets(rows, length, rows)
        lp, norm = ref.log_softmax(x, scale)
        _, live = ref.taken(lp, t)
        lse = norm.float()
        d = torch.randn(rows, generator=g)
        d[::7] = 0.0
        out, buf = out_like(x, opad, oshift)
        got = itr.red_logprob_grad(x, t.to(DEV), lse.to(DEV), d.to(DEV), scale=scale, out=out)
        assert got is out
        guard_intact(buf, out)
        c = d.double() * scale
        # the lse is given in 32 bits: its rounding shifts every probability of the row
        ref.assert_grad(out, ref.target_grad(lp, norm, t, live, c), lp.exp(), c, t, what="grad",
                        extra=2.0 ** -23 * float(norm.abs().max()))


@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_logprob_extremes(dtype):
    """Masked entries (-inf, the type's lowest value), rows of nothing else, a
    masked target, NaN in ignored rows and in columns beyond the row."""
    low = torch.finfo(dtype).min
    for length in (5, 700, 5001, 40000):
        x, _ = logits(12, length, dtype, length, pad=2)
        t = torch.randint(0, length, (12,), generator=gen(1))
        x[0, length // 2:] = -math.inf
        t[0] = 1
        x[1, :length - 1] = -math.inf     # one entry left
        t[1] = length - 1
        x[2] = -math.inf                  # none left
        x[3, :] = low                     # an additive mask over everything: uniform
        x[4, 2:] = low
        t[4] = 0
        x[5, 1] = -math.inf               # the target itself is masked
        t[5] = 1
        x[6] = math.nan                   # ignored
        t[6] = -100
        x[7, length - 1] = math.nan       # taking part
        t[7] = 0
        x[8, 0] = math.inf
        t[8] = 1
        x[9] = 0.0
        x[10, 0] = -low                   # the largest value against the lowest
        x[10, 1:] = low
        t[10] = 0
        x[11, ::2] = -math.inf
        t[11] = 1
        logp, lse = itr.red_logprob(x, t.to(DEV))
        lp, norm = ref.log_softmax(x, 1.0)
        want, live = ref.taken(lp, t)
        norm = torch.where(live, norm, torch.zeros_like(norm))
        want[8] = norm[8] = math.nan
        assert logp[2].item() == lse[2].item() == -math.inf
        ref.assert_logp(logp[:8], want[:8])
        assert math.isnan(logp[8].item())
        ref.assert_logp(logp[9:], want[9:])
        finite = torch.tensor([0, 1, 4, 5, 6, 9, 10, 11])
        ref.assert_logp(lse.cpu()[finite], norm[finite], "lse")
        d = torch.linspace(-1, 1, 12) + 0.01
        got = itr.red_logprob_grad(x, t.to(DEV), lse, d.to(DEV)).cpu()
        # where the normaliser is of the order of the lowest value, fp32 has no room for its log count
        rows = torch.tensor([0, 1, 2, 4, 5, 6, 9, 10, 11])
        c = d.double()
        g = ref.target_grad(lp, norm, t, live, c)
        ref.assert_grad(got[rows], g[rows], lp.exp()[rows], c[rows], t[rows],
                        extra=2.0 ** -23 * float(norm[finite][:7].abs().max()) if dtype == torch.float16 else 4e-6)
        assert bool((got[2] == 0).all()) and bool((got[6] == 0).all())
        assert bool(got[7].isnan().all())


@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("length", [40, 700, 3000, 5001, 9000, 40000])
@pytest.mark.parametrize("copies", [1, 60, 200])
def test_extremes_by_every_mapping(dtype, length, copies):
    """The extreme rows once more, among few rows and among many (other
    kernels), through every loss: masked entries, the type's lowest value in
    part of a row and throughout, a lone entry, NaN and infinity."""
    if length * copies > 2_100_000:
        pytest.skip("as large as needed")
    low = torch.finfo(dtype).min
    kinds = 9
    rows = kinds * copies
    x, _ = logits(rows, length, dtype, length + copies, pad=3)
    t = torch.full((rows,), 1)
    one = torch.zeros(rows, dtype=torch.bool)
    one[::copies] = True
    k = torch.arange(rows) // copies
    x[k == 0, length // 2:] = -math.inf
    x[k == 1, :length - 2] = -math.inf
    t[k == 1] = length - 1
    x[k == 2] = -math.inf               # nothing left
    x[k == 3] = low                     # uniform
    x[k == 4, 2:] = low
    x[k == 5, :length - 2] = low        # a prefix far below the rest
    t[k == 5] = length - 2
    x[k == 6, length - 1] = math.nan
    x[k == 7, length // 2] = math.inf
    x[k == 8] = -low                    # uniform at the other end
    lp, norm = ref.log_softmax(x, 1.0)
    want, live = ref.taken(lp, t)
    sane = (k != 6) & (k != 7)
    logp, lse = itr.red_logprob(x, t.to(DEV))
    ref.assert_logp(logp[sane.to(DEV)], want[sane], "logp")
    assert bool(logp.cpu()[~sane].isnan().all())
    old = torch.where(want.isfinite(), want, torch.zeros_like(want)).float()
    ones = torch.ones(rows)
    loss, got, stats, grad = itr.red_policy(x, t.to(DEV), old.to(DEV), -ones.to(DEV))
    ref.assert_logp(got[sane.to(DEV)], want[sane], "policy logp")
    assert bool((loss.cpu()[k == 2] == 0).all()) and bool((grad[(k == 2).to(DEV)] == 0).all())
    assert bool(grad[(~sane).to(DEV)].isnan().all()) and bool(loss.cpu()[~sane].isnan().all())
    on = sane & (k != 2)
    # the ratio is 1 up to the rounding of old and the error of logp; -min(r A, ...) falls with logp for A = -1
    c = torch.ones(rows, dtype=torch.float64)
    g = ref.target_grad(lp, norm, t, live, c)
    p = lp.exp()
    ref.assert_grad(grad.cpu()[on], g[on], p[on], c[on], t[on], extra=3e-5, what="policy")
    ids = torch.tensor([[1, 2 % length, length - 1]]).repeat(rows, 1)
    vals = torch.zeros((rows, 3))
    loss, stats, grad = itr.red_distill(x, ids.to(DEV), vals.to(DEV))
    assert bool((grad[(k == 2).to(DEV)] == 0).all()) and bool((loss.cpu()[k == 2] == 0).all())
    assert bool(grad[(~sane).to(DEV)].isnan().all())
    q = torch.full((rows, 3), 1 / 3, dtype=torch.float64)
    mass = torch.zeros_like(p).scatter_add_(1, ids, q)
    ref.assert_grad(grad.cpu()[on], (p - mass)[on], (p + mass)[on], c[on], extra=3e-5, what="distill")
    # the gradient from lse, where fp32 has room for it beside the row's logits
    near = on & (k != 3) & (k != 8)
    got = itr.red_logprob_grad(x, t.to(DEV), lse, ones.to(DEV))
    ref.assert_grad(got.cpu()[near], g[near], p[near], c[near], t[near],
                    extra=2.0 ** -23 * float(norm[near].abs().max()), what="grad")
    assert bool((got[(k == 2).to(DEV)] == 0).all())


def test_preference_with_a_token_ruled_out():
    """A rejected answer that the policy cannot give costs nothing; a chosen one
    costs everything."""
    for length in (50, 9000):
        x, _ = logits(4, length, torch.float32, 3)
        t = torch.tensor([1, 2, 3, 4], device=DEV)
        x[3, 4] = -math.inf
        off = torch.tensor([0, 1, 2, 3, 4], device=DEV)
        loss, seq, stats, grad = itr.red_preference(x, t, off)
        assert loss[1].item() == 0.0 and math.isfinite(loss[0].item()) and seq[3].item() == -math.inf
        assert bool((grad[1] == 0).all()) and bool((grad[3] == 0).all()) and bool((grad[0] != 0).any())
        swapped = torch.tensor([4, 3, 2, 1], device=DEV)
        loss = itr.red_preference(x.flip(0), swapped, off, grad=False)[0]
        assert loss[0].item() == math.inf


def policy_inputs(rows, logp, seed):
    g = gen(seed)
    old = logp.float() + torch.randn(rows, generator=g) * 0.3
    rf = logp.float() + torch.randn(rows, generator=g) * 0.4
    adv = torch.randn(rows, generator=g)
    w = torch.rand(rows, generator=g) + 0.1
    w[torch.rand(rows, generator=g) < 0.2] = 0.0
    return old, rf, adv, w


@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("rows,length", SHAPES)
def test_policy(rows, length, dtype):
    low, high = 0.2, 0.3
    for pad, shift, opad, oshift, scale, kl in ((0, 0, None, 0, 1.0, 0.0), (3, 1, 3, 1, 0.8, 0.1),
                                                 (64, 0, 5, 3, 1.25, 0.04)):
        x, _ = logits(rows, length, dtype, rows + length, pad, shift)
        t = targets(rows, length, rows)
        lp, norm = ref.log_softmax(x, scale)
        logp, live = ref.taken(lp, t)
        old, rf, adv, w = policy_inputs(rows, logp, rows)
        gs = 3.0
        buf = None
        out = None
        if opad is not None:
            out, buf = out_like(x, opad, oshift)
        loss, got_lp, stats, grad = itr.red_policy(x, t.to(DEV), old.to(DEV), adv.to(DEV), ref_logp=rf.to(DEV),
                                                   weight=w.to(DEV), clip_low=low, clip_high=high, kl_coef=kl,
                                                   scale=scale, grad_scale=gs, grad=out)
        if buf is not None:
            guard_intact(buf, out)
        live = live & (w != 0)
        lw = w.double() * live
        want, c, drift, clipped = ref.policy(logp, old.double(), rf.double(), adv.double(), lw, low, high, kl)
        # 1.2e-5 of logp's error enters through e^(logp - old) and e^(ref - logp)
        size = lw * ((logp - old.double()).exp() * adv.double().abs() +
                     (kl * (1 + (rf.double() - logp).exp()) if kl else 0.0))
        assert (loss.cpu().double() - want).abs().max() <= (3e-5 * size + 1e-12).max()
        assert bool((loss.cpu()[~live] == 0).all())
        ref.assert_logp(got_lp, torch.where(live, logp, torch.zeros_like(logp)))
        tot = stats.cpu().double()
        assert abs(tot[0] - want.sum()) <= 3e-5 * size.sum() + 1e-9
        assert abs(tot[1] - (drift * lw).sum()) <= 3e-5 * (lw * (1 + (rf.double() - logp).exp())).sum() + 1e-9
        assert abs(tot[2] - (clipped * lw).sum()) <= 1e-6 * lw.sum() + 1e-9
        assert abs(tot[3] - lw.sum()) <= 1e-6 * lw.sum()
        ref.assert_grad(grad, ref.target_grad(lp, norm, t, live, c * gs * scale), lp.exp(), size * gs * scale, t,
                        extra=3e-5, what="grad")
        lone = itr.red_policy(x, t.to(DEV), old.to(DEV), adv.to(DEV), ref_logp=rf.to(DEV), weight=w.to(DEV),
                              clip_low=low, clip_high=high, kl_coef=kl, scale=scale, grad=False)
        assert lone[3] is None and torch.equal(lone[0], loss) and torch.equal(lone[2], stats)


def test_policy_extremes():
    """Empty and masked rows, NaN where nothing takes part, ratios that overflow."""
    rows, length = 9, 300
    x, _ = logits(rows, length, torch.float32, 5, pad=4)
    t = torch.arange(rows)
    old, adv = torch.full((rows,), -5.0), torch.ones(rows)
    w = torch.ones(rows)
    x[0] = -math.inf                      # nothing left
    x[1] = math.nan
    w[1] = 0.0
    x[2] = math.nan
    t[2] = -100
    x[3, 3] = -math.inf                   # the taken token is masked: ratio 0
    old[4], adv[4] = -1000.0, 0.0         # an infinite ratio of no advantage
    old[5], adv[5] = -1000.0, 1.0         # an infinite ratio, clipped
    old[1] = adv[1] = math.nan
    old[2] = adv[2] = math.nan
    adv[6] = -1.0
    loss, logp, stats, grad = itr.red_policy(x, t.to(DEV), old.to(DEV), adv.to(DEV), weight=w.to(DEV))
    for v in (loss, stats, grad):
        assert bool(v.isfinite().all())
    assert logp[0].item() == logp[3].item() == -math.inf
    for r in (0, 1, 2, 3, 4, 5):
        assert bool((grad[r] == 0).all()), r
    assert loss[0] == 0 and loss[1] == 0 and loss[2] == 0 and loss[3] == 0 and loss[4] == 0
    assert abs(loss[5].item() + 1.2) < 1e-6
    assert stats[3].item() == 7.0


def distill_reference(x, ids, vals, lse, w, scale, gs):
    lp, norm = ref.log_softmax(x, scale)
    rows, length = x.shape
    kept = (ids >= 0) & (ids < length)
    v = torch.where(kept, vals.double() * scale, torch.full(ids.shape, -math.inf, dtype=torch.float64))
    if lse is None:
        logq = torch.log_softmax(v, 1)
        mass = (v > -math.inf).any(1, keepdim=True)
        logq = torch.where(mass, logq, torch.full_like(logq, -math.inf))
    else:
        logq = v - lse.double()[:, None]
    q = torch.where(kept, logq.exp(), torch.zeros_like(logq))
    at = torch.where(kept, ids, torch.zeros_like(ids))
    term = torch.where(q > 0, q * (logq - lp.gather(1, at)), torch.zeros_like(q))
    size = torch.where(q > 0, q * (logq.abs() + lp.gather(1, at).abs() + 30), torch.zeros_like(q)).sum(1)
    g = lp.exp() * q.sum(1, keepdim=True)
    g.scatter_add_(1, at, -q)
    c = w.double() * gs * scale
    on = ((w != 0) & ~torch.isinf(norm))
    zero = torch.zeros((), dtype=torch.float64)
    loss = torch.where(on, term.sum(1) * w.double(), zero)
    size = torch.where(on, size * w.double().abs(), zero)
    mass = torch.zeros_like(g).scatter_add_(1, at, q)
    return loss, size, torch.where(on[:, None], g * c[:, None], zero), c, lp.exp() * q.sum(1, keepdim=True) + mass


def check_distill(x, ids, vals, lse, w, scale, gs, grad=None):
    buf = None
    if grad is not None:
        grad, buf = grad
    loss, stats, got = itr.red_distill(x, ids.to(DEV), vals.to(DEV), lse=None if lse is None else lse.to(DEV),
                                       weight=w.to(DEV), scale=scale, grad_scale=gs, grad=grad)
    if buf is not None:
        guard_intact(buf, grad)
    want, size, g, c, mass = distill_reference(x, ids, vals, lse, w, scale, gs)
    # logq and logp are off by 1.2e-5 absolute and 4e-7 relative each, q by 3e-5 relative
    assert bool(((loss.cpu().double() - want).abs() <= 4e-5 * size + 1e-9).all())
    assert abs(stats[0].item() - want.sum().item()) <= 4e-5 * size.sum().item() + 1e-9
    assert abs(stats[1].item() - w.double().sum().item()) <= 1e-6 * w.double().abs().sum().item() + 1e-9
    ref.assert_grad(got, g, mass, c, extra=3e-5)
    lone = itr.red_distill(x, ids.to(DEV), vals.to(DEV), lse=None if lse is None else lse.to(DEV), weight=w.to(DEV),
                           scale=scale, grad=False)
    assert lone[2] is None and torch.equal(lone[0], loss)


@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("rows,length", SHAPES)
def test_distill(rows, length, dtype):
    g = gen(rows * 7 + length)
    for n, (pad, shift, opad, oshift, scale, k) in enumerate(((0, 0, 0, 0, 1.0, 64), (3, 1, 3, 1, 0.5, 20),
                                                              (64, 0, 5, 3, 1.25, 130))):
        x, _ = logits(rows, length, dtype, rows + length, pad, shift)
        k = min(k, length)
        teacher = x.cpu().float() + torch.randn((rows, length), generator=g)
        top = torch.topk(teacher, k, 1)
        ids, vals = top.indices.clone(), top.values.to(ref.DTYPES[(n + rows) % 3])
        lse = torch.logsumexp(teacher.double() * scale, 1).float() if n != 1 else None
        ids[::3, (k + 1) // 2:] = -1
        w = torch.rand(rows, generator=g)
        w[1::5] = 0.0
        check_distill(x, ids, vals, lse, w, scale, 2.0, out_like(x, opad, oshift))


@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 100, 257, 1000, 1024])
def test_distill_entries(k):
    """Entries per row: ids that come twice, ids out of range, rows without
    any, a teacher's -inf, the row's first and last columns."""
    rows, length = 7, 1031
    g = gen(k)
    x, _ = logits(rows, length, torch.float32, k)
    ids = torch.stack([torch.randperm(length, generator=g)[:k] for _ in range(rows)])
    vals = torch.randn((rows, k), generator=g) * 2
    ids[0, 0], ids[0, -1] = 0, length - 1
    ids[1] = ids[1, 0]                    # one id k times
    ids[2, ::2] = ids[2, 0]
    ids[3, : k // 2] = length             # out of range
    ids[4] = -1                           # no entry at all
    vals[5, k // 2] = -math.inf           # an entry of no mass
    x[6, ids[6, k - 1]] = 4.0
    w = torch.ones(rows)
    check_distill(x, ids, vals, None, w, 1.0, 1.0)
    check_distill(x, ids, vals, torch.full((rows,), 9.0), w, 0.5, 1.0)


def test_distill_extremes():
    rows, length, k = 6, 2000, 8
    for dtype in ref.DTYPES:
        x, _ = logits(rows, length, dtype, 3, pad=1)
        ids = torch.arange(k).repeat(rows, 1) * 7
        vals = torch.randn((rows, k), generator=gen(1))
        w = torch.ones(rows)
        x[0] = -math.inf                  # nothing left
        x[1] = math.nan
        w[1] = 0.0
        vals[1] = math.nan
        x[2, 100:] = -math.inf            # masked entries beside the teacher's
        x[3, 0] = -math.inf               # the teacher has mass where the student has none
        x[4, 60:] = torch.finfo(dtype).min
        x[5, 1999] = math.nan
        loss, stats, grad = itr.red_distill(x, ids.to(DEV), vals.to(DEV), weight=w.to(DEV))
        assert loss[0] == 0 and loss[1] == 0 and loss[3].item() == math.inf
        assert bool((grad[:2] == 0).all()) and bool(grad[3].isfinite().all())
        assert math.isnan(loss[5].item()) and bool(grad[5].isnan().all())
        check_distill(x[2:3], ids[2:3], vals[2:3], None, w[2:3], 1.0, 1.0)
        check_distill(x[4:5], ids[4:5], vals[4:5], None, w[4:5], 1.0, 1.0)


def preference_reference(x, t, offsets, rf, w, kind, beta, margin, eps, average, scale, gs):
    lp, norm = ref.log_softmax(x, scale)
    logp, live = ref.taken(lp, t)
    live = live & ~(torch.isinf(norm) & (norm < 0))
    pairs = offsets.numel() // 2
    sums, counts = torch.zeros(2 * pairs, dtype=torch.float64), torch.ones(2 * pairs, dtype=torch.float64)
    rows_of = []
    for q in range(2 * pairs):
        lo, hi = int(offsets[q]), int(offsets[q + 1])
        idx = torch.arange(lo, hi)[live[lo:hi]]
        rows_of.append(idx)
        if average:
            counts[q] = max(1, idx.numel())
        sums[q] = logp[idx].sum() / counts[q]
    gain = sums - (rf.double() if rf is not None else 0.0)
    u = beta * (gain[:pairs] - gain[pairs:]) - margin
    loss, du = ref.pair_loss(u, kind, beta, eps)
    wd = w.double()
    c = torch.zeros(x.shape[0], dtype=torch.float64)
    for q in range(2 * pairs):
        sign = 1.0 if q < pairs else -1.0
        c[rows_of[q]] = sign * du[q % pairs] * wd[q % pairs] * beta * gs * scale / counts[q]
    member = torch.zeros(x.shape[0], dtype=torch.bool)
    for idx in rows_of:
        member[idx] = True
    # the sums' errors: 1.2e-5 and 4e-7 |logp| per token
    slack = torch.stack([(1.2e-5 + 4e-7 * logp[idx].abs()).sum() / counts[q] if idx.numel() else torch.zeros(()).double()
                         for q, idx in enumerate(rows_of)]) if pairs else torch.zeros(0).double()
    return lp, norm, sums, slack, u, loss * wd, du, member, c


@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("rows,length,pairs", [(2, 5, 1), (40, 33, 3), (300, 1024, 5), (64, 4099, 8), (31, 20001, 1),
                                               (900, 257, 200)])
def test_preference(rows, length, pairs, average, kind, dtype):
    g = gen(rows + pairs)
    x, _ = logits(rows, length, dtype, rows, pad=rows % 3, shift=rows % 2)
    t = targets(rows, length, rows, 0.3)
    inner = torch.randint(0, rows + 1, (2 * pairs - 1,), generator=g).sort().values
    first, last = (0, rows) if pairs == 1 else (min(1, int(inner[0])), max(rows - 2, int(inner[-1])))
    offsets = torch.cat([torch.tensor([first]), inner, torch.tensor([last])])
    beta, margin, eps, scale, gs = (0.5, 0.1, 0.1 if kind == "sigmoid" else 0.0, 0.9, 2.0)
    w = torch.rand(pairs, generator=g) + 0.05
    rf = None
    if rows % 2 == 0:
        rf = torch.randn(2 * pairs, generator=g) * 3 - 5
    out, buf = out_like(x, 1, 1)
    loss, seq, stats, grad = itr.red_preference(
        x, t.to(DEV), offsets.to(DEV), ref_logp=None if rf is None else rf.to(DEV), weight=w.to(DEV), kind=kind,
        beta=beta, margin=margin, smoothing=eps, average=average, scale=scale, grad_scale=gs, grad=out)
    guard_intact(buf, out)
    lp, norm, sums, slack, u, want, du, member, c = preference_reference(
        x, t, offsets, rf, w, kind, beta, margin, eps, average, scale, gs)
    assert bool(((seq.cpu().double() - sums).abs() <= slack + 2e-7 * sums.abs()).all())
    du_u = beta * (slack[:pairs] + slack[pairs:]) + 2e-7 * u.abs() + 1e-7   # error of u
    slope = du.abs() + (du_u * 2 / beta ** 2 if kind == "squared" else du_u)
    tol = w.double() * du_u * (slope + 1e-6) + 4e-6 * want.abs() + 1e-9
    assert bool(((loss.cpu().double() - want).abs() <= tol).all())
    tot = stats.cpu().double()
    assert abs(tot[0] - want.sum()) <= tol.sum() + 1e-6
    assert abs(tot[1] - (w.double() * u).sum()) <= (w.double() * du_u).sum() + 1e-6
    assert abs(tot[2] - (w.double() * (u > 0)).sum()) <= 1e-5
    assert abs(tot[3] - w.double().sum()) <= 1e-5
    # the coefficient moves with u by the loss's curvature: at most 1/4, 0 and 2 / beta^2
    curve = {"sigmoid": 0.25, "hinge": 0.0, "squared": 2.0 / beta ** 2}[kind]
    rel = 3e-5 + float((curve * du_u / du.abs().clamp(min=1e-3)).max())
    size = c.abs() * (1 + 1e-3 / max(1e-9, float(du.abs().min()) if float(du.abs().min()) > 0 else 1.0))
    ref.assert_grad(grad, ref.target_grad(lp, norm, t, member, c), lp.exp(), size, t, extra=rel)


def test_preference_edges():
    """No pairs, empty sequences, sequences without a live token, rows of -inf."""
    x, _ = logits(10, 50, torch.float32, 1)
    t = torch.randint(0, 50, (10,), generator=gen(2)).to(DEV)
    loss, seq, stats, grad = itr.red_preference(x, t, torch.zeros(1, dtype=torch.int64, device=DEV))
    assert loss.numel() == 0 and bool((stats == 0).all()) and bool((grad == 0).all())
    off = torch.zeros(5, dtype=torch.int64, device=DEV)
    loss, seq, stats, grad = itr.red_preference(x, t, off)
    assert bool((seq == 0).all()) and bool((grad == 0).all())
    assert torch.allclose(loss.cpu(), torch.full((2,), math.log(2.0)), atol=1e-6)
    x[3] = -math.inf
    t[4] = -100
    off = torch.tensor([3, 5, 10], device=DEV)      # the chosen sequence holds nothing live
    loss, seq, stats, grad = itr.red_preference(x, t, off, average=True)
    assert seq[0].item() == 0.0 and bool(loss.isfinite().all()) and bool(grad.isfinite().all())
    assert bool((grad[:5] == 0).all()) and bool((grad[5:] != 0).any(1).all())
    empty = x[:0]
    loss, seq, stats, grad = itr.red_preference(empty, t[:0], torch.zeros(3, dtype=torch.int64, device=DEV))
    assert abs(loss.item() - math.log(2.0)) < 1e-6 and grad.shape == (0, 50)


# Pairs of one call and of the same call with more, empty pairs: other kernels
# sum them, each result within 1.5e-7 of its sums' sizes.
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("rows,length", [(60, 5003), (25, 33000), (200, 300)])
def test_preference_pairs_by_either_kernel(rows, length, average):
    pairs, more = 6, 40
    x, _ = logits(rows, length, torch.bfloat16, 3, pad=5)
    t = targets(rows, length, 4, 0.2).to(DEV)
    t[rows // 3] = length                 # out of range
    x[rows // 2] = -math.inf
    off = torch.linspace(2, rows - 3, 2 * pairs + 1).long()
    off[3] = off[4]                       # an empty rejected sequence
    w = torch.tensor([1.0, 0.0, 0.5, 2.0, 1.0, 1.0])
    rf = torch.randn(2 * pairs, generator=gen(1)) * 3
    kw = dict(beta=0.3, margin=0.2, smoothing=0.1, average=average)
    a = itr.red_preference(x, t, off.to(DEV), ref_logp=rf.to(DEV), weight=w.to(DEV), **kw)
    # chosen sequences come first, then the rejected ones: the empty pairs go between and behind
    mid, end = off[pairs].repeat(more), off[-1].repeat(more)
    off2 = torch.cat([off[:pairs], mid, off[pairs:], end])
    pad = torch.zeros(more)
    b = itr.red_preference(x, t, off2.to(DEV), ref_logp=torch.cat([rf[:pairs], pad, rf[pairs:], pad]).to(DEV),
                           weight=torch.cat([w, pad]).to(DEV), **kw)
    size = float(a[1].abs().max()) + 10.0
    n = pairs + more
    assert (a[0] - b[0][:pairs]).abs().max() <= 1e-6 * size
    seq = torch.cat([b[1][:pairs], b[1][n:n + pairs]])
    assert (a[1] - seq).abs().max() <= 4e-7 * size
    assert (a[2] - b[2]).abs().max() <= 1e-5 * size
    assert bool((b[0][pairs:] == 0).all()) and bool(a[0][1] == 0)
    # c differs by du's 0.3 * 1e-6 * size, and bf16 by a rounding
    assert bool(((a[3].float() - b[3].float()).abs() <= 2.0 ** -7 * a[3].float().abs() + 1e-6 * size).all())
    dead = torch.zeros(rows, dtype=torch.bool)
    dead[:2], dead[-3:], dead[rows // 3], dead[rows // 2] = True, True, True, True
    dead |= (t.cpu() < 0)
    dead[int(off[1]):int(off[2])] = True  # chosen of the pair without weight
    assert bool((a[3].cpu()[dead] == 0).all()) and bool((b[3].cpu()[dead] == 0).all())


def test_no_rows():
    x = torch.empty((0, 40), device=DEV)
    none = torch.empty(0, device=DEV)
    t = torch.empty(0, dtype=torch.int64, device=DEV)
    logp, lse = itr.red_logprob(x, t)
    assert logp.numel() == 0 and itr.red_logprob_grad(x, t, lse, none).shape == (0, 40)
    _, _, stats, grad = itr.red_policy(x, t, none, none)
    assert bool((stats == 0).all()) and grad.shape == (0, 40)
    _, stats, grad = itr.red_distill(x, torch.empty((0, 3), dtype=torch.int64, device=DEV), torch.empty((0, 3), device=DEV))
    assert bool((stats == 0).all()) and grad.shape == (0, 40)


# Differences: rows hold the same logits with one moved by +-h.  The loss is
# off by 1.2e-5 (logp), so a quotient by 2h = 1/8 is off by 2e-4; the third
# derivative of log-softmax stays below 1/8, so h^2/6 of it is 1e-4.
H, DIFF = 0.0625, 4e-4


def moved(x):
    """(2 * n, n): the row x with entry j up by H, then down by H."""
    n = x.numel()
    eye = torch.eye(n) * H
    return torch.cat([x + eye, x - eye]).to(DEV)


def quotient(loss, n):
    return ((loss[:n] - loss[n:]) / (2 * H)).cpu().double()


def test_differences():
    n = 11
    g = gen(9)
    x = torch.randn(n, generator=g) * 1.5
    many = moved(x)
    y = torch.full((2 * n,), 4, device=DEV)
    logp, _ = itr.red_logprob(many, y)
    one = x[None].to(DEV)
    lp, lse = itr.red_logprob(one, y[:1])
    got = itr.red_logprob_grad(one, y[:1], lse, torch.ones(1, device=DEV))[0].cpu().double()
    assert (quotient(logp, n) - got).abs().max() < DIFF

    # policy, unclipped: the ratio stays within its bounds at every step; |dL/dlogp| < 2
    old, adv, rf = lp.cpu() - 0.02, torch.tensor([1.3]), lp.cpu() + 0.5
    kw = dict(kl_coef=0.2, clip_low=0.5, clip_high=0.5)
    rep = lambda v: v.expand(2 * n).contiguous().to(DEV)  # noqa: E731
    loss = itr.red_policy(many, y, rep(old), rep(adv), ref_logp=rep(rf), grad=False, **kw)[0]
    got = itr.red_policy(one, y[:1], old.to(DEV), adv.to(DEV), ref_logp=rf.to(DEV), **kw)[3][0].cpu().double()
    assert (quotient(loss, n) - got).abs().max() < 5 * DIFF

    ids, vals = torch.tensor([[1, 7, 4, 7]]), torch.randn((1, 4), generator=g)
    for lse_t in (None, torch.tensor([2.0])):
        args = (ids.expand(2 * n, 4).contiguous().to(DEV), vals.expand(2 * n, 4).contiguous().to(DEV))
        loss = itr.red_distill(many, *args, lse=None if lse_t is None else rep(lse_t), grad=False)[0]
        got = itr.red_distill(one, ids.to(DEV), vals.to(DEV), lse=None if lse_t is None else lse_t.to(DEV))[2][0]
        assert (quotient(loss, n) - got.cpu().double()).abs().max() < 2 * DIFF

    # preference: pair i's chosen sequence is the moved row, its rejected one the row itself
    flat = torch.cat([many, one.expand(2 * n, n)])
    tok = torch.cat([y, torch.full((2 * n,), 2, device=DEV)])
    off = torch.arange(4 * n + 1, device=DEV)
    for kind in ("sigmoid", "squared"):
        loss = itr.red_preference(flat, tok, off, kind=kind, beta=0.5, grad=False)[0]
        pair = torch.cat([one, one])
        got = itr.red_preference(pair, torch.tensor([4, 2], device=DEV), torch.arange(3, device=DEV), kind=kind,
                                 beta=0.5)[3][0].cpu().double()
        assert (quotient(loss, n) - got).abs().max() < 20 * DIFF * got.abs().max() + DIFF


@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("rows,length", [(3, 100), (200, 1000), (40, 9001), (3, 70001)])
def test_in_place_and_repeatable(rows, length, dtype):
    """A gradient in place of the logits equals one beside them, and the same
    call gives the same bits."""
    x, _ = logits(rows, length, dtype, 4, pad=3)
    t = targets(rows, length, 5).to(DEV)
    f = torch.randn(rows, generator=gen(6)).to(DEV)
    ids = torch.randint(0, length, (rows, 12), generator=gen(7)).to(DEV)
    vals = torch.randn((rows, 12), generator=gen(8)).to(DEV)
    off = torch.tensor([0, rows // 2, rows], device=DEV)
    calls = [
        lambda v, g: itr.red_policy(v, t, f - 5, f, grad=g),
        lambda v, g: itr.red_distill(v, ids, vals, grad=g),
        lambda v, g: itr.red_preference(v, t, off, grad=g),
        lambda v, g: (itr.red_logprob_grad(v, t, itr.red_logprob(v, t)[1], f, out=g),),
    ]
    for call in calls:
        first, again = call(x, None), call(x, None)
        for a, b in zip(first, again):
            assert torch.equal(a, b)
        spot = torch.empty((rows, x.stride(0)), dtype=dtype, device=DEV)[:, :length]
        spot.copy_(x)
        inplace = call(spot, spot)
        for a, b in zip(first[:-1], inplace[:-1]):
            assert torch.equal(a, b)
        assert torch.equal(first[-1], spot)


def test_side_stream_and_graph():
    rows, length = 64, 5003
    x, _ = logits(rows, length, torch.bfloat16, 4)
    t = targets(rows, length, 5).to(DEV)
    f = torch.randn(rows, generator=gen(6)).to(DEV)
    off = torch.tensor([0, 20, 64], device=DEV)
    want = [itr.red_policy(x, t, f - 5, f), itr.red_preference(x, t, off)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [itr.red_policy(x, t, f - 5, f, stream=side), itr.red_preference(x, t, off, stream=side)]
    side.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [itr.red_policy(x, t, f - 5, f), itr.red_preference(x, t, off)]
    for _ in range(2):
        for out in held:
            for v in out:
                v.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, held):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dtype,length", [(torch.float32, 200001), (torch.float32, 65536), (torch.bfloat16, 131072),
                                          (torch.float16, 50257), (torch.bfloat16, 20000), (torch.float32, 3001)])
def test_many_rows_per_cta(dtype, length):
    """Several rows per CTA at lengths that fit the kernel's shared memory
    several times, about once and not at all; live and ignored rows mixed."""
    rows = 1000 if length < 60000 else 480
    g = torch.Generator(device=DEV)
    g.manual_seed(length)
    x = (torch.randn((rows, length), generator=g, device=DEV) * 3).to(dtype)
    t = torch.randint(0, length, (rows,), generator=g, device=DEV)
    t[torch.rand(rows, generator=g, device=DEV) < 0.4] = -1
    old = torch.full((rows,), -10.0, device=DEV)
    adv = torch.randn(rows, generator=g, device=DEV)
    ids = torch.randint(0, length, (rows, 40), generator=g, device=DEV)
    vals = torch.randn((rows, 40), generator=g, device=DEV)
    w = torch.rand(rows, generator=g, device=DEV)
    w[::3] = 0.0
    logp, lse = itr.red_logprob(x, t)
    _, _, _, pgrad = itr.red_policy(x, t, old, adv, clip_high=1e4)
    _, _, dgrad = itr.red_distill(x, ids, vals, weight=w)
    for lo in range(0, rows, 40):
        part = slice(lo, lo + 40)
        z = x[part].double()
        norm = torch.logsumexp(z, 1)
        p = (z - norm[:, None]).exp()
        live = t[part] >= 0
        at = t[part].clamp(min=0)
        i = torch.arange(z.shape[0], device=DEV)
        want = torch.where(live, z[i, at] - norm, torch.zeros_like(norm))
        ref.assert_logp(logp[part], want, "logp")
        ref.assert_logp(lse[part], torch.where(live, norm, torch.zeros_like(norm)), "lse")
        free = (want + 10.0).exp() * adv[part].double()
        held = (want + 10.0).exp().clamp(0.8, 1e4 + 1) * adv[part].double()
        c = torch.where(live & (free <= held), -free, torch.zeros_like(free))
        grad = -p * c[:, None]
        grad[i, at] += c
        ref.assert_grad(pgrad[part], grad, p.cpu(), c.cpu(), at.cpu(), extra=3e-5, what="policy")
        q = torch.softmax(vals[part].double(), 1)
        mass = torch.zeros_like(p).scatter_add_(1, ids[part], q)
        wd = w[part].double()
        ref.assert_grad(dgrad[part], (p - mass) * wd[:, None], (p + mass).cpu(), wd.cpu(), extra=3e-5, what="distill")


@pytest.mark.parametrize("dtype,length,rows", [
    (torch.bfloat16, 300, 46000), (torch.float32, 201, 46000), (torch.float16, 901, 23500), (torch.float32, 700, 15600),
    (torch.bfloat16, 1300, 15600), (torch.bfloat16, 2001, 11700), (torch.float16, 2900, 7800),
    (torch.float32, 1999, 7800), (torch.bfloat16, 5500, 3900), (torch.bfloat16, 8001, 3900), (torch.float32, 4003, 3900),
    (torch.bfloat16, 150, 46000)])
def test_many_short_rows(dtype, length, rows):
    """More rows than run at once several times over, each length by another
    number of lanes and registers; rows of odd starts, masked, empty or ignored."""
    g = torch.Generator(device=DEV)
    g.manual_seed(length)
    x = (torch.randn((rows, length + 3), generator=g, device=DEV) * 3).to(dtype)[:, :length]
    r = torch.arange(rows, device=DEV)
    x[r % 50 == 3, length // 2:] = -math.inf
    x[r % 50 == 4] = -math.inf
    x[r % 50 == 5, :length - 1] = torch.finfo(dtype).min
    t = torch.randint(0, length // 2, (rows,), generator=g, device=DEV)
    t[r % 50 == 5] = length - 1
    t[torch.rand(rows, generator=g, device=DEV) < 0.3] = -1
    t[r == rows - 1] = 0
    old = torch.full((rows,), -8.0, device=DEV)
    adv = torch.randn(rows, generator=g, device=DEV)
    logp, lse = itr.red_logprob(x, t)
    loss, plogp, _, grad = itr.red_policy(x, t, old, adv, clip_high=1e6)
    some = torch.cat([r[:200], r[-200:], r[::61]])
    for part in some.split(100):
        y = t[part].cpu()
        p, norm = ref.log_softmax(x[part], 1.0)
        want, live = ref.taken(p, y)
        ref.assert_logp(logp[part], want, "logp")
        ref.assert_logp(plogp[part], want, "policy logp")
        ref.assert_logp(lse[part], torch.where(live, norm, torch.zeros_like(norm)), "lse")
        a = adv[part].cpu().double()
        ratio = (want + 8.0).exp()
        c = torch.where(live & (ratio * a <= ratio.clamp(min=0.8) * a), -ratio * a, torch.zeros_like(a))
        c[want == -math.inf] = 0.0
        ref.assert_grad(grad[part], ref.target_grad(p, norm, y, live, c), p.exp(), (ratio * a).abs(), y,
                        extra=3e-5, what="policy")


def test_offsets_past_32_bits():
    """Rows whose elements start beyond 2^32 in the logits and in the gradient."""
    length = 65536
    rows = (1 << 32) // length + 3
    x = torch.zeros((rows, length), dtype=torch.bfloat16, device=DEV)
    t = torch.full((rows,), -100, dtype=torch.int64, device=DEV)
    part = torch.randn((2, length), generator=gen(1)).to(torch.bfloat16)
    x[-2:] = part.to(DEV)
    t[-2:] = torch.tensor([5, 65535], device=DEV)
    lp, norm = ref.log_softmax(part, 1.0)
    tt = torch.tensor([5, 65535])
    want, live = ref.taken(lp, tt)
    logp, lse = itr.red_logprob(x, t)
    ref.assert_logp(logp[-2:], want)
    assert bool((logp[:-2] == 0).all())
    c = torch.tensor([1.0, -2.0])
    d = torch.zeros(rows, device=DEV)
    d[-2:] = c.to(DEV)
    itr.red_logprob_grad(x, t, lse, d, out=x)
    ref.assert_grad(x[-2:], ref.target_grad(lp, norm, tt, live, c.double()), lp.exp(), c.double(), tt, extra=4e-6)
    x[-2:] = part.to(DEV)
    f = torch.full((rows,), -11.0, device=DEV)
    loss, got, stats, grad = itr.red_policy(x, t, f, torch.ones_like(f), clip_high=1e3, grad=x)
    r = (want - -11.0).exp()
    ref.assert_grad(x[-2:], ref.target_grad(lp, norm, tt, live, -r), lp.exp(), r, tt, extra=3e-5)


def test_binding_checks():
    x, _ = logits(4, 9, torch.float32, 1)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    f = torch.zeros(4, device=DEV)
    with pytest.raises(ValueError):
        itr.red_logprob(x.double(), t)
    with pytest.raises(ValueError):
        itr.red_logprob(x, t.int())
    with pytest.raises(ValueError):
        itr.red_logprob(x, t[:3])
    with pytest.raises(ValueError):
        itr.red_logprob(x.t(), torch.zeros(9, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        itr.red_policy(x, t, f, f, grad=torch.empty((4, 9), dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError):
        itr.red_policy(x, t, f.cpu(), f)
    with pytest.raises(ValueError):
        itr.red_distill(x, t[:, None], f)
    with pytest.raises(ValueError):
        itr.red_preference(x, t, torch.zeros(4, dtype=torch.int64, device=DEV))
    with pytest.raises(itr.RedError):
        itr.red_policy(x, t, f, f, kl_coef=0.1)
    with pytest.raises(itr.RedError):
        itr.red_logprob(x, t, scale=0.0)
