"""The losses over rows of logits refuse bad arguments on the host, before
any CUDA call."""
import math

import pytest

P, Q, I, F = 0x1000, 0x2000, 0x4000, 0x8000


@pytest.fixture(scope="module")
def itr():
    from int_tensor_reductions_gb300 import _build
    import int_tensor_reductions_gb300 as itr
    _build.build_lib()
    return itr


def logprob(itr, dtype=0, x=P, rows=4, length=8, ld=8, scale=1.0, target=I, logp=F, lse=Q):
    return itr.lib().red_logprob(dtype, x, rows, length, ld, scale, target, logp, lse, None)


def grad(itr, dtype=0, x=P, rows=4, length=8, ld=8, scale=1.0, target=I, lse=F, dlogp=F, dx=Q, ldd=8):
    return itr.lib().red_logprob_grad(dtype, x, rows, length, ld, scale, target, lse, dlogp, dx, ldd, None)


def distill(itr, dtype=0, x=P, rows=4, length=8, ld=8, scale=1.0, k=3, ids=I, vdtype=0, vals=F, lse=None, weight=None,
            gs=1.0, loss=F, stats=F, dx=Q, ldd=8):
    return itr.lib().red_distill(dtype, x, rows, length, ld, scale, k, ids, vdtype, vals, lse, weight, gs, loss,
                                 stats, dx, ldd, None)


def policy(itr, dtype=0, x=P, rows=4, length=8, ld=8, scale=1.0, target=I, old=F, rf=None, adv=F, weight=None, low=0.2,
           high=0.2, kl=0.0, gs=1.0, loss=F, logp=F, stats=F, dx=Q, ldd=8):
    return itr.lib().red_policy(dtype, x, rows, length, ld, scale, target, old, rf, adv, weight, low, high, kl, gs,
                                loss, logp, stats, dx, ldd, None)


def preference(itr, dtype=0, x=P, rows=4, length=8, ld=8, scale=1.0, target=I, offsets=I, pairs=1, rf=None, weight=None,
               kind=0, beta=0.1, margin=0.0, smoothing=0.0, average=0, gs=1.0, loss=F, seq=F, stats=F, work=F, dx=Q,
               ldd=8):
    return itr.lib().red_preference(dtype, x, rows, length, ld, scale, target, offsets, pairs, rf, weight, kind, beta,
                                    margin, smoothing, average, gs, loss, seq, stats, work, dx, ldd, None)


CALLS = [logprob, grad, distill, policy, preference]
SHARED = [dict(dtype=1), dict(dtype=4), dict(dtype=-1), dict(rows=-1), dict(length=0), dict(length=(1 << 30) + 1, ld=1 << 31),
          dict(ld=7), dict(rows=1 << 40, ld=1 << 20), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
          dict(scale=math.inf), dict(x=None), dict(x=P + 2), dict(dtype=3, x=P + 1)]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad", SHARED)
def test_shared_refusals(itr, call, bad):
    assert call(itr, **bad) == itr.RED_EINVAL
    assert call.__name__.split("_")[0] in itr.red_last_error() or "grad" in itr.red_last_error()


@pytest.mark.parametrize("call", CALLS[1:])
@pytest.mark.parametrize("bad", [dict(ldd=7), dict(dx=Q + 2), dict(dx=P, ldd=9), dict(rows=1 << 40, ldd=1 << 20)])
def test_gradient_refusals(itr, call, bad):
    assert call(itr, **bad) == itr.RED_EINVAL


@pytest.mark.parametrize("call,bad", [
    (logprob, dict(target=None)), (logprob, dict(target=I + 4)), (logprob, dict(logp=None)), (logprob, dict(lse=F + 2)),
    (grad, dict(dx=None)), (grad, dict(target=None)), (grad, dict(lse=None)), (grad, dict(dlogp=F + 1)),
    (distill, dict(k=0)), (distill, dict(k=1025)), (distill, dict(vdtype=1)), (distill, dict(ids=None)),
    (distill, dict(ids=I + 4)), (distill, dict(vals=None)), (distill, dict(vals=F + 2)), (distill, dict(lse=F + 2)),
    (distill, dict(weight=F + 1)), (distill, dict(loss=None)), (distill, dict(stats=None)),
    (distill, dict(gs=math.inf)),
    (policy, dict(low=-0.1)), (policy, dict(low=1.5)), (policy, dict(high=-0.1)), (policy, dict(high=math.nan)),
    (policy, dict(kl=0.1)), (policy, dict(kl=math.nan, rf=F)), (policy, dict(gs=math.nan)), (policy, dict(old=None)),
    (policy, dict(adv=None)), (policy, dict(rf=F + 2)), (policy, dict(weight=F + 2)), (policy, dict(loss=None)),
    (policy, dict(logp=None)), (policy, dict(stats=F + 1)), (policy, dict(target=None)),
    (preference, dict(pairs=-1)), (preference, dict(kind=3)), (preference, dict(kind=-1)), (preference, dict(beta=0.0)),
    (preference, dict(beta=math.inf)), (preference, dict(margin=math.nan)), (preference, dict(smoothing=0.6)),
    (preference, dict(smoothing=0.1, kind=1)), (preference, dict(gs=math.inf)), (preference, dict(stats=None)),
    (preference, dict(target=None)), (preference, dict(offsets=None)), (preference, dict(offsets=I + 4)),
    (preference, dict(rf=F + 2)), (preference, dict(weight=F + 2)), (preference, dict(loss=None)),
    (preference, dict(seq=None)), (preference, dict(work=None)),
])
def test_own_refusals(itr, call, bad):
    assert call(itr, **bad) == itr.RED_EINVAL
    assert itr.red_last_error()


def test_nothing_to_do(itr):
    assert logprob(itr, rows=0, x=None, target=None, logp=None, lse=None) == itr.RED_OK
    assert grad(itr, rows=0, x=None, target=None, lse=None, dlogp=None, dx=None) == itr.RED_OK


def test_binding_refuses_cpu_tensors(itr):
    import torch
    x, t, f = torch.zeros((2, 4)), torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    for call in (lambda: itr.red_logprob(x, t), lambda: itr.red_logprob_grad(x, t, f, f),
                 lambda: itr.red_policy(x, t, f, f), lambda: itr.red_distill(x, t[:, None], f[:, None]),
                 lambda: itr.red_preference(x, t, torch.tensor([0, 1, 2]))):
        with pytest.raises(ValueError):
            call()
