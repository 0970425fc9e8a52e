"""The root-mean-square norm and the balance loss refuse bad arguments on the
host, before any CUDA call."""
import math

import pytest

X, R, W, Y, T, F, I, Q = (0x10000 * i for i in range(1, 9))


@pytest.fixture(scope="module")
def itr():
    from int_tensor_reductions_gb300 import _build
    import int_tensor_reductions_gb300 as itr
    _build.build_lib()
    return itr


def norm(itr, dtype=3, x=X, rows=4, length=16, ldx=16, res=R, ldr=16, wtype=3, w=W, eps=1e-6, y=Y, ldy=16, total=T,
         ldt=16, rstd=F):
    return itr.lib().red_rmsnorm(dtype, x, rows, length, ldx, res, ldr, wtype, w, eps, y, ldy, total, ldt, rstd, None)


def quant(itr, dtype=3, x=X, rows=4, length=16, ldx=16, res=R, ldr=16, wtype=3, w=W, eps=1e-6, kind=1, block=0, y=Y,
          ldy=16, scales=Q, total=T, ldt=16, rstd=F):
    return itr.lib().red_rmsnorm_quant(dtype, x, rows, length, ldx, res, ldr, wtype, w, eps, kind, block, y, ldy, scales,
                                       total, ldt, rstd, None)


def grad(itr, dtype=3, dy=Y, lddy=16, x=X, rows=4, length=16, ldx=16, rstd=F, wtype=3, w=W, dt=T, ldt=16, dx=R, ldd=16,
         dw=Q):
    return itr.lib().red_rmsnorm_grad(dtype, dy, lddy, x, rows, length, ldx, rstd, wtype, w, dt, ldt, dx, ldd, dw, None)


def balance(itr, dtype=3, x=X, rows=4, experts=16, ld=16, ids=I, k=2, live=None, kind=0, coef=1.0, z=0.0, gs=1.0,
            counts=Q, prob=F, stats=T, dx=Y, ldd=16):
    return itr.lib().red_balance(dtype, x, rows, experts, ld, ids, k, live, kind, coef, z, gs, counts, prob, stats, dx,
                                 ldd, None)


@pytest.mark.parametrize("call", [norm, quant, grad])
@pytest.mark.parametrize("bad", [dict(dtype=1), dict(dtype=-1), dict(rows=-1), dict(rows=1 << 40), dict(length=0),
                                 dict(length=16385, ldx=16385), dict(wtype=2), dict(wtype=1), dict(w=W + 1), dict(x=None),
                                 dict(x=X + 1), dict(ldx=15), dict(ldx=1 << 45), dict(rstd=F + 2)])
def test_shared_refusals(itr, call, bad):
    assert call(itr, **bad) == itr.RED_EINVAL
    assert "rmsnorm" in itr.red_last_error()


@pytest.mark.parametrize("call,bad", [
    (call, bad) for call in (norm, quant) for bad in
    (dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(y=None), dict(ldy=15), dict(res=None), dict(total=None),
     dict(res=R + 1), dict(total=T + 1), dict(ldr=15), dict(ldt=15), dict(total=X, ldt=24), dict(total=Y))] + [
    (norm, dict(y=X, ldy=24)), (norm, dict(y=R, ldy=24)), (norm, dict(y=Y + 1)),
    (quant, dict(kind=0)), (quant, dict(kind=3)), (quant, dict(block=16)), (quant, dict(block=-32)),
    (quant, dict(block=256)), (quant, dict(scales=None)), (quant, dict(scales=Q + 2)), (quant, dict(y=X)),
    (grad, dict(dy=None)), (grad, dict(dx=None)), (grad, dict(lddy=15)), (grad, dict(ldd=15)), (grad, dict(ldt=15)),
    (grad, dict(dx=Y, ldd=24)), (grad, dict(dx=X, ldd=24)), (grad, dict(dx=T, ldd=24)), (grad, dict(rstd=None)),
    (grad, dict(dw=Q + 1)),
    (balance, dict(dtype=1)), (balance, dict(rows=-1)), (balance, dict(rows=1 << 30)), (balance, dict(experts=0)),
    (balance, dict(experts=4097, ld=4097, ldd=4097)), (balance, dict(k=0)), (balance, dict(k=17)), (balance, dict(ld=15)),
    (balance, dict(ldd=15)), (balance, dict(ids=None)), (balance, dict(ids=I + 4)), (balance, dict(kind=2)),
    (balance, dict(coef=math.inf)), (balance, dict(z=math.nan)), (balance, dict(gs=math.nan)),
    (balance, dict(kind=1, z=0.1)), (balance, dict(counts=None)), (balance, dict(counts=Q + 4)), (balance, dict(prob=None)),
    (balance, dict(stats=F + 2)), (balance, dict(x=None)), (balance, dict(x=X + 1)), (balance, dict(dx=X, ldd=24)),
    (balance, dict(dx=Y + 1))])
def test_own_refusals(itr, call, bad):
    assert call(itr, **bad) == itr.RED_EINVAL
    assert itr.red_last_error()


def test_nothing_to_do(itr):
    assert norm(itr, rows=0, x=None, res=None, y=None, total=None, rstd=None) == itr.RED_OK
    assert quant(itr, rows=0, x=None, res=None, y=None, total=None, rstd=None, scales=None) == itr.RED_OK
    assert grad(itr, rows=0, dy=None, x=None, dx=None, dt=None, rstd=None, dw=None) == itr.RED_OK


def test_binding_refuses_cpu_tensors(itr):
    import torch
    x, w, f = torch.zeros((2, 8)), torch.ones(8), torch.ones(2)
    ids = torch.zeros((2, 1), dtype=torch.int64)
    for call in (lambda: itr.red_rmsnorm(x, w), lambda: itr.red_rmsnorm_quant(x, w),
                 lambda: itr.red_rmsnorm_grad(x, x, f, w), lambda: itr.red_balance(x, ids)):
        with pytest.raises(ValueError):
            call()
