"""red_linear_logprob and its backward refuse bad arguments on the host, before
any CUDA call."""
import math

import pytest

P, W, I, F, S = 0x1000, 0x20000, 0x4000, 0x8000, 0x100000
BIG = 1 << 50


@pytest.fixture(scope="module")
def itr():
    from int_tensor_reductions_gb300 import _build
    import int_tensor_reductions_gb300 as itr
    _build.build_lib()
    return itr


def forward(itr, dtype=3, h=P, rows=4, dim=16, ldh=16, w=W, vocab=9, ldw=16, scale=1.0, target=I, logp=F, lse=F, work=S,
            size=BIG):
    return itr.lib().red_linear_logprob(dtype, h, rows, dim, ldh, w, vocab, ldw, scale, target, logp, lse, work, size,
                                        None)


def backward(itr, dtype=3, h=P, rows=4, dim=16, ldh=16, w=W, vocab=9, ldw=16, scale=1.0, target=I, lse=F, dlogp=F,
             dlse=None, dh=P + 64, ldd=16, dw=W + 64, lddw=16, work=S, size=BIG):
    return itr.lib().red_linear_logprob_grad(dtype, h, rows, dim, ldh, w, vocab, ldw, scale, target, lse, dlogp, dlse,
                                             dh, ldd, dw, lddw, work, size, None)


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("bad", [
    dict(dtype=0), dict(dtype=1), dict(dtype=-1), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(dim=0),
    dict(dim=(1 << 20) + 1, ldh=1 << 21, ldw=1 << 21), dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(rows=1 << 24, vocab=1 << 23), dict(scale=0.0),
    dict(scale=math.nan), dict(scale=math.inf), dict(h=None), dict(h=P + 8), dict(w=None), dict(w=W + 2), dict(ldh=8),
    dict(ldh=20), dict(ldw=15), dict(ldw=17), dict(ldw=1 << 40), dict(target=None), dict(target=I + 4), dict(lse=None),
    dict(lse=F + 2), dict(work=None), dict(work=S + 16), dict(size=0), dict(size=1000)])
def test_shared_refusals(itr, call, bad):
    assert call(itr, **bad) == itr.RED_EINVAL
    assert "linear" in itr.red_last_error()


@pytest.mark.parametrize("call,bad", [
    (forward, dict(logp=None)), (forward, dict(logp=F + 1)), (backward, dict(dlogp=None)), (backward, dict(dlogp=F + 2)),
    (backward, dict(dlse=F + 1)), (backward, dict(dh=None, dw=None)), (backward, dict(dh=P + 4)),
    (backward, dict(dw=W + 4)), (backward, dict(ldd=8)), (backward, dict(ldd=18)), (backward, dict(lddw=8)),
    (backward, dict(lddw=18)), (backward, dict(dw=W)), (backward, dict(dw=P)), (backward, dict(dh=W)),
    (backward, dict(dh=W + 64)), (backward, dict(dh=P, ldd=24))])
def test_own_refusals(itr, call, bad):
    assert call(itr, **bad) == itr.RED_EINVAL
    assert itr.red_last_error()


def test_nothing_to_do(itr):
    assert forward(itr, rows=0, h=None, target=None, logp=None, lse=None, work=None, size=0) == itr.RED_OK
    assert backward(itr, rows=0, h=None, target=None, lse=None, dlogp=None, dh=None, dw=None, work=None,
                    size=0) == itr.RED_OK


def test_scratch_sizes(itr):
    """The scratch grows with the rows and never with rows times vocabulary of a large call's gradients."""
    size = itr.lib().red_linear_work_bytes
    assert size(-1, 8, 8, 0) == size(1, 0, 8, 1) == size(1, 8, 0, 0) == itr.RED_EINVAL
    assert size(0, 8, 8, 0) == size(0, 8, 8, 1) == 0
    assert size(4, 64, 1000, 1) >= 256 * 64 * 2 + 16 * 1000 * 2
    assert size(400, 64, 1000, 1) >= 512 * 64 * 2 + 512 * 1000 * 2
    wide = size(8192, 4096, 131072, 1)
    assert wide == size(8192, 4096, 262144, 1) < 8192 * 131072 * 2


def test_binding_refuses_cpu_tensors(itr):
    import torch
    h, w = torch.zeros((2, 8), dtype=torch.float16), torch.zeros((5, 8), dtype=torch.float16)
    t, f = torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    for call in (lambda: itr.red_linear_logprob(h, w, t), lambda: itr.red_linear_logprob_grad(h, w, t, f, f)):
        with pytest.raises(ValueError):
            call()
