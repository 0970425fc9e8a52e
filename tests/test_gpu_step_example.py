"""examples/training_step.py runs, and its gradients are those of the whole step.

The chain rounds to bf16 (half a step is 2**-8 of a value) the stream's norms, the
layer's product and, on the way back, each gradient that is handed on: at most eight
roundings between the loss and a parameter, each of which moves a gradient's norm by no
more than 2**-8 of it in the mean (the maps between them are of condition about 1).  The
gradients are compared in the norm, with 8 * 2**-8.
"""
import importlib.util
import math
import os

import pytest
import torch

from conftest import ROOT
from gpu_util import lib_ready

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    lib_ready()
    path = os.path.join(ROOT, "examples", "training_step.py")
    spec = importlib.util.spec_from_file_location("training_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def definition(example, model, tokens, target, ids):
    """(losses, gradients) of the step in 64 bits, with the same experts chosen."""
    p = {k: v.double().requires_grad_() for k, v in model.params.items()}
    stream = model.embed[tokens].double().requires_grad_()
    live = target >= 0

    def norm(x, g):
        return x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * g

    n1 = norm(stream, p["g1"])
    router = (n1 @ p["router"])[live]
    prob = torch.softmax(router, 1)
    share = torch.bincount(ids[live].flatten(), minlength=example.EXPERTS).double() / ids[live].numel()
    balance = example.BALANCE * example.EXPERTS * (share * prob.mean(0)).sum()
    balance = balance + example.ROUTER_Z * torch.logsumexp(router, 1).square().mean()
    n2 = norm(n1 @ p["layer"] + stream, p["g2"])
    z = (n2 @ p["head"].t())[live]
    lse = torch.logsumexp(z, 1)
    likelihood = (lse - z.gather(1, target[live][:, None])[:, 0]).mean()
    normaliser = lse.square().mean()
    (likelihood + example.Z * normaliser + balance).backward()
    return (likelihood, normaliser, balance), {**{k: v.grad for k, v in p.items()}, "stream": stream.grad}


@pytest.mark.parametrize("rows", [3, 100, 700])
def test_gradients(example, rows):
    device = torch.device("cuda")
    model = example.Model(11, device)
    gen = torch.Generator(device=device)
    gen.manual_seed(rows)
    tokens = torch.randint(0, example.VOCAB, (rows,), generator=gen, device=device)
    target = torch.randint(0, example.VOCAB, (rows,), generator=gen, device=device)
    target[::3] = -100
    losses, grads, ids = example.step(model, tokens, target)
    want, exact = definition(example, model, tokens, target, ids)
    for got, w in zip(losses.tolist(), want):
        assert abs(got - w.item()) <= 8 * 2.0 ** -8 * abs(w.item())
    for name, w in exact.items():
        off = float((grads[name].double() - w).norm() / w.norm())
        assert off <= 8 * 2.0 ** -8, f"{name}: {off}"


def test_it_runs(example):
    history = example.main(steps=4)
    assert len(history) == 4 and all(math.isfinite(v) for row in history for v in row)
