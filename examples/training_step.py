"""One training step of a small language model with the operators around its
end, forward and backward, on one GPU.

A residual stream of token embeddings, a norm, a layer with a router beside it,
the norm of the sum, and the vocabulary's likelihood without the logits:

    n1          = rmsnorm(stream)                      red_rmsnorm
    router      = n1 R, two experts per token          red_balance: counts, loss, gradient
    delta       = n1 M
    n2, total   = rmsnorm(delta + stream)              red_rmsnorm with the residual
    logp, lse   = log-probabilities of the targets     red_linear_logprob
    loss        = mean(-logp + z lse^2) + balance loss

and back through red_linear_logprob_grad and red_rmsnorm_grad, whose `dtotal`
takes the gradient that reaches the stream around the layer.  The plain matrix
products are torch's.  Run: python examples/training_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int_tensor_reductions_gb300 as itr  # noqa: E402

VOCAB, WIDTH, EXPERTS, CHOSEN = 5003, 256, 16, 2
BALANCE, ROUTER_Z, Z = 0.01, 1e-3, 1e-4


class Model:
    def __init__(self, seed, device):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def randn(*shape, width):
            return torch.randn(shape, generator=gen, device=device) * width

        self.embed = randn(VOCAB, WIDTH, width=1.0).bfloat16()
        self.params = {
            "g1": 1.0 + randn(WIDTH, width=0.1),
            "router": randn(WIDTH, EXPERTS, width=WIDTH ** -0.5),
            "layer": randn(WIDTH, WIDTH, width=WIDTH ** -0.5).bfloat16(),
            "g2": 1.0 + randn(WIDTH, width=0.1),
            "head": randn(VOCAB, WIDTH, width=1.5 * WIDTH ** -0.5).bfloat16(),
        }


def step(model, tokens, target):
    """(losses, gradients, the experts that were chosen); a target of -100 is no part of the loss."""
    p = model.params
    live = target >= 0
    mean = 1.0 / max(1, int(live.sum()))

    stream = model.embed[tokens]
    n1, _, r1 = itr.red_rmsnorm(stream, p["g1"])
    router = n1.float() @ p["router"]
    ids = torch.topk(router, CHOSEN, 1).indices
    counts, _, stats, d_router = itr.red_balance(router, ids, live=live, coef=BALANCE, z_coef=ROUTER_Z)
    delta = n1 @ p["layer"]
    n2, total, r2 = itr.red_rmsnorm(delta, p["g2"], residual=stream)
    logp, lse = itr.red_linear_logprob(n2, p["head"], target)

    d_logp = torch.full_like(logp, -mean)
    d_n2, d_head = itr.red_linear_logprob_grad(n2, p["head"], target, lse, d_logp, dlse=lse * (2.0 * Z * mean))
    d_total, d_g2 = itr.red_rmsnorm_grad(d_n2, total, r2, p["g2"])       # of delta and of the stream
    d_n1 = (d_total @ p["layer"].t()).float() + d_router @ p["router"].t()
    d_stream, d_g1 = itr.red_rmsnorm_grad(d_n1.bfloat16(), stream, r1, p["g1"], dtotal=d_total)
    grads = {"g1": d_g1, "router": n1.float().t() @ d_router, "layer": n1.t() @ d_total, "g2": d_g2, "head": d_head,
             "stream": d_stream}
    likelihood = itr.red_full("sum", logp) * mean
    normaliser = itr.red_full("sum", lse * lse) * mean
    losses = torch.cat([-likelihood, normaliser, stats[:1], counts.max().float()[None]])
    return losses, grads, ids


def main(steps=30, rows=2000, rate=0.3):
    device = torch.device("cuda")
    model = Model(3, device)
    gen = torch.Generator(device=device)
    gen.manual_seed(5)
    tokens = torch.randint(0, VOCAB, (rows,), generator=gen, device=device)
    target = (tokens * 7 + 3) % VOCAB
    target[torch.rand(rows, generator=gen, device=device) < 0.2] = -100
    history = []
    for _ in range(steps):
        losses, grads, _ = step(model, tokens, target)
        for name, value in model.params.items():
            value -= (rate * grads[name].float() * (20.0 if name == "head" else 1.0)).to(value.dtype)
        history.append(losses)
    history = torch.stack(history).tolist()
    print(f"-log p {history[0][0]:.3f} -> {history[-1][0]:.3f}, mean lse^2 {history[0][1]:.1f} -> {history[-1][1]:.1f}, "
          f"router's loss {history[0][2]:.4f} -> {history[-1][2]:.4f}, most tokens of one expert "
          f"{history[0][3]:.0f} -> {history[-1][3]:.0f}")
    return history


if __name__ == "__main__":
    main()
