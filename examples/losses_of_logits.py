"""The losses over logits as a training program uses them, on one GPU.

A toy language model (an embedding of the two previous tokens and a linear
head) goes through the stages that the operators are for:

1. distillation: its logits against a teacher's top 16 (red_distill);
2. preference: pairs of packed answers, scored by the distilled model kept as
   reference (red_logprob, red_rows_ragged), then trained on the pairs
   (red_preference);
3. policy: answers sampled from the model, rewarded for even tokens, with the
   clipped loss and a KL term towards the reference (red_policy), several
   steps per batch of samples;
4. and a custom loss on log-probabilities, with its gradient by hand
   (red_logprob, red_logprob_grad).

The gradient by the logits goes on through the head with plain matrix
products.  Run: python examples/losses_of_logits.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int_tensor_reductions_gb300 as itr  # noqa: E402

VOCAB, WIDTH, LENGTH = 1000, 128, 24


class Model:
    """Features of a position from its two previous tokens, and a head."""

    def __init__(self, seed, device):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        self.embed = torch.randn((2, VOCAB, WIDTH), generator=gen, device=device) * 0.7
        self.head = torch.randn((WIDTH, VOCAB), generator=gen, device=device) * 0.1

    def copy(self):
        new = object.__new__(Model)
        new.embed, new.head = self.embed, self.head.clone()
        return new

    def features(self, tokens):
        """(rows, WIDTH) for a batch of sequences (n, LENGTH)."""
        before = torch.nn.functional.pad(tokens, (2, 0))[:, :LENGTH + 1]
        h = self.embed[0][before[:, :-1]] + self.embed[1][before[:, 1:]]
        return torch.tanh(h).reshape(-1, WIDTH)

    def logits(self, h):
        return (h @ self.head).bfloat16()

    def step(self, h, grad, rate):
        """Descent along the gradient by the logits."""
        self.head -= rate * (h.t() @ grad.float())


def sequences(n, seed, device):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    return torch.randint(0, VOCAB, (n, LENGTH), generator=gen, device=device)


def distill(student, teacher, steps=120, seed=1):
    losses = []
    for i in range(steps):
        tokens = sequences(32, seed + i, student.head.device)
        h = student.features(tokens)
        top = torch.topk(teacher.logits(teacher.features(tokens)), 16, 1)
        weight = torch.full((h.shape[0],), 1.0 / h.shape[0], device=h.device)
        logits = student.logits(h)
        _, stats, grad = itr.red_distill(logits, top.indices, top.values, weight=weight, grad=logits)  # in place
        student.step(h, grad, 12.0)
        losses.append(stats[0])
    return torch.stack(losses).tolist()


def preference(model, steps=30, pairs=16, seed=500):
    """Chosen answers repeat their first token more often than rejected ones."""
    device = model.head.device
    chosen, rejected = sequences(pairs, seed, device), sequences(pairs, seed + 1, device)
    chosen[:, 4::2] = chosen[:, 3:4]
    tokens = torch.cat([chosen, rejected])
    target = tokens.clone()
    target[:, :3] = -100                                    # the prompt
    target = target.reshape(-1)
    offsets = torch.arange(2 * pairs + 1, device=device) * LENGTH
    h = model.features(tokens)
    # the reference's sums over the packed answers: log-probabilities, then ragged rows
    logp, _ = itr.red_logprob(model.logits(h), target)
    ref = itr.red_rows_ragged("sum", logp, offsets)
    weight = torch.full((pairs,), 1.0 / pairs, device=device)
    history = []
    for _ in range(steps):
        _, _, stats, grad = itr.red_preference(model.logits(h), target, offsets, ref_logp=ref, weight=weight, beta=0.1)
        model.step(h, grad, 0.3)
        history.append(stats.clone())
    return torch.stack(history).tolist()                    # loss, margin, share of pairs told apart, 1


def policy(model, reference, rounds=15, inner=4, answers=64, seed=900):
    device = model.head.device
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    rewards = []
    for i in range(rounds):
        tokens = sequences(answers, seed + 10 + i, device)
        h = model.features(tokens)                          # contexts of the positions
        noise = torch.rand((h.shape[0], VOCAB), generator=gen, device=device).clamp(min=1e-9)
        sampled = (model.logits(h).float() - (-noise.log()).log()).argmax(1)    # from the softmax
        reward = (sampled % 2 == 0).float()
        rewards.append(reward.mean())
        target = sampled.clone()
        target.view(answers, LENGTH)[:, :3] = -100          # the prompt was not sampled
        adv = reward - reward.mean()
        old, _ = itr.red_logprob(model.logits(h), target)
        ref, _ = itr.red_logprob(reference.logits(h), target)
        weight = torch.full_like(adv, 1.0 / int((target >= 0).sum()))
        for _ in range(inner):
            _, _, stats, grad = itr.red_policy(model.logits(h), target, old, adv, ref_logp=ref, weight=weight,
                                               kl_coef=0.02, grad_scale=1.0)
            model.step(h, grad, 15.0)
    return torch.stack(rewards).tolist()


def likelihood(model, steps=20, seed=2000):
    """Mean log-probability of a fixed batch, raised by its gradient."""
    tokens = sequences(16, seed, model.head.device)
    h, target = model.features(tokens), tokens.reshape(-1)
    up = torch.full((target.numel(),), -1.0 / target.numel(), device=h.device)
    values = []
    for _ in range(steps):
        logits = model.logits(h)
        logp, lse = itr.red_logprob(logits, target)
        values.append(itr.red_full("sum", logp) / target.numel())
        model.step(h, itr.red_logprob_grad(logits, target, lse, up), 3.0)
    return torch.cat(values).tolist()


def main():
    device = torch.device("cuda")
    teacher, student = Model(7, device), Model(7, device)
    teacher.head *= 6.0
    student.head *= 0.2
    d = distill(student, teacher)
    print(f"distillation   KL to the teacher's top 16: {d[0]:.3f} -> {d[-1]:.3f}")
    reference = student.copy()
    p = preference(student.copy())
    print(f"preference     loss {p[0][0]:.3f} -> {p[-1][0]:.3f}, pairs told apart {p[0][2]:.0%} -> {p[-1][2]:.0%}")
    r = policy(student, reference)
    print(f"policy         reward {r[0]:.3f} -> {r[-1]:.3f}")
    v = likelihood(student.copy())
    print(f"likelihood     mean log-probability {v[0]:.3f} -> {v[-1]:.3f}")
    return d, p, r, v


if __name__ == "__main__":
    main()
