"""64-bit definition of red_linear_logprob and its backward, and what their
arithmetic may be off by.

Tolerances (u = 2**-24, v = half an eps of the 16-bit type):
  * a logit is a sum of dim products.  The tensor cores add 16 at a time, each
    step off by less than an ulp (they round toward zero), up to 64 steps in a
    row, and the sums of those are added in fp32: off by less than
    (64 + 32 + dim / 512) * 2u of the sum A of the products' magnitudes.
  * logp and lse: their logits, and the fp32 arithmetic of a softmax
    (1.2e-5 + 4e-7 of the value: three roundings per argument, two ulp per
    exponential, 128 additions in a row and a tree).
  * p: relative, the error of z - lse plus 3e-5; lse is given in fp32.
  * g is rounded once (v, or half the smallest f16 of the coefficients'
    power of two); its products' sums are off by at most 2u per step of 16;
    the result is rounded once more.
"""
import torch

U = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38}


class Reference:
    """Everything in 64 bits, on the device of the inputs."""

    def __init__(self, hidden, weight, target, scale=1.0):
        self.dt, self.scale = hidden.dtype, scale
        rows, vocab = hidden.shape[0], weight.shape[0]
        self.live = (target >= 0) & (target < vocab)
        self.h = torch.where(self.live[:, None], hidden.double(), 0.0)
        self.w = weight.double()
        self.at = torch.where(self.live, target, 0)
        z = self.h @ self.w.t() * scale
        size = self.h.abs() @ self.w.abs().t() * scale
        steps = 96 + hidden.shape[1] / 512
        self.dz = size.amax(1) * steps * 2 * U
        zero = torch.zeros(rows, dtype=torch.float64, device=hidden.device)
        norm = torch.logsumexp(z, 1)
        self.lse = torch.where(self.live, norm, zero)
        self.logp = torch.where(self.live, z.gather(1, self.at[:, None])[:, 0] - norm, zero)
        self.p = (z - norm[:, None]).exp()

    def check_forward(self, logp, lse):
        for got, want, name in ((logp, self.logp, "logp"), (lse, self.lse, "lse")):
            off = (got.double() - want).abs()
            tol = torch.where(self.live, 2 * self.dz + 1.2e-5 + 4e-7 * want.abs(), 0.0)
            bad = ~(off <= tol)
            assert not bad.any(), f"{name}: {int(bad.sum())} off, first {got[bad][0]} for {want[bad][0]} +- {tol[bad][0]}"

    def gradients(self, dlogp, dlse=None):
        d = torch.where(self.live, dlogp.double(), 0.0)
        n = torch.zeros_like(d) if dlse is None else torch.where(self.live, dlse.double(), 0.0)
        by_p = ((n - d) * self.scale)[:, None] * self.p
        g = by_p.clone()
        g[torch.arange(g.shape[0], device=g.device), self.at] += d * self.scale
        rel = (2 * self.dz + 3e-5 + 4 * U * self.lse.abs())[:, None]
        unit = float(torch.maximum(d.abs(), (n - d).abs()).max()) * self.scale
        dg = by_p.abs() * rel + HALF[self.dt] * (g.abs() + by_p.abs() * rel) + 2 * TINY[self.dt] * unit
        # a row out of the loss has exactly nothing
        dg = torch.where((self.live & ((d != 0) | (n != 0)))[:, None], dg, 0.0)
        self.g, self.dg = g, dg
        want_h, want_w = g @ self.w, g.t() @ self.h
        size_h, size_w = g.abs() @ self.w.abs(), g.abs().t() @ self.h.abs()
        tol_h = dg @ self.w.abs() + size_h * (g.shape[1] / 16 + 16) * 2 * U
        tol_w = dg.t() @ self.h.abs() + size_w * (g.shape[0] / 16 + 16) * 2 * U
        return [(want, tol + HALF[self.dt] * (want.abs() + tol) + TINY[self.dt])
                for want, tol in ((want_h, tol_h), (want_w, tol_w))]

    def check_gradients(self, grad_hidden, grad_weight, dlogp, dlse=None):
        for got, (want, tol), name in zip((grad_hidden, grad_weight), self.gradients(dlogp, dlse), ("hidden", "weight")):
            if got is None:
                continue
            bad = ~((got.double() - want).abs() <= tol)
            assert not bad.any(), (f"grad_{name}: {int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}: "
                                   f"{got[bad][0]} for {want[bad][0]} +- {tol[bad][0]}")
            if name == "hidden":
                out = ~self.live | ((dlogp == 0) & (torch.zeros_like(dlogp) if dlse is None else dlse).eq(0))
                assert bool((got[out] == 0).all()), "a row out of the loss has a gradient"
