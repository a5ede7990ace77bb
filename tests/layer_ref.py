"""Plain 64-bit forms of the layer's operators, and the error a correct kernel may have against them.

Bounds.  bf16 rounds with unit roundoff 2^-8.  A product summed over n terms in binary32 (by tensor cores, which may
truncate instead of rounding) is within n * 2^-23 of the sum of the terms' magnitudes.  The activations' slopes are
below 1.13 in magnitude, and the kernels' exponential and quotient are good to 2^-19 relatively.
"""
import math

import torch

BF16 = 2.0 ** -8
F32 = 2.0 ** -23
SLOPE = 1.13
MATH = 2.0 ** -19


def act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope(name, z):
    z = z.detach().clone().requires_grad_()
    return torch.autograd.grad(act(name, z).sum(), z)[0]


def forward(x, w, b, name):
    """z, y and the bounds of their errors before they are rounded to bf16."""
    x, w = x.double(), w.double()
    z = x @ w.t()
    err = (x.abs() @ w.abs().t()) * x.shape[1] * F32
    if b is not None:
        z = z + b.double()
    err = err + z.abs() * F32
    if name != "swiglu":
        y = act(name, z)
        return z, err, y, err * SLOPE + (y.abs() + z.abs()) * MATH
    g, u = z.chunk(2, 1)
    eg, eu = err.chunk(2, 1)
    s = act("silu", g)
    y = s * u
    return z, err, y, SLOPE * eg * u.abs() + s.abs() * eu + (y.abs() + (g * u).abs()) * MATH


def dgrad(dy, w, name, pre):
    dy, w = dy.double(), w.double()
    d = dy @ w
    err = (dy.abs() @ w.abs()) * dy.shape[1] * F32
    if name == "none":
        return d, err
    pre = pre.double()
    if name == "swiglu":
        g, u = pre.chunk(2, 1)
        sl, s = slope("silu", g), act("silu", g)
        dz = torch.cat([d * u * sl, d * s], 1)
        e = torch.cat([SLOPE * err * u.abs() + (d * u).abs() * 4 * MATH, err * s.abs() + (d * s).abs() * 4 * MATH], 1)
        return dz, e
    return d * slope(name, pre), SLOPE * err + d.abs() * 4 * MATH * (1 + pre.abs().clamp(max=32))


def close(got, want, err, what, half=BF16):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    ok = ~want.isnan()
    bad = (got - want).abs()[ok] > (want.abs() * half * 1.01 + err * (1 + half) + 1e-37)[ok]
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst "
                                 f"{float((got - want).abs()[ok].max())}")


class Routed:
    """Rank buffers whose rows belong to (source, expert) ranges, in the receive layout of a dispatch: counts is
    [rank][source][expert].  Rows past the last range belong to nobody."""

    def __init__(self, counts, slack=3):
        self.counts = counts
        self.k, self.sources, self.experts = len(counts), len(counts[0]), len(counts[0][0])
        self.seg = torch.zeros(self.k, self.sources * self.experts + 1, dtype=torch.int64)
        self.of = []  # expert of every row, -1: nobody's
        self.cap = []
        for d in range(self.k):
            flat = [n for s in counts[d] for n in s]
            self.seg[d, 1:] = torch.tensor(flat).cumsum(0)
            of = torch.cat([torch.full((n,), i % self.experts) for i, n in enumerate(flat)] + [torch.full((slack,), -1)])
            self.of.append(of.cuda() if torch.cuda.is_available() else of)
            self.cap.append(len(of))
        if torch.cuda.is_available():
            self.seg = self.seg.cuda()

    def rows(self, d, e):
        return torch.nonzero(self.of[d] == e).flatten()


def random_counts(k, sources, experts, most, seed, empty=0.25):
    g = torch.Generator().manual_seed(seed)
    n = torch.randint(0, most + 1, (k, sources, experts), generator=g)
    n[torch.rand(k, sources, experts, generator=g) < empty] = 0
    return n.tolist()
