"""Layer norm's gradient against differences, at rows that 8 bits hold exactly, for the tests.

``rows`` have mean 0 and variance 1 to the last bit and elements of +-0.5 and +-1.5, so the kept rows are the
norm's own and only the sums' roundings and the differences' own errors are left.  The loss
sum(dy * y) has a dy with a large mean and a large part along the rows, so that both terms that the norm's
gradient takes away are large; along ones and along the rows themselves the norm does not change, so
there the derivative is 0."""
import torch

import checkpoint_reference as ref

STEP = 1e-5


def rows(count, cols, seed):
    """3/8 of the elements +-1.5, the others +-0.5, as many of either sign: cols is a multiple of 16."""
    gen = torch.Generator().manual_seed(seed)
    one = torch.tensor([1.5, -1.5] * (cols // 16 * 3) + [0.5, -0.5] * (cols // 16 * 5), dtype=torch.float64)
    return torch.stack([one[torch.randperm(cols, generator=gen)] for _ in range(count)])


def upstream(h, seed):
    gen = torch.Generator().manual_seed(seed)
    return (3.0 + 2.0 * h + torch.randn(h.shape, generator=gen, dtype=torch.float64)).float()


def weight(cols, seed):
    return (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)).float()


def directions(h, dx, seed):
    gen = torch.Generator().manual_seed(seed)
    return {"ones": torch.ones_like(h), "rows": h, "gradient": dx / dx.abs().max(),
            "random": torch.rand(h.shape, generator=gen, dtype=torch.float64) * 2 - 1}


def off(h, dy, w, dx, far):
    """For each direction, per row: (how far dx's derivative is from the difference, how far it may be).

    Per row, dx is off by `far` an element; the difference by STEP^2 / 6 of the third derivative: with steps
    u of at most 1.5 an element, mean, variance and root change by so much that an element's is below
    2000 (|h| <= 1.5, std 1: the derivatives of order k of the inverse root are at most k! (2 * 1.5)^k)."""
    g = dy.double() * w.double()
    out = {}
    for name, u in directions(h, dx, 11).items():
        def y(t):
            c = t - t.mean(1, keepdim=True)
            return c / c.square().mean(1, keepdim=True).sqrt()
        want = (g * (y(h + STEP * u) - y(h - STEP * u))).sum(1) / (2 * STEP)
        bound = (far * u.abs()).sum(1) + (STEP ** 2 / 6 * 2000 + 2.0 ** -50 / STEP) * g.abs().sum(1)
        out[name] = ((dx * u).sum(1) - want).abs(), bound
    return out


def bound(h, dy, w):
    rstd = torch.ones(h.shape[0])
    return ref.grad_bounds(dy, h, w, rstd, torch.float32, torch.float32)[0]
