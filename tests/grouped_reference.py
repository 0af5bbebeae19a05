"""Products grouped by rows from their definitions, in 64 bits, for the tests.

``bound`` is how far the library's result may be off: the fp32 sum of `terms` products as
``linear_reference.product_bound`` derives it (2^-23 of the magnitudes for each 64 terms and 64 more),
and one rounding."""
import torch

from linear_reference import TINY, UNIT


def clamp(offsets, rows):
    """The rows' limits that the library takes: at least 0, at most `rows`, none before the last."""
    out, most = [], 0
    for o in offsets:
        most = max(most, min(max(int(o), 0), rows))
        out.append(most)
    return out


def spans(offsets, rows):
    o = clamp(offsets, rows)
    return list(zip(o, o[1:]))


def bound(value, magnitude, terms, dtype):
    e = (terms / 64 + 64) * 2.0 ** -23 * magnitude
    return e + UNIT[dtype] * (value.abs() + e) + TINY[dtype]


def product(x, B, offsets, nt):
    """(result, bound) of x·B[e]ᵀ (nt) or x·B[e] for the rows of each group; 0 and 0 for the others."""
    out = torch.zeros(x.shape[0], B.shape[1 if nt else 2], dtype=torch.float64, device=x.device)
    far = torch.zeros_like(out)
    for e, (i, j) in enumerate(spans(offsets, x.shape[0])):
        a, b = x[i:j].double(), B[e].double()
        b = b.t() if nt else b
        out[i:j] = a @ b
        far[i:j] = bound(out[i:j], a.abs() @ b.abs(), b.shape[0], x.dtype)
    return out, far


def matrices(dD, A, offsets):
    """(dB, bound): dD_eᵀ·A_e for each group."""
    groups = len(offsets) - 1
    out = torch.zeros(groups, dD.shape[1], A.shape[1], dtype=torch.float64, device=A.device)
    far = torch.zeros_like(out)
    for e, (i, j) in enumerate(spans(offsets, A.shape[0])):
        if j > i:
            d, a = dD[i:j].double(), A[i:j].double()
            out[e] = d.t() @ a
            far[e] = bound(out[e], d.abs().t() @ a.abs(), j - i, A.dtype)
    return out, far


def adapters(x, W, down, up, offsets, chosen, scales):
    """(D, bound) of x·Wᵀ + scales[a]·(x·down[a]ᵀ)·up[a]ᵀ, a each row's adapter.

    The shared sum and h = scales[a]·x·down[a]ᵀ are off as any fp32 sum here; h, where it is held as
    two 16-bit numbers, by the second's rounding of what the first left, half a step of half a step
    (and half the least subnormal); the sum over the ranks by what h is, and as another sum."""
    rows, K = x.shape
    a64, w64 = x.double(), W.double()
    D = a64 @ w64.t()
    far = (K / 64 + 64) * 2.0 ** -23 * (a64.abs() @ w64.abs().t())
    for e, (i, j) in enumerate(spans(offsets, rows)):
        a = int(chosen[e])
        if j == i or not 0 <= a < down.shape[0]:
            continue
        s = 1.0 if scales is None else float(scales[a])
        d64, u64, xs = down[a].double(), up[a].double(), a64[i:j]
        h = s * (xs @ d64.t())
        unit = UNIT[x.dtype]
        eh = abs(s) * (K / 64 + 64) * 2.0 ** -23 * (xs.abs() @ d64.abs().t()) + (2.0 ** -23 + unit * unit) * h.abs() + TINY[x.dtype]
        D[i:j] += h @ u64.t()
        far[i:j] += eh @ u64.abs().t() + (x.shape[1] / 64 + 64) * 2.0 ** -23 * ((h.abs() + eh) @ u64.abs().t())
    return D, far + UNIT[x.dtype] * (D.abs() + far) + TINY[x.dtype]
