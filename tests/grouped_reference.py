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
