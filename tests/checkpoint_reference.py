"""Rows of microscaled 8-bit floats and layer norm's passes from them, from their definitions in 64
bits, for the tests."""
import torch

import linear_reference as ref
from linear_reference import TINY, U32, UNIT

E4M3 = ref.e4m3_values()  # codes 0 .. 126


def blocks(t):
    """[rows, cols] as [rows, blocks, 32], zeros past the row's end."""
    rows, cols = t.shape
    full = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=t.device)
    full[:, :cols] = t
    return full.view(rows, -1, 32)


def scale_codes(amax):
    """E8M0 codes of 2^(floor(log2(amax)) - 8), the exponent at least -127."""
    e = torch.where(amax > 0, torch.frexp(amax).exponent.double() - 1 - 8, torch.tensor(-127.0, dtype=torch.float64, device=amax.device))
    return (e.clamp(min=-127) + 127).long()


def nearest(v):
    """v rounded to E4M3, ties to the even code, magnitudes past 448 to 448."""
    table = torch.tensor(E4M3, dtype=torch.float64, device=v.device)
    return torch.sign(v) * table[ref.nearest(v.abs(), E4M3)]


def values(kept):
    """What kept rows stand for."""
    codes, scales = kept
    shape = codes.shape
    codes, scales = codes.reshape(-1, shape[-1]).view(torch.uint8).long(), scales.reshape(-1, scales.shape[-1])
    table = torch.tensor(E4M3 + [float("nan")], dtype=torch.float64, device=codes.device)
    v = table[codes % 128] * (1.0 - 2.0 * (codes // 128).double())
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, float("nan"), s)
    return (v * s.repeat_interleave(32, 1)[:, :shape[-1]]).view(shape)


def keep(h):
    """(codes float8_e4m3fn, scales uint8) of h by the definition."""
    b = blocks(h.double())
    code = scale_codes(b.abs().amax(2))
    v = nearest(b / torch.exp2(code.double() - 127)[:, :, None]).view(h.shape[0], -1)[:, :h.shape[1]]
    return v.float().to(torch.float8_e4m3fn).contiguous(), code.to(torch.uint8)


def check_kept(kept, h, far):
    """Whether kept rows hold h, known to within `far`: each scale is that of a largest magnitude in
    that range, and each element, in its block's scale, rounds from some value in its range."""
    scales = kept[1].reshape(-1, kept[1].shape[-1]).long()
    v = values(kept).reshape(h.shape)
    b, e = blocks(h), blocks(far.expand_as(h))
    low, high = (b.abs() - e).clamp(min=0).amax(2), (b.abs() + e).amax(2)
    assert bool(((scale_codes(low) <= scales) & (scales <= scale_codes(high))).all()), "scales"
    s = torch.exp2(scales.double() - 127)[:, :, None]
    got = blocks(v)
    least, most = nearest((b - e) / s) * s, nearest((b + e) / s) * s
    assert bool(((least <= got) & (got <= most)).all()), "codes"


def h_bounds(x, eps):
    """(h, how far an fp32 computation of it may be off): ``linear_reference.norm_bounds`` of the norm
    without weights, before its rounding (that of fp32 is a thousandth of the sums')."""
    h, _, _ = ref.norm(x, None, None, eps)
    return h, ref.norm_bounds(x, None, None, eps, torch.float32)[0]


def grad(dy, h, weight, rstd):
    dy, rstd = dy.double(), rstd.double()[:, None]
    g = dy if weight is None else dy * weight.double()
    dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)


def grad_bounds(dy, h, weight, rstd, dtype, wdtype):
    """As ``linear_reference.norm_grad_bounds``, with h exact: g has 1 rounding, g * h 2 more; the row
    sums pass through at most 64 + n / 1024 additions, the column sums through rows / 152 + 64."""
    dx, dw, db = grad(dy, h, weight, rstd)
    dy, r = dy.double(), rstd.double()[:, None]
    rows, n = h.shape
    chain = 64 + n / 1024
    h = h.abs()
    g = (dy if weight is None else dy * weight.double()).abs()
    c2 = (g * h).mean(1, keepdim=True)
    e = r * (6 * U32 * (g + g.mean(1, keepdim=True) + h * c2) + (chain + 3) * U32 * g.mean(1, keepdim=True) + h * (chain + 6) * U32 * c2)
    column = rows / 152 + 64
    e_dw, e_db = (column + 4) * U32 * (dy.abs() * h).sum(0), (column + 1) * U32 * dy.abs().sum(0)
    return (e + UNIT[dtype] * (dx.abs() + e) + TINY[dtype], e_dw + UNIT[wdtype] * (dw.abs() + e_dw) + TINY[wdtype],
            e_db + UNIT[wdtype] * (db.abs() + e_db) + TINY[wdtype])


def restore(kept, weight, bias, dtype):
    """(y, bound): the product and the sum have one fp32 rounding each, y one to `dtype`."""
    h = values(kept)
    w = 1.0 if weight is None else weight.double()
    b = 0.0 if bias is None else bias.double()
    y = h * w + b
    e = 2 * U32 * ((h * w).abs() + (0.0 if bias is None else bias.double().abs()))
    return y, e + UNIT[dtype] * (y.abs() + e) + TINY[dtype]
