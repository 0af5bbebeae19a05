"""The linear layer's operators from their definitions, in 64 bits, for the tests.

Everything is float64 torch on the tensors' own device; nothing of the package is used.  A quantised
matrix is built here code by code (value tables and a search for the nearest), apart from any
arithmetic the library does.
"""
import torch

U32 = 2.0 ** -24                                      # half a unit in the last place of fp32
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}  # half the least subnormal
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def norm(x, weight, bias, eps):
    x = x.double()
    mean = x.mean(-1)
    var = (x - mean[..., None]).square().mean(-1)
    rstd = (var + eps).rsqrt()
    y = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * weight.double()
    if bias is not None:
        y = y + bias.double()
    return y, mean, rstd


def norm_bounds(x, weight, bias, eps, dtype):
    """How far y, mean and rstd of an fp32 computation, y rounded once to `dtype`, may be off.

    A sum of n terms in which no value passes through more than 64 additions is off by at most 64 U32
    times the sum of magnitudes.  Hence mean: 64 U32 mean|x| (and its division, 1 more); the centred
    values: that and one rounding; rstd: half of the variance's relative error (squares 2, sum 64,
    division, eps, and the mean's error squared over the variance) and the root's and quotient's
    own roundings; y: the product of these, two more roundings and the one to `dtype`."""
    y, mean, rstd = norm(x, weight, bias, eps)
    x = x.double()
    n = x.shape[-1]
    chain = 64 + n / 1024
    e_mean = (chain + 2) * U32 * x.abs().mean(-1)
    centred = (x - mean[..., None]).abs()
    rel_rstd = (chain + 8) * U32 + rstd.square() * (e_mean.square() + 2 * e_mean * U32 * centred.mean(-1))
    w = 1.0 if weight is None else weight.double().abs()
    b = 0.0 if bias is None else bias.double().abs()
    xhat = centred * rstd[..., None]
    e_y = w * (rstd[..., None] * (e_mean[..., None] + 2 * U32 * centred) + xhat * (rel_rstd[..., None] + 4 * U32)) + 2 * U32 * b
    return e_y + UNIT[dtype] * (y.abs() + e_y) + TINY[dtype], e_mean + TINY[torch.float32], rel_rstd * rstd


def norm_grad(dy, x, weight, mean, rstd):
    dy, x = dy.double(), x.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    h = (x - mean) * rstd
    g = dy if weight is None else dy * weight.double()
    dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)


def norm_grad_bounds(dy, x, weight, mean, rstd, dtype, wdtype):
    """The same for the gradient, mean and rstd taken as given: h has 2 roundings, g 1, g * h 4; the
    row sums pass through at most 64 + n / 1024 additions, the column sums through rows / 304 + 64."""
    dx, dw, db = norm_grad(dy, x, weight, mean, rstd)
    dy, x = dy.double(), x.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    rows, n = x.shape
    chain = 64 + n / 1024
    h = ((x - mean) * rstd).abs()
    g = (dy if weight is None else dy * weight.double()).abs()
    e_c1 = (chain + 3) * U32 * g.mean(1, keepdim=True)
    c2 = (g * h).mean(1, keepdim=True)
    e_c2 = (chain + 6) * U32 * c2
    e_dx = rstd * (6 * U32 * (g + g.mean(1, keepdim=True) + h * c2) + e_c1 + h * e_c2)
    column = rows / 304 + 64
    e_dw = (column + 4) * U32 * (dy.abs() * h).sum(0)
    e_db = (column + 1) * U32 * dy.abs().sum(0)
    return (e_dx + UNIT[dtype] * (dx.abs() + e_dx) + TINY[dtype], e_dw + UNIT[wdtype] * (dw.abs() + e_dw) + TINY[wdtype],
            e_db + UNIT[wdtype] * (db.abs() + e_db) + TINY[wdtype])


def e4m3_values():
    """Value of each E4M3 code 0 .. 126."""
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return v


def nearest(v, table):
    """Index of the value of the ascending `table` nearest to v >= 0, ties to the even index, past
    the last one the last."""
    table = torch.tensor(table, dtype=torch.float64, device=v.device)
    hi = torch.searchsorted(table, v.contiguous()).clamp(1, len(table) - 1)
    lo = hi - 1
    dlo, dhi = v - table[lo], table[hi] - v
    up = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    return torch.where(up, hi, lo)


def quantize(x, fmt, exponent=0):
    """(codes [rows, padded cols], scale codes [rows, blocks]) by the definition."""
    block = 32 if fmt == "mx" else 16
    rows, cols = x.shape
    full = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=x.device)
    full[:, :cols] = x.double()
    b = full.view(rows, -1, block)
    amax = b.abs().amax(2)
    bad = ~torch.isfinite(amax)
    a = torch.where(bad, 0.0, amax)
    if fmt == "mx":
        e = torch.where(a > 0, torch.frexp(a).exponent.double() - 1, torch.tensor(-200.0, device=x.device, dtype=torch.float64))
        e = (e - 2).clamp(-127, 127)
        scale_codes, scale = (e + 127).long(), torch.exp2(e)
    else:
        scale_codes = nearest((a / 6 * 2.0 ** -exponent).clamp(2.0 ** -9, 448.0), e4m3_values())
        scale = torch.tensor(e4m3_values(), dtype=torch.float64, device=x.device)[scale_codes] * 2.0 ** exponent
    mag = nearest(torch.where(torch.isfinite(b), b.abs(), 0.0) / scale[:, :, None], E2M1)
    codes = mag + 8 * torch.signbit(b).long()
    codes = torch.where(bad[:, :, None], 0, codes)
    scale_codes = torch.where(bad, 255 if fmt == "mx" else 127, scale_codes)
    return codes.view(rows, -1), scale_codes


def tile(scale_codes):
    """[rows, blocks] as the stored [row tiles, block tiles, 32, 4, 4], zeros where there is none."""
    rows, blocks = scale_codes.shape
    out = torch.zeros(-(-rows // 128), -(-blocks // 4), 32, 4, 4, dtype=torch.uint8, device=scale_codes.device)
    r = torch.arange(rows, device=scale_codes.device)[:, None]
    k = torch.arange(blocks, device=scale_codes.device)[None, :]
    out[r // 128, k // 4, r % 32, r % 128 // 32, k % 4] = scale_codes.to(torch.uint8)
    return out


def pack(codes):
    return (codes[:, 0::2] + 16 * codes[:, 1::2]).to(torch.uint8)


def values(codes, scale_codes, fmt, exponent=0):
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    if fmt == "mx":
        scale = torch.exp2(scale_codes.double() - 127)
        scale = torch.where(scale_codes == 255, float("nan"), scale)
    else:
        t = torch.tensor(e4m3_values() + [float("nan")], dtype=torch.float64, device=codes.device)
        scale = t[scale_codes.long()] * 2.0 ** exponent
    rows, blocks = scale_codes.shape
    return (table[codes].view(rows, blocks, -1) * scale[:, :, None]).view(rows, -1)


def product_bound(a, b, dtype, alpha=1.0):
    """(D, how far off it may be) for values a, b: each of the K / 64 steps of the fp32 accumulation,
    in whatever order and with truncation where the hardware truncates, is off by at most 2^-23 of
    the magnitudes summed so far, 64 more for the sums inside the steps and over K slices; then
    alpha and one rounding."""
    d = alpha * (a @ b.T)
    mag = abs(alpha) * (a.abs() @ b.abs().T)
    e = (a.shape[1] / 64 + 64) * 2.0 ** -23 * mag
    return d, e + UNIT[dtype] * (d.abs() + e) + TINY[dtype]
