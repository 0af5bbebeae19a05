"""The operators of a pre-norm linear layer, as cases to measure: layer norm, its gradient, the
quantisation to microscaled 4-bit floats, and the product of two such matrices.

    norm       y, mean, rstd of layer norm over the last axis
    norm_grad  dx, dweight, dbias of layer norm, from what the forward pass left
    quantize   x to 4-bit floats with a scale per block of its rows, and the values they stand for
    product    D = A * B^T of two such matrices, summed in 32 bits, rounded once

A quantised matrix of `rows` x `cols` is held as
    data    uint8 [rows, ceil(cols / 32) * 16]: two E2M1 codes per byte, the even column in the low
            nibble, columns past `cols` zero
    scales  uint8 [ceil(rows / 128), groups / 4 rounded up, 32, 4, 4]: the scale code of row
            128 i + 32 g + l and block 4 j + k at [i, j, l, g, k], zero where there is none.
Format "mx" has blocks of 32 and power-of-two scales (E8M0), format "nv" blocks of 16 and E4M3
scales, times 2^exponent for the whole matrix.

``own = False`` runs the plain form of each: elementary torch operations in 32 bits, rounded once
at the end.  ``own = True`` calls the framework.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5
DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}
SIZE = {"float16": 2, "bfloat16": 2, "float32": 4}


def listed():
    return [
        # one new token of a decoder before its next linear layer: the time is the call's latency
        {"name": "norm one token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "float16", "weights": "float16", "gap": 0},
        # a prompt (or a training batch) of 8192 tokens, weights kept in 32 bits
        {"name": "norm 8192 tokens", "op": "norm", "rows": 8192, "cols": 4096, "dtype": "bfloat16", "weights": "float32", "gap": 0},
        # an odd width in 32 bits, rows inside a wider buffer: nothing is aligned
        {"name": "norm odd width", "op": "norm", "rows": 1023, "cols": 5003, "dtype": "float32", "weights": "float32", "gap": 6},
        # the training step of the second case: the weight's gradient sums 8192 rows
        {"name": "norm gradient 8192 tokens", "op": "norm_grad", "rows": 8192, "cols": 4096, "dtype": "bfloat16", "weights": "float32", "gap": 0},
        # a short ragged batch of odd width, all in 16 bits: few rows share the weight's gradient
        {"name": "norm gradient ragged", "op": "norm_grad", "rows": 517, "cols": 1021, "dtype": "float16", "weights": "float16", "gap": 0},
        # the activations of a prompt, quantised before each linear layer
        {"name": "quantize 8192 tokens mx", "op": "quantize", "rows": 8192, "cols": 4096, "dtype": "float16", "format": "mx", "exponent": 0},
        # one token's activations
        {"name": "quantize one token nv", "op": "quantize", "rows": 1, "cols": 8192, "dtype": "bfloat16", "format": "nv", "exponent": 0},
        # one token through a square linear layer: the weights are read once, the time is theirs
        {"name": "product one token mx", "op": "product", "rows": 1, "cols": 8192, "inner": 8192, "dtype": "float16", "format": "mx"},
        # a decoding batch of 64 through the wide projection of a feed-forward layer
        {"name": "product 64 tokens nv", "op": "product", "rows": 64, "cols": 28672, "inner": 4096, "dtype": "bfloat16", "format": "nv"},
        # a ragged prompt: rows, columns and depth end inside a tile
        {"name": "product ragged nv", "op": "product", "rows": 1000, "cols": 1529, "inner": 2088, "dtype": "float16", "format": "nv"},
        # a prompt of 2048 tokens through a square layer
        {"name": "product 2048 tokens mx", "op": "product", "rows": 2048, "cols": 4096, "inner": 4096, "dtype": "float16", "format": "mx"},
        # the largest: 8192 tokens through the wide projection, bound by the tensor cores
        {"name": "product 8192 tokens mx", "op": "product", "rows": 8192, "cols": 28672, "inner": 4096, "dtype": "float16", "format": "mx"},
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm", "norm_grad", "quantize", "product"])
    if op in ("norm", "norm_grad"):
        dtype = rng.choice(["float16", "bfloat16", "float32"])
        return {"op": op, "rows": size(1, 8192), "cols": size(64, 8192), "dtype": dtype,
                "weights": rng.choice([dtype, "float32"]), "gap": rng.choice([0, 0, 8, 6])}
    if op == "quantize":
        return {"op": op, "rows": size(1, 8192), "cols": size(64, 8192), "dtype": rng.choice(["float16", "bfloat16", "float32"]),
                "format": rng.choice(["mx", "nv"]), "exponent": 0}
    return {"op": op, "rows": size(1, 8192), "cols": size(64, 14336), "inner": size(64, 8192),
            "dtype": rng.choice(["float16", "bfloat16"]), "format": rng.choice(["mx", "nv"])}


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _stream(gen, rows, cols, dtype, gap=0):
    """A residual stream: unit variance, an offset, a few channels far larger than the rest.  The
    rows are `cols` wide inside rows of cols + gap."""
    x = torch.randn(rows, cols + gap, generator=gen, device="cuda")
    loud = torch.rand(cols + gap, generator=gen, device="cuda") < 0.002
    x = (x + 0.3) * torch.where(loud, 12.0, 1.0)
    return x.to(dtype)[:, :cols]


def _norm_inputs(case, seed):
    gen = _generator(seed)
    dtype, wtype = DTYPES[case["dtype"]], DTYPES[case["weights"]]
    s = {"x": _stream(gen, case["rows"], case["cols"], dtype, case["gap"]),
         "weight": (1 + 0.1 * torch.randn(case["cols"], generator=gen, device="cuda")).to(wtype),
         "bias": (0.1 * torch.randn(case["cols"], generator=gen, device="cuda")).to(wtype)}
    if case["op"] == "norm_grad":
        s["dy"] = _stream(gen, case["rows"], case["cols"], dtype, case["gap"])
        x = s["x"].float()
        s["mean"] = x.mean(1)
        s["rstd"] = ((x - s["mean"][:, None]).square().mean(1) + EPS).rsqrt()
    return s


def _quantize_input(case, seed):
    x = _stream(_generator(seed), case["rows"], case["cols"], DTYPES[case["dtype"]])
    if case["rows"] > 1:
        x[-1] = 0  # a padding token
    return x


def prepare(case, seed):
    if case["op"] in ("norm", "norm_grad"):
        return {"case": case, **_norm_inputs(case, seed)}
    if case["op"] == "quantize":
        return {"case": case, "x": _quantize_input(case, seed)}
    gen = _generator(seed)
    # activations after a norm, and weights of a linear layer; each quantised as the program keeps it
    exponents = (0, -8) if case["format"] == "nv" else (0, 0)
    s = {"case": case, "exponents": exponents}
    for name, rows, scale, exponent in (("a", case["rows"], 1.0, exponents[0]), ("b", case["cols"], 0.02, exponents[1])):
        x = scale * torch.randn(rows, case["inner"], generator=gen, device="cuda")
        codes, scales = _codes(x, case["format"], exponent)
        s[name] = (codes[:, 1::2] << 4) | codes[:, 0::2]
        s[name + "_scales"] = _tiled(scales)
    return s


# -------------------------------------------------------------- plain form --

def _blocks(x, fmt):
    """x in 32 bits as [rows, blocks, block], zeros past its columns (to a multiple of 32)."""
    block = 32 if fmt == "mx" else 16
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[1] % 32))
    return x.reshape(x.shape[0], -1, block)


def _pow2(codes):
    """2^(code - 127) of E8M0 codes; NaN for 255."""
    bits = torch.where(codes == 0, 1 << 22, codes.int() << 23)
    return torch.where(codes == 255, math.nan, bits.view(torch.float32))


def _scale_of(blocks, fmt, exponent):
    """The scale code of each block and the value it stands for."""
    amax = blocks.abs().amax(2)
    bad = ~torch.isfinite(amax)
    if fmt == "mx":  # 2^(floor(log2(amax)) - 2): the largest element's exponent meets E2M1's largest
        codes = ((amax.view(torch.int32) >> 23) - 2).clamp(0, 254)
        codes = torch.where(bad, 255, codes).to(torch.uint8)
        return codes, _pow2(codes)
    s = (amax / 6 * 2.0 ** -exponent).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    codes = torch.where(bad, 127, s.view(torch.uint8))
    return codes, codes.view(torch.float8_e4m3fn).float() * 2.0 ** exponent


def _index(t):
    """The index in E2M1 of |t|, ties to the even one, the largest past it."""
    t = t.abs()
    return ((t > 0.25).byte() + (t >= 0.75).byte() + (t > 1.25).byte() + (t >= 1.75).byte() + (t > 2.5).byte()
            + (t >= 3.5).byte() + (t > 5.0).byte())


def _codes(x, fmt, exponent):
    blocks = _blocks(x, fmt)
    scales, value = _scale_of(blocks, fmt, exponent)
    t = blocks / value[:, :, None]
    codes = _index(t) | (torch.signbit(blocks).byte() << 3)
    codes = torch.where(torch.isnan(value)[:, :, None], 0, codes)
    return codes.reshape(x.shape[0], -1).byte(), scales


def _tiled(scales):
    """[rows, blocks] scale codes as [row tiles, block tiles, 32, 4, 4]."""
    rows, blocks = scales.shape
    s = torch.nn.functional.pad(scales, (0, -blocks % 4, 0, -rows % 128))
    return s.reshape(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()


def _values(data, scales, fmt, exponent):
    """The 32-bit values of a quantised matrix, its zero columns included."""
    rows, blocks = data.shape[0], data.shape[1] // (16 if fmt == "mx" else 8)
    flat = scales.permute(0, 3, 2, 1, 4).reshape(scales.shape[0] * 128, -1)[:rows, :blocks]
    if fmt == "mx":
        value = _pow2(flat)
    else:
        value = flat.contiguous().view(torch.float8_e4m3fn).float() * 2.0 ** exponent
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=data.device)
    v = table[torch.stack((data & 15, data >> 4), 2).int()]
    return (v.reshape(rows, blocks, -1) * value[:, :, None]).reshape(rows, -1)


def _plain(s):
    case = s["case"]
    if case["op"] == "norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        centred = x - mean
        rstd = (centred.square().mean(1, keepdim=True) + EPS).rsqrt()
        y = centred * rstd * s["weight"].float() + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if case["op"] == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["weight"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        wtype = s["weight"].dtype
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0).to(wtype), "dbias": dy.sum(0).to(wtype)}
    if case["op"] == "quantize":
        blocks = _blocks(s["x"], case["format"])
        _, value = _scale_of(blocks, case["format"], case["exponent"])
        t = blocks / value[:, :, None]
        table = torch.tensor(E2M1, device=t.device)
        v = torch.copysign(table[_index(t).int()], t) * value[:, :, None]
        return {"values": v.reshape(v.shape[0], -1)[:, :case["cols"]].to(torch.bfloat16)}
    a = _values(s["a"], s["a_scales"], case["format"], s["exponents"][0])
    b = _values(s["b"], s["b_scales"], case["format"], s["exponents"][1])
    return {"d": (a @ b.T).to(DTYPES[case["dtype"]])}


def run(state):
    if not own:
        return _plain(state)
    import blackwell_tensor_core_02_gb300 as g

    case = state["case"]
    if case["op"] == "norm":
        y, mean, rstd = g.layer_norm(state["x"], state["weight"], state["bias"], EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if case["op"] == "norm_grad":
        dx, dweight, dbias = g.layer_norm_backward(state["dy"], state["x"], state["weight"], state["mean"], state["rstd"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if case["op"] == "quantize":
        q = g.quantize_fp4(state["x"], case["format"], exponent=case["exponent"])
        return {"values": g.dequantize_fp4(q, torch.bfloat16)}
    a = g.Fp4Tensor(state["a"], state["a_scales"], case["inner"], case["format"], state["exponents"][0])
    b = g.Fp4Tensor(state["b"], state["b_scales"], case["inner"], case["format"], state["exponents"][1])
    return {"d": g.gemm_fp4_nt(a, b, dtype=DTYPES[case["dtype"]])}


# -------------------------------------------------------------------- work --

def work(case):
    rows, cols, size = case["rows"], case["cols"], SIZE[case["dtype"]]
    if case["op"] == "norm":  # x and the two weights in, y and the two statistics out
        return {"bytes": 2 * rows * cols * size + 2 * cols * SIZE[case["weights"]] + 8 * rows, "flops": 8 * rows * cols}
    if case["op"] == "norm_grad":  # dy, x, weight and the statistics in, dx and the weights' gradients out
        return {"bytes": 3 * rows * cols * size + 3 * cols * SIZE[case["weights"]] + 8 * rows, "flops": 14 * rows * cols}
    if case["op"] == "quantize":  # x in, the values (16 bits) out
        return {"bytes": rows * cols * (size + 2), "flops": 4 * rows * cols}
    inner = -(-case["inner"] // 32) * 32
    block = 32 if case["format"] == "mx" else 16
    return {"bytes": (rows + cols) * (inner // 2 + inner // block) + rows * cols * size, "flops": 2 * rows * cols * case["inner"]}


# ------------------------------------------------------------ in 64 bits --

def _exact_values(data, scales, fmt, exponent):
    """The values of a quantised matrix from the formats' definitions: sign, exponent, mantissa."""
    rows = data.shape[0]
    codes = torch.empty(rows, data.shape[1] * 2, dtype=torch.int64, device=data.device)
    codes[:, 0::2] = (data % 16).long()
    codes[:, 1::2] = (data // 16).long()
    sign = 1.0 - 2.0 * (codes // 8).double()
    e, m = (codes // 2) % 4, (codes % 2).double()
    v = sign * torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1) * (1 + 0.5 * m))
    block = 32 if fmt == "mx" else 16
    r = torch.arange(rows, device=data.device)[:, None]
    k = torch.arange(codes.shape[1], device=data.device)[None, :] // block
    c = scales.long()[r // 128, k // 4, r % 32, r % 128 // 32, k % 4]
    if fmt == "mx":
        return v * torch.exp2(c.double() - 127)
    se, sm = c // 8 % 16, (c % 8).double()
    s = torch.where(se == 0, sm / 8 * 2.0 ** -6, torch.exp2(se.double() - 7) * (1 + sm / 8))
    return v * s * 2.0 ** exponent


def exact(case, seed):
    if case["op"] == "norm":
        s = _norm_inputs(case, seed)
        x, n = s["x"].double(), case["cols"]
        mean = x.sum(1) / n
        var = ((x - mean[:, None]) ** 2).sum(1) / n
        y = (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * s["weight"].double() + s["bias"].double()
        return {"y": y, "mean": mean, "rstd": 1 / torch.sqrt(var + EPS)}
    if case["op"] == "norm_grad":
        s, n = _norm_inputs(case, seed), case["cols"]
        dy, x, w = s["dy"].double(), s["x"].double(), s["weight"].double()
        mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
        h = (x - mean) * rstd
        c1 = (dy * w).sum(1, keepdim=True) / n
        c2 = (dy * w * h).sum(1, keepdim=True) / n
        return {"dx": (dy * w - c1 - h * c2) * rstd, "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}
    if case["op"] == "quantize":
        x, block = _quantize_input(case, seed).double(), 32 if case["format"] == "mx" else 16
        full = torch.zeros(x.shape[0], -(-x.shape[1] // block) * block, dtype=torch.float64, device=x.device)
        full[:, :x.shape[1]] = x
        b = full.view(x.shape[0], -1, block)
        amax = b.abs().max(2, keepdim=True).values
        if case["format"] == "mx":
            s = torch.exp2((torch.frexp(amax).exponent - 3).clamp(-127, 127).double())
        else:
            t = amax / 6 / 2.0 ** case["exponent"]
            ulp = torch.exp2((torch.frexp(t).exponent - 1).clamp(-6, 8).double() - 3)
            s = (torch.round(t / ulp) * ulp).clamp(2.0 ** -9, 448) * 2.0 ** case["exponent"]
        r = b.abs() / s
        step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))
        v = torch.sign(b) * torch.clamp(torch.round(r / step) * step, max=6.0) * s
        return {"values": v.view(x.shape[0], -1)[:, :x.shape[1]]}
    s = prepare(case, seed)
    a = _exact_values(s["a"], s["a_scales"], case["format"], s["exponents"][0])
    b = _exact_values(s["b"], s["b_scales"], case["format"], s["exponents"][1])
    return {"d": torch.mm(a, b.t())}
