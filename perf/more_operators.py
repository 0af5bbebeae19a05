"""The operators that make a linear layer one of many, as cases to measure: products grouped by
expert and their gradients, low-rank adapters of many requests beside a shared projection, and layer
norm that keeps 8 bits an element for its backward pass.

    experts     D[r] = A[r] * B[e]^T for the rows r of group e: rows sorted by expert, each group with
                a matrix of its own
    tokens      its gradient for the rows, dA[r] = dD[r] * B[e]
    weights     its gradient for the matrices, dB[e] = dD_e^T * A_e; zeros for a group without rows
    adapters    D[r] = x[r] * W^T + scale[a] * (x[r] * down[a]^T) * up[a]^T, a the adapter of the request
                that row r belongs to; a request without an adapter (-1) has the shared product alone
    keep        layer norm that keeps its normalised rows h = (x - mean) * rstd in 8 bits, and the
                result once more from what it kept
    keep_grad   layer norm's gradient from the kept rows

Group e (or request e) has rows offsets[e] to offsets[e + 1] - 1; rows behind the last one have no
group, and their results are zeros.  Kept rows are E4M3 codes with one power-of-two scale (E8M0) for
32 elements of a row, 2^(floor(log2(amax)) - 8): a float8_e4m3fn matrix and one byte a block.

``own = False`` runs the plain form of each: elementary torch operations in 32 bits, rounded once
at the end.  ``own = True`` calls the framework.
"""
import math
import random

import torch

own = False

EPS = 1e-5
DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}
SIZE = {"float16": 2, "bfloat16": 2, "float32": 4}


def listed():
    return [
        # one token through the two experts of 64 that its router chose: the call's latency
        {"name": "experts one token", "op": "experts", "rows": 2, "groups": 64, "cols": 2048, "inner": 1024, "spare": 0, "dtype": "bfloat16"},
        # a decoding batch of 64 tokens, two experts each: every expert's matrix is read for a few rows
        {"name": "experts 64 tokens", "op": "experts", "rows": 128, "groups": 8, "cols": 14336, "inner": 4096, "spare": 0, "dtype": "bfloat16"},
        # the largest: a prompt (or training batch) of 8192 routed rows through the wide projection
        {"name": "experts 8192 rows", "op": "experts", "rows": 8192, "groups": 8, "cols": 14336, "inner": 4096, "spare": 0, "dtype": "bfloat16"},
        # a training step's gradient for the tokens: many small experts, odd widths, a buffer of fixed capacity
        {"name": "tokens ragged", "op": "tokens", "rows": 3001, "groups": 32, "cols": 1416, "inner": 2040, "spare": 71, "dtype": "float16"},
        # the gradient for the experts' matrices of a batch of 8192 routed rows
        {"name": "weights 8192 rows", "op": "weights", "rows": 8192, "groups": 8, "cols": 4096, "inner": 4096, "spare": 0, "dtype": "bfloat16"},
        # the same of a short batch: sums of a few rows, experts without any
        {"name": "weights ragged", "op": "weights", "rows": 517, "groups": 32, "cols": 1416, "inner": 2040, "spare": 11, "dtype": "float16"},
        # one new token of one request
        {"name": "adapters one token", "op": "adapters", "rows": 1, "requests": 1, "adapters": 4, "rank": 8, "cols": 4096, "inner": 4096, "dtype": "float16"},
        # a decoding batch: 64 requests of one token, 32 adapters among them
        {"name": "adapters 64 requests", "op": "adapters", "rows": 64, "requests": 64, "adapters": 32, "rank": 16, "cols": 4096, "inner": 4096, "dtype": "bfloat16"},
        # prompts of eleven requests in one batch
        {"name": "adapters 4100 tokens", "op": "adapters", "rows": 4100, "requests": 11, "adapters": 5, "rank": 64, "cols": 4096, "inner": 4096, "dtype": "bfloat16"},
        # the forward pass of a training batch, and what the backward pass reads in place of the input
        {"name": "keep 8192 tokens", "op": "keep", "rows": 8192, "cols": 4096, "dtype": "bfloat16", "weights": "float32"},
        # its backward pass
        {"name": "keep gradient 8192 tokens", "op": "keep_grad", "rows": 8192, "cols": 4096, "dtype": "bfloat16", "weights": "float32"},
        # a short ragged batch of odd width: rows start anywhere and end inside a block of 32
        {"name": "keep gradient ragged", "op": "keep_grad", "rows": 517, "cols": 1021, "dtype": "float16", "weights": "float16"},
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(lo, min(hi, int(round(v / step)) * step))

    op = rng.choice(["experts", "tokens", "weights", "adapters", "keep", "keep_grad"])
    if op in ("keep", "keep_grad"):
        dtype = rng.choice(["float16", "bfloat16", "float32"])
        return {"op": op, "rows": size(1, 8192), "cols": size(64, 4096), "dtype": dtype, "weights": rng.choice([dtype, "float32"])}
    dtype = rng.choice(["float16", "bfloat16"])
    if op == "adapters":
        rows = size(1, 4096)
        return {"op": op, "rows": rows, "requests": size(1, min(rows, 128)), "adapters": size(1, 32), "rank": rng.choice([8, 16, 24, 32, 64, 128]),
                "cols": size(64, 8192, 8), "inner": size(64, 4096, 8), "dtype": dtype}
    groups, cols, inner = size(1, 64), size(64, 14336, 8), size(64, 4096, 8)
    while groups * cols * inner > 8 * 14336 * 4096:
        groups = (groups + 1) // 2
    return {"op": op, "rows": size(1, 8192), "groups": groups, "cols": cols, "inner": inner, "spare": rng.choice([0, 0, 13]), "dtype": dtype}


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _offsets(case, seed):
    """Where each group's rows start, and the last one's end: the choices of a router that likes some
    experts better than others."""
    rng = random.Random(int(seed) * 7919 + 17)
    liked = [math.exp(0.6 * rng.gauss(0, 1)) for _ in range(case["groups"])]
    counts = [0] * case["groups"]
    for e in rng.choices(range(case["groups"]), liked, k=case["rows"]):
        counts[e] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    return offsets


def _requests(case, seed):
    """Where each request's rows start, and its adapter: lengths of at least one token."""
    rng = random.Random(int(seed) * 6007 + 5)
    cuts = sorted(rng.sample(range(1, case["rows"]), case["requests"] - 1))
    adapters = [rng.randrange(-1, case["adapters"]) for _ in range(case["requests"])]
    adapters[0] = rng.randrange(case["adapters"])
    return [0, *cuts, case["rows"]], adapters


def _randn(gen, shape, size, dtype):
    return (size * torch.randn(shape, generator=gen, device="cuda")).to(dtype)


def _stream(gen, rows, cols, dtype):
    """A residual stream: unit variance, an offset, a few channels far larger than the rest."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    loud = torch.rand(cols, generator=gen, device="cuda") < 0.002
    return ((x + 0.3) * torch.where(loud, 12.0, 1.0)).to(dtype)


def _matrices(gen, groups, cols, inner, dtype):
    """One matrix for each group, made one by one (32 bits of them all would take the card's time)."""
    b = torch.empty(groups, cols, inner, device="cuda", dtype=dtype)
    for e in range(groups):
        b[e] = 0.02 * torch.randn(cols, inner, generator=gen, device="cuda")
    return b


def _kept(gen, rows, cols):
    """What the forward pass keeps: E4M3 codes of normalised rows and a scale code for 32 of them."""
    h = _stream(gen, rows, cols, torch.float32)
    h = (h - h.mean(1, keepdim=True)) / h.std(1, keepdim=True, unbiased=False).clamp(min=1e-3)
    return _to_codes(h)


def prepare(case, seed):
    gen = _generator(seed)
    dtype, op = DTYPES[case["dtype"]], case["op"]
    s = {"case": case}
    if op in ("experts", "tokens", "weights"):
        offsets = _offsets(case, seed)
        rows = case["rows"] + case["spare"]
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        s["most"] = max(b - a for a, b in zip(offsets, offsets[1:]))
        if op != "tokens":
            s["a"] = _randn(gen, (rows, case["inner"]), 1.0, dtype)
        if op != "experts":
            s["dd"] = _randn(gen, (rows, case["cols"]), 0.1, dtype)
        if op != "weights":
            s["b"] = _matrices(gen, case["groups"], case["cols"], case["inner"], dtype)
        if case["spare"]:  # what a buffer of fixed capacity holds behind its rows
            for name in ("a", "dd"):
                if name in s:
                    s[name][case["rows"]:] = math.nan
        return s
    if op == "adapters":
        offsets, adapters = _requests(case, seed)
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        s["adapters"] = torch.tensor(adapters, dtype=torch.int32, device="cuda")
        s["x"] = _randn(gen, (case["rows"], case["inner"]), 1.0, dtype)
        s["w"] = _randn(gen, (case["cols"], case["inner"]), 0.02, dtype)
        s["down"] = _randn(gen, (case["adapters"], case["rank"], case["inner"]), case["inner"] ** -0.5, dtype)
        s["up"] = _randn(gen, (case["adapters"], case["cols"], case["rank"]), 0.05, dtype)
        s["scales"] = 0.5 + 1.5 * torch.rand(case["adapters"], generator=gen, device="cuda")
        return s
    wtype = DTYPES[case["weights"]]
    s["weight"] = (1 + 0.1 * torch.randn(case["cols"], generator=gen, device="cuda")).to(wtype)
    s["bias"] = (0.1 * torch.randn(case["cols"], generator=gen, device="cuda")).to(wtype)
    if op == "keep":
        s["x"] = _stream(gen, case["rows"], case["cols"], dtype)
    else:
        s["dy"] = _stream(gen, case["rows"], case["cols"], dtype)
        s["codes"], s["scales"] = _kept(gen, case["rows"], case["cols"])
        s["rstd"] = 0.5 + torch.rand(case["rows"], generator=gen, device="cuda")
    return s


# -------------------------------------------------------------- plain form --

def _group_of(offsets, rows):
    """The group of each row; the number of groups for rows behind the last one."""
    at = torch.arange(rows, device=offsets.device)
    return (at[:, None] >= offsets[None, 1:].long()).sum(1)


def _by_group(t, offsets, most):
    """[rows, n] as [groups, most, n] in 32 bits, zeros past a group's rows."""
    at = offsets[:-1, None].long() + torch.arange(most, device=t.device)
    there = at < offsets[1:, None].long()
    return torch.where(there[:, :, None], t[at.clamp(max=t.shape[0] - 1)].float(), 0.0)


def _by_row(t, offsets, rows):
    """The other way."""
    group = _group_of(offsets, rows)
    last = offsets.numel() - 1
    e = group.clamp(max=last - 1)
    at = torch.arange(rows, device=t.device) - offsets.long()[e]
    return torch.where((group < last)[:, None], t[e, at.clamp(0, t.shape[1] - 1)], 0.0)


def _to_codes(h):
    """h in 32 bits as E4M3 codes [rows, cols] and E8M0 codes [rows, blocks of 32]."""
    rows, cols = h.shape
    blocks = torch.nn.functional.pad(h, (0, -cols % 32)).reshape(rows, -1, 32)
    amax = blocks.abs().amax(2)
    e = ((amax.view(torch.int32) >> 23) - 127 - 8).clamp(-127, 127)
    q = torch.ldexp(blocks, -e[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.reshape(rows, -1)[:, :cols].contiguous(), (e + 127).to(torch.uint8)


def _from_codes(codes, scales):
    cols = codes.shape[1]
    e = (scales.int() - 127).repeat_interleave(32, 1)[:, :cols]
    return torch.ldexp(codes.float(), e)


def _again(case):
    """The type of the result from kept rows: that of the products it goes into."""
    return torch.bfloat16 if case["dtype"] == "float32" else DTYPES[case["dtype"]]


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    dtype = DTYPES[case["dtype"]]
    if op in ("experts", "tokens", "weights"):
        offsets, most, rows = s["offsets"], s["most"], case["rows"] + case["spare"]
        if op == "experts":
            d = torch.bmm(_by_group(s["a"], offsets, most), s["b"].float().transpose(1, 2))
            return {"d": _by_row(d, offsets, rows).to(dtype)}
        if op == "tokens":
            d = torch.bmm(_by_group(s["dd"], offsets, most), s["b"].float())
            return {"da": _by_row(d, offsets, rows).to(dtype)}
        return {"db": torch.bmm(_by_group(s["dd"], offsets, most).transpose(1, 2), _by_group(s["a"], offsets, most)).to(dtype)}
    if op == "adapters":
        x, rank, count = s["x"].float(), case["rank"], case["adapters"]
        adapter = s["adapters"][_group_of(s["offsets"], case["rows"])]
        chosen = adapter[:, None] == torch.arange(count, device=x.device)
        h = (x @ s["down"].float().reshape(count * rank, -1).T).reshape(-1, count, rank)
        h = h * torch.where(chosen, s["scales"], 0.0)[:, :, None]
        up = s["up"].float().transpose(1, 2).reshape(count * rank, -1)
        return {"d": (x @ s["w"].float().T + h.reshape(-1, count * rank) @ up).to(dtype)}
    if op == "keep":
        x = s["x"].float()
        centred = x - x.mean(1, keepdim=True)
        rstd = (centred.square().mean(1, keepdim=True) + EPS).rsqrt()
        h = centred * rstd
        weight, bias = s["weight"].float(), s["bias"].float()
        again = _from_codes(*_to_codes(h)) * weight + bias
        return {"y": (h * weight + bias).to(dtype), "rstd": rstd[:, 0], "again": again.to(_again(case))}
    dy, rstd, h = s["dy"].float(), s["rstd"][:, None], _from_codes(s["codes"], s["scales"])
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    wtype = s["weight"].dtype
    return {"dx": dx.to(dtype), "dweight": (dy * h).sum(0).to(wtype), "dbias": dy.sum(0).to(wtype)}


def run(state):
    if not own:
        return _plain(state)
    import blackwell_tensor_core_02_gb300 as g

    s, op = state, state["case"]["op"]
    if op == "experts":
        return {"d": g.grouped_gemm_nt(s["a"], s["b"], s["offsets"])}
    if op == "tokens":
        return {"da": g.grouped_gemm_nn(s["dd"], s["b"], s["offsets"])}
    if op == "weights":
        return {"db": g.grouped_gemm_tn(s["dd"], s["a"], s["offsets"])}
    if op == "adapters":
        return {"d": g.gemm_lora_nt(s["x"], s["w"], s["down"], s["up"], s["offsets"], s["adapters"], scales=s["scales"])}
    if op == "keep":
        y, kept, rstd = g.layer_norm_checkpoint(s["x"], s["weight"], s["bias"], EPS)
        return {"y": y, "rstd": rstd, "again": g.layer_norm_restore(kept, s["weight"], s["bias"], _again(s["case"]))}
    kept = g.Fp8Rows(s["codes"], s["scales"])
    dx, dweight, dbias = g.layer_norm_backward_checkpoint(s["dy"], kept, s["weight"], s["rstd"])
    return {"dx": dx, "dweight": dweight, "dbias": dbias}


# -------------------------------------------------------------------- work --

def work(case):
    rows, cols, size, op = case["rows"], case["cols"], SIZE[case["dtype"]], case["op"]
    if op in ("experts", "tokens"):  # the rows in and out, the matrices of the groups that have any
        some = min(case["groups"], rows)
        return {"bytes": size * (rows * (cols + case["inner"]) + some * cols * case["inner"]), "flops": 2 * rows * cols * case["inner"]}
    if op == "weights":
        return {"bytes": size * (rows * (cols + case["inner"]) + case["groups"] * cols * case["inner"]), "flops": 2 * rows * cols * case["inner"]}
    if op == "adapters":  # the rows in and out, the shared matrix, the adapters in use
        some, inner, rank = min(case["adapters"], case["requests"]), case["inner"], case["rank"]
        return {"bytes": size * (rows * (cols + inner) + cols * inner + some * rank * (cols + inner)),
                "flops": 2 * rows * (cols * inner + rank * (cols + inner))}
    if op == "keep":  # x and the weights in, y, the statistic and the result again out
        return {"bytes": rows * cols * (2 * size + 2) + 2 * cols * SIZE[case["weights"]] + 4 * rows, "flops": 12 * rows * cols}
    # dy, the kept rows, weight and statistic in, dx and the weights' gradients out
    return {"bytes": rows * (2 * cols * size + cols + -(-cols // 32) + 4) + 3 * cols * SIZE[case["weights"]], "flops": 14 * rows * cols}


# ------------------------------------------------------------ in 64 bits --

def _exact_kept(h):
    """The values of the kept rows from the formats' definitions: a block's scale, then each element
    to the nearest multiple of its own power of two."""
    rows, cols = h.shape
    full = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=h.device)
    full[:, :cols] = h
    b = full.view(rows, -1, 32)
    amax = b.abs().max(2, keepdim=True).values
    scale = torch.exp2((torch.frexp(amax).exponent - 9).clamp(-127, 127).double())
    t = b / scale
    ulp = torch.exp2((torch.frexp(t).exponent - 1).clamp(-6, 8).double() - 3)
    return (torch.clamp(torch.round(t / ulp) * ulp, -448, 448) * scale).view(rows, -1)[:, :cols]


def _exact_values(codes, scales):
    """Sign, exponent and mantissa of E4M3 codes, and their blocks' powers of two."""
    c = codes.view(torch.uint8).long()
    e, m = c // 8 % 16, (c % 8).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, torch.exp2(e.double() - 7) * (1 + m / 8)) * (1.0 - 2.0 * (c // 128).double())
    at = torch.arange(codes.shape[1], device=codes.device) // 32
    return v * torch.exp2(scales.double() - 127)[:, at]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("experts", "tokens", "weights"):
        offsets = _offsets(case, seed)
        spans = list(zip(offsets, offsets[1:]))
        if op == "weights":
            db = torch.zeros(case["groups"], case["cols"], case["inner"], dtype=torch.float64, device="cuda")
            for e, (i, j) in enumerate(spans):
                if j > i:
                    db[e] = torch.mm(s["dd"][i:j].double().t(), s["a"][i:j].double())
            return {"db": db}
        src, width, name = (s["a"], case["cols"], "d") if op == "experts" else (s["dd"], case["inner"], "da")
        out = torch.zeros(src.shape[0], width, dtype=torch.float64, device="cuda")
        for e, (i, j) in enumerate(spans):
            if j > i:
                m = s["b"][e].double()
                out[i:j] = torch.mm(src[i:j].double(), m.t() if op == "experts" else m)
        return {name: out}
    if op == "adapters":
        offsets, adapters = _requests(case, seed)
        x = s["x"].double()
        d = torch.mm(x, s["w"].double().t())
        for a, i, j in zip(adapters, offsets, offsets[1:]):
            if a >= 0:
                d[i:j] += float(s["scales"][a]) * torch.mm(torch.mm(x[i:j], s["down"][a].double().t()), s["up"][a].double().t())
        return {"d": d}
    n, w = case["cols"], s["weight"].double()
    if op == "keep":
        x, b = s["x"].double(), s["bias"].double()
        centred = x - (x.sum(1) / n)[:, None]
        rstd = 1 / torch.sqrt((centred ** 2).sum(1) / n + EPS)
        h = centred * rstd[:, None]
        return {"y": h * w + b, "rstd": rstd, "again": _exact_kept(h) * w + b}
    dy, rstd, h = s["dy"].double(), s["rstd"].double()[:, None], _exact_values(s["codes"], s["scales"])
    c1 = (dy * w).sum(1, keepdim=True) / n
    c2 = (dy * w * h).sum(1, keepdim=True) / n
    return {"dx": (dy * w - c1 - h * c2) * rstd, "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}
