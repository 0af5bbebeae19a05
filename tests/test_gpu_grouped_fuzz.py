"""Random sizes, offsets, options, strides and values of the grouped products, adapters and checkpoints
against their definitions in 64 bits, with what lies around operands and results.

GROUPED_FUZZ_CASES and GROUPED_FUZZ_SEED (environment) change the number of cases of each of the three series
and the seed, for longer sweeps; the defaults are 40 and 2026."""
import math
import os
import random

import pytest

import checkpoint_reference as cref
import grouped_reference as gref
import linear_reference as lref
from test_gpu_lora_range import want as far_adapters

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
CASES, SEED = int(os.environ.get("GROUPED_FUZZ_CASES", "40")), int(os.environ.get("GROUPED_FUZZ_SEED", "2026"))
NAN = float("nan")


class Draw:
    def __init__(self, kind, i):
        self.rng = random.Random(f"{kind} {SEED} {i}")
        self.gen = torch.Generator(device="cuda").manual_seed(SEED * 100003 + i)

    def choice(self, *of):
        return self.rng.choice(of)

    def size(self, most, unit=8):
        if self.rng.random() < 0.3:
            return unit * self.rng.randint(1, max(1, 40 // unit))
        return unit * max(1, int(2 ** self.rng.uniform(0, math.log2(max(2, most / unit)))))

    def slab(self, shape, dtype, scale=1.0, unit=8, fill=NAN):
        """(a tensor of that shape inside a larger one that holds `fill`, the larger one); `scale`: of its
        random values, None for `fill`."""
        big = [s + (0 if self.rng.random() < 0.5 else unit * self.rng.randint(1, 4)) for s in shape]
        lead, strides, step = unit * self.choice(0, 0, 1, 5), [], 1
        for b in reversed(big):
            strides.insert(0, step)
            step *= b
        whole = torch.full((step + lead + 64,), fill, dtype=dtype, device="cuda")
        view = whole.as_strided(shape, strides, lead)
        if scale is not None:
            view.copy_(torch.randn(shape, generator=self.gen, device="cuda") * scale)
        return view, whole

    def offsets(self, groups, rows):
        """Cuts, most often sorted and within the rows, as a list and as either type on the device."""
        k = self.rng.random()
        if k < 0.6:
            cuts = sorted(self.rng.randint(0, rows) for _ in range(groups + 1))
            if self.rng.random() < 0.6 and groups:
                cuts[0], cuts[-1] = 0, rows
        elif k < 0.8:
            cuts = [min(rows, e * (rows // max(groups, 1))) for e in range(groups + 1)]
        elif k < 0.9:
            some = self.rng.randint(0, rows)
            cuts = sorted(self.choice(0, some, rows) for _ in range(groups + 1))
        else:
            cuts = [self.rng.randint(-5, rows + 9) for _ in range(groups + 1)]
        return cuts, torch.tensor(cuts, dtype=self.choice(torch.int32, torch.int64), device="cuda")

    def options(self, g, kind):
        if self.rng.random() < 0.4:
            return None
        if kind == "tn":
            o = self.choice(dict(tile=self.choice(0, 64, 128, 256), split=self.choice(0, -1)),
                            dict(tile=self.choice(64, 128), split=self.choice(1, 2, 4, 8)))
        elif kind == "adapters":
            o = self.choice(dict(tile=256), dict(split=-1), dict(tile=self.choice(0, 16, 32, 64, 128), split=self.choice(0, 1, 2, 4, 8)))
        else:
            o = self.choice(dict(tile=self.choice(0, 32, 64, 128, 256), split=-1), dict(tile=256),
                            dict(tile=self.choice(0, 16, 32, 64, 128), split=self.choice(0, 1, 2, 4, 8)))
        return g.GroupedOptions(**o, max_clusters=self.choice(0, 0, 1, 7, 300), timeout_ns=2_000_000_000)


def near(got, want, far):
    off = (got.double() - want).abs()
    assert bool((off <= far).all()), ((~(off <= far)).nonzero()[:4].tolist(), float((off - far).max()))


def untouched(whole, view, fill):
    view.fill_(fill)
    assert bool((whole == fill).all())


@pytest.mark.parametrize("i", range(CASES))
def test_grouped_products(gpu_lib, i):
    g, d = gpu_lib, Draw("grouped", i)
    dtype = d.choice(F16, BF16)
    groups = d.choice(1, 2, 3, 8, d.rng.randint(0, 60), d.rng.randint(1, 300))
    rows = d.choice(1, d.rng.randint(0, 40), int(2 ** d.rng.uniform(0, 12.5)))
    N, K = d.size(1600), d.size(1600)
    groups = min(groups, max(1, 2 ** 26 // (N * K)))
    cuts, offsets = d.offsets(groups, rows)
    A, dD, B = d.slab((rows, K), dtype)[0], d.slab((rows, N), dtype)[0], d.slab((groups, N, K), dtype, 0.1)[0]
    ends = gref.clamp(cuts, rows)
    first, last = ends[0], ends[-1]
    if d.rng.random() < 0.5:  # rows without a group hold anything
        A[:first], A[last:], dD[:first], dD[last:] = NAN, float("inf"), float("inf"), NAN
    for kind in ("nt", "nn", "tn"):
        o, given = d.options(g, kind), d.rng.random() < 0.5
        if kind == "tn":
            out, whole = d.slab((groups, N, K), dtype, None, fill=7.0)
            near(g.grouped_gemm_tn(dD, A, offsets, out if given else None, options=o), *gref.matrices(dD, A, cuts))
        else:
            x, call, width = (A, g.grouped_gemm_nt, N) if kind == "nt" else (dD, g.grouped_gemm_nn, K)
            out, whole = d.slab((rows, width), dtype, None, fill=7.0)
            got = call(x, B, offsets, out if given else None, options=o)
            want, far = gref.product(x, B, cuts, kind == "nt")
            near(got[first:last], want[first:last], far[first:last])
            if not given:
                assert not bool(got[:first].any()) and not bool(got[last:].any())
            out = out[first:last]
        if given:
            untouched(whole, out, 7.0)
    assert g.grouped_device_status()[0] == 0


@pytest.mark.parametrize("i", range(CASES))
def test_adapters(gpu_lib, i):
    g, d = gpu_lib, Draw("adapters", i)
    dtype, many = d.choice(F16, BF16), d.rng.randint(0, 9)
    requests = d.choice(1, 2, 4, d.rng.randint(0, 70), d.rng.randint(1, 600))
    rows = d.choice(1, d.rng.randint(0, 70), d.rng.randint(200, 300), int(2 ** d.rng.uniform(0, 11.5)))
    N, K, rank = d.size(1600), d.size(2500), d.choice(8, 16, 24, 32, 64, 72, 128, 8 * d.rng.randint(1, 16))
    cuts, offsets = d.offsets(requests, rows)
    if d.rng.random() < 0.3 and 0 < rows <= 1024:  # a row each
        requests, cuts = rows, list(range(rows + 1))
        offsets = torch.tensor(cuts, device="cuda", dtype=torch.int32)
    x, W = d.slab((rows, K), dtype)[0], d.slab((N, K), dtype, 0.05)[0]
    down, up = d.slab((many, rank, K), dtype, K ** -0.5)[0], d.slab((many, N, rank), dtype, 0.3)[0]
    scales = None if d.rng.random() < 0.3 else torch.rand(many, device="cuda", generator=d.gen) + 0.5
    chosen = [d.rng.randint(-1, d.choice(1, max(many, 1), many + 2)) for _ in range(requests)]
    reference = gref.adapters
    if scales is not None and dtype == F16 and d.rng.random() < 0.5:  # h far from 1, by up's size or not
        for a in range(many):
            e = d.rng.randint(-12, 12)
            scales[a] *= 2.0 ** (2 * e)
            up[a] *= 2.0 ** -e
        scales *= 2.0 ** d.rng.randint(-3, 0)
        x *= torch.exp2(-torch.randint(0, 12, (rows, 1), generator=d.gen, device="cuda").float()).half()
        chosen = [a if a < many else -1 for a in chosen]
        reference = far_adapters
    adapters, o = torch.tensor(chosen, dtype=torch.int32, device="cuda"), d.options(g, "adapters")
    out, whole = d.slab((rows, N), dtype, None, fill=7.0)
    given = d.rng.random() < 0.5
    got = g.gemm_lora_nt(x, W, down, up, offsets, adapters, out if given else None, scales=scales, options=o)
    want, far = reference(x, W, down, up, cuts, chosen, scales)
    # values that round past fp16's largest are infinities of their sign
    near(torch.where(want.abs() + far < 65519, got.double(), 0.0) if dtype == F16 else got,
         torch.where(want.abs() + far < 65519, want, 0.0) if dtype == F16 else want, far)
    if given:
        untouched(whole, out, 7.0)
    assert g.grouped_device_status()[0] == 0


@pytest.mark.parametrize("i", range(CASES))
def test_checkpoints(gpu_lib, i):
    g, d = gpu_lib, Draw("checkpoints", i)
    dtype = d.choice(F16, BF16, F32)
    wdtype = d.choice(None, dtype, F32)
    cols = d.choice(d.rng.randint(1, 70), d.size(9000), d.rng.randint(1, 9000), d.choice(16384, 16385, 12288, 17000, 20480))
    rows = d.choice(1, d.rng.randint(0, 20), max(1, int(2 ** d.rng.uniform(0, 22) / cols)))
    x, dy = (d.slab((rows, cols), dtype, s, unit=d.choice(1, 2, 8))[0] for s in (2.0, 1.0))
    x += d.choice(0, 0.5, 30)
    w = b = None
    if wdtype is not None:
        if d.rng.random() < 0.9:
            w = d.slab((cols,), wdtype, 0.2, unit=d.choice(1, 8))[0].add_(1.0)
        if d.rng.random() < 0.9:
            b = d.slab((cols,), wdtype, 0.3, unit=d.choice(1, 8))[0]
    eps = d.choice(1e-5, 1e-3, 0.0 if cols > 4 else 1e-5)
    (out, whole), given = d.slab((rows, cols), dtype, None, unit=d.choice(1, 2, 8), fill=7.0), d.rng.random() < 0.5
    y, kept, rstd = g.layer_norm_checkpoint(x, w, b, eps, out=out if given else None)
    if rows:
        want, _, want_rstd = lref.norm(x, w, b, eps)
        far, _, far_rstd = lref.norm_bounds(x, w, b, eps, dtype)
        near(y, want, far)
        near(rstd, want_rstd, far_rstd)
        cref.check_kept(kept, *cref.h_bounds(x, eps))
    if given:
        untouched(whole, out, 7.0)
    if rows > 2 and d.rng.random() < 0.3:  # some of the rows
        k = d.rng.randint(1, rows - 1)
        kept, rstd, dy, rows = g.Fp8Rows(kept.codes[k:], kept.scales[k:]), rstd[k:], dy[k:], rows - k
    t = d.rng.choice([t for t in (F16, BF16, F32) if all(v is None or v.dtype in (t, F32) for v in (w, b))])
    out, whole = d.slab((rows, cols), t, None, unit=d.choice(1, 2, 8), fill=7.0)
    got = g.layer_norm_restore(kept, w, b, t, out=out if given else None)
    if rows:
        near(got, *cref.restore(kept, w, b, t))
    if given:
        untouched(whole, out, 7.0)
    out, whole = d.slab((rows, cols), dtype, None, unit=d.choice(1, 2, 8), fill=7.0)
    grad_dtype = None if w is not None else d.choice(None, F32, dtype)
    grads = g.layer_norm_backward_checkpoint(dy, kept, w, rstd, dx=out if given else None, grad_dtype=grad_dtype)
    if rows:
        h, wd = cref.values(kept), grad_dtype or (dy.dtype if w is None else w.dtype)
        for got, want, far in zip(grads, cref.grad(dy, h, w, rstd), cref.grad_bounds(dy, h, w, rstd, dtype, wd)):
            if got is not None:
                near(got, want, far)
    if given:
        untouched(whole, out, 7.0)
