"""Microscaled 4-bit floats on the GPU: quantisation bit for bit and the product against 64 bits."""
import pytest

import linear_reference as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TIMEOUT = -7


@pytest.fixture(scope="module")
def g(gpu_lib):
    gpu_lib.load_linear()
    return gpu_lib


def normal(seed, rows, cols, dtype=F32, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=gen, device="cuda") * scale).to(dtype)


def check_quantize(g, x, fmt, exponent=0):
    q = g.quantize_fp4(x, fmt, exponent=exponent)
    codes, scales = ref.quantize(x, fmt, exponent)
    want = ref.pack(codes)
    assert q.data.shape == want.shape and (q.rows, q.cols, q.format, q.exponent) == (*x.shape, fmt, exponent)
    assert torch.equal(q.scales, ref.tile(scales))
    # a zero's sign is the input's; both codes of zero stand for it
    bad = q.data != want
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} bytes differ, first {bad.nonzero()[0].tolist()}"
    return q, codes, scales


SHAPES = [(1, 1), (1, 16), (1, 32), (3, 33), (127, 64), (128, 65), (129, 130), (2, 4096), (300, 1000), (257, 2088)]


@pytest.mark.parametrize("fmt,exponent", [("mx", 0), ("nv", 0), ("nv", -8), ("nv", 5)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES, ids=lambda v: str(v))
def test_quantize_bit_for_bit(g, rows, cols, dtype, fmt, exponent):
    x = normal(rows * cols, rows, cols, dtype, 3.0)
    if rows > 1:
        x[-1] = 0
    q, codes, scales = check_quantize(g, x, fmt, exponent)
    want = ref.values(codes, scales, fmt, exponent)[:, :cols]
    for out in (F32, BF16, F16):
        assert torch.equal(g.dequantize_fp4(q, out).double(), want.to(out).double())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_ties_and_every_scale(g, fmt):
    """Blocks whose elements are every tie of E2M1 and its neighbours, times powers of two over
    fp32's range (for "nv" over its scales' range), the block's largest set by the last element."""
    block = 32 if fmt == "mx" else 16
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=torch.float64, device="cuda")
    lo, hi = ((-140, 120) if fmt == "mx" else (-12, 8))
    rows = []
    for e in range(lo, hi):
        base = torch.cat([ties, -ties])
        v = base.repeat(block // 16)
        near = v.clone()
        near[::2] *= 1 + 2.0 ** -22
        near[1::2] *= 1 - 2.0 ** -22
        near[7::8] = near[7::8].sign() * 6
        rows += [v * 2.0 ** e, near * 2.0 ** e]
    check_quantize(g, torch.stack(rows).float(), fmt)


@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("fmt,exponent", [("mx", 0), ("nv", 0), ("nv", -8)])
def test_sign_of_zeros(g, fmt, exponent, dtype):
    """A zero of either sign, and a value too small for its block, keep their sign: in blocks of
    ordinary values, of zeros alone, at the end of a row, and where the scale is at its largest."""
    x = normal(12, 7, 100, dtype)
    x[0, ::3], x[1, 1::3], x[2], x[3] = -0.0, 0.0, -0.0, 0.0
    x[4, ::2], x[4, 1::2], x[6, 1:] = -6e-8, 6e-8, -0.0
    x[5, ::4], x[6, 0] = -0.0, 65504.0
    q, codes, scales = check_quantize(g, x, fmt, exponent)
    assert bool((q.data[2, :48] == 0x88).all()) and not q.data[2, 50:].any() and not q.data[3].any()
    want = ref.values(codes, scales, fmt, exponent)[:, :100]
    for out in (F32, BF16):
        v = g.dequantize_fp4(q, out)
        assert torch.equal(v.double(), want) and torch.equal(torch.signbit(v), torch.signbit(x))


@pytest.mark.parametrize("exponent", [-100, 100])
def test_extreme_exponents(g, exponent):
    x = normal(4, 8, 64) * 2.0 ** exponent
    check_quantize(g, x, "nv", exponent)
    check_quantize(g, normal(4, 8, 64) * 1e30, "nv", exponent)
    check_quantize(g, normal(4, 8, 64) * 1e-30, "nv", exponent)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_infinities_and_nan_poison_their_block(g, fmt):
    x = normal(5, 4, 256)
    x[0, 3], x[1, 100], x[2, 255] = float("nan"), float("inf"), float("-inf")
    q, codes, scales = check_quantize(g, x, fmt)
    v = g.dequantize_fp4(q)
    block = 32 if fmt == "mx" else 16
    for r, c in ((0, 3), (1, 100), (2, 255)):
        b = c // block * block
        assert v[r, b:b + block].isnan().all()
    assert int(v.isnan().sum()) == 3 * block
    other = g.quantize_fp4(normal(6, 40, 256), fmt)
    d = g.gemm_fp4_nt(q, other)
    assert d[:3].isnan().all() and torch.isfinite(d[3]).all()
    d = g.gemm_fp4_nt(other, q)
    assert d[:, :3].isnan().all() and torch.isfinite(d[:, 3]).all()


@pytest.mark.parametrize("gap,shift", [(8, 0), (5, 0), (0, 1), (16, 8)])
def test_strided_and_unaligned_rows(g, gap, shift):
    buf = normal(7, 1, 40 * (200 + gap) + shift, F16)[0]
    x = buf[shift:].view(40, 200 + gap)[:, :200]
    for fmt in ("mx", "nv"):
        q, codes, scales = check_quantize(g, x, fmt)
        out = torch.full((40, 200 + gap + 1), -7.0, dtype=F32, device="cuda")
        g.dequantize_fp4(q, out=out[:, :200])
        assert torch.equal(out[:, :200].double(), ref.values(codes, scales, fmt)[:, :200]) and bool((out[:, 200:] == -7).all())


@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols", [1, 2, 5, 7, 8, 9, 15, 17, 23, 25, 31, 40, 130, 500, 509, 512, 515, 525, 1037])
def test_values_into_rows_that_start_anywhere(g, cols, dtype):
    """Each offset of the first row within 16 bytes; nothing beside the rows is touched."""
    rows = 11
    q, codes, scales = check_quantize(g, normal(cols, rows, cols), "nv")
    want = ref.values(codes, scales, "nv")[:, :cols].to(dtype)
    for shift in range(8):
        for gap in (0, 3):
            buf = torch.full((rows * (cols + gap) + 64,), -7.0, dtype=dtype, device="cuda")
            inside = torch.zeros_like(buf, dtype=torch.bool)
            view = lambda t: t[32 + shift:32 + shift + rows * (cols + gap)].view(rows, cols + gap)[:, :cols]
            view(inside).fill_(True)
            g.dequantize_fp4(q, dtype, out=view(buf))
            assert torch.equal(view(buf), want), (shift, gap)
            assert bool((buf[~inside] == -7).all()), (shift, gap)


def test_empty_matrices(g):
    for rows, cols in ((0, 64), (5, 0), (0, 0)):
        q = g.quantize_fp4(torch.empty(rows, cols, dtype=F16, device="cuda"))
        assert g.dequantize_fp4(q).shape == (rows, cols)
    a = g.quantize_fp4(torch.empty(5, 0, dtype=F16, device="cuda"))
    b = g.quantize_fp4(torch.empty(7, 0, dtype=F16, device="cuda"))
    d = torch.full((5, 7), float("nan"), dtype=F16, device="cuda")
    assert not g.gemm_fp4_nt(a, b, d).any()
    none = g.quantize_fp4(torch.empty(0, 64, dtype=F16, device="cuda"))
    some = g.quantize_fp4(normal(1, 7, 64))
    assert g.gemm_fp4_nt(none, some).shape == (0, 7) and g.gemm_fp4_nt(some, none).shape == (7, 0)


# ------------------------------------------------------------------ product --

def operands(g, M, N, K, fmt, seed=0, exponents=(0, -6)):
    ea, eb = exponents if fmt == "nv" else (0, 0)
    x, w = normal(seed + M + 3 * K, M, K), normal(seed + N + 7 * K, N, K, scale=0.05)
    a, b = g.quantize_fp4(x, fmt, exponent=ea), g.quantize_fp4(w, fmt, exponent=eb)
    return a, b, ref.values(*ref.quantize(x, fmt, ea), fmt, ea), ref.values(*ref.quantize(w, fmt, eb), fmt, eb)


def check_product(g, M, N, K, fmt, dtype=F16, options=None, alpha=1.0):
    a, b, va, vb = operands(g, M, N, K, fmt)
    # rows on both sides of D keep what they hold
    buf = torch.full((M + 2, N), -7.0, dtype=dtype, device="cuda")
    d = g.gemm_fp4_nt(a, b, buf[1:M + 1], alpha=alpha, options=options)
    status, info = g.fp4_device_status()
    assert status == 0, (status, hex(info))
    want, bound = ref.product_bound(va, vb, dtype, alpha)
    err = (d.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((err / bound).max())}, first {bad.nonzero()[0].tolist()}"
    assert bool((buf[0] == -7).all()) and bool((buf[M + 1] == -7).all())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("tile,swap", [(16, 1), (16, 2), (32, 1), (32, 2), (64, 1), (64, 2), (128, 1), (128, 2), (256, 0)])
def test_one_tile_of_each_kind(g, fmt, tile, swap):
    other = min(tile, 128)
    M, N = (256, 256) if tile == 256 else ((128, other) if swap == 1 else (other, 128))
    for K in (64, 256, 1024):
        check_product(g, M, N, K, fmt, options=g.Fp4Options(tile=tile, swap=swap))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 130, 32), (3, 129, 33), (16, 1000, 520), (17, 257, 2088), (33, 128, 4096),
                                   (65, 385, 300), (130, 300, 256), (255, 511, 768), (500, 1529, 1000), (1000, 520, 96)])
def test_ragged_shapes_and_types(g, M, N, K, fmt):
    for dtype in (F16, BF16, F32):
        check_product(g, M, N, K, fmt, dtype)
        check_product(g, N, M, K, fmt, dtype)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("ks", [2, 4, 8])
@pytest.mark.parametrize("tile,swap", [(16, 2), (32, 1), (64, 2), (128, 1)])
def test_k_split_over_a_cluster(g, fmt, ks, tile, swap):
    M, N = (11, 700) if swap == 2 else (700, 150 if tile == 128 else 29)
    for K in (ks * 256, 2048 + 96, 8192):
        check_product(g, M, N, K, fmt, options=g.Fp4Options(tile=tile, swap=swap, cluster_k=ks))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype,N", [(F16, 1024), (BF16, 1000), (F32, 1024), (F16, 1001)])
@pytest.mark.parametrize("clusters", [1, 2, 3, 0])
def test_pairs_over_several_tiles(g, fmt, dtype, N, clusters):
    """A capped grid: each pair runs several tiles, both accumulators in turn."""
    check_product(g, 900, N, 1300, fmt, dtype, g.Fp4Options(tile=256, max_clusters=clusters))


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("N", [1, 6, 63, 64, 65, 127, 129, 135, 191, 193, 250, 257, 263, 320, 385, 511, 513])
def test_pairs_store_rows_that_start_anywhere(g, N, dtype):
    """D at each offset within 16 bytes holds the bits of whole aligned rows' product, and nothing
    beside it is touched."""
    M, K, whole = 300, 320, 520
    a, b, _, _ = operands(g, M, whole, K, "mx")
    options = g.Fp4Options(tile=256)
    want = g.gemm_fp4_nt(a, b, dtype=dtype, options=options)[:, :N]
    part = g.quantize_fp4(g.dequantize_fp4(b)[:N].contiguous(), "mx")
    for shift in range(8):
        buf = torch.full((M * N + 64,), -7.0, dtype=dtype, device="cuda")
        d = g.gemm_fp4_nt(a, part, buf[32 + shift:32 + shift + M * N].view(M, N), options=options)
        assert torch.equal(d, want), shift
        assert bool((buf[:32 + shift] == -7).all()) and bool((buf[32 + shift + M * N:] == -7).all()), shift


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_products_of_one_term_are_exact(g, fmt):
    """One element a row that is not zero: D holds the products of values, each exact."""
    n, K = 192, 512
    x, w = torch.zeros(n, K, device="cuda"), torch.zeros(n, K, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    at = torch.randint(0, K, (n,), generator=gen, device="cuda")
    x[torch.arange(n), at] = torch.randn(n, generator=gen, device="cuda")
    w[torch.arange(n), at] = torch.randn(n, generator=gen, device="cuda")
    a, b = g.quantize_fp4(x, fmt), g.quantize_fp4(w, fmt)
    va, vb = ref.values(*ref.quantize(x, fmt), fmt), ref.values(*ref.quantize(w, fmt), fmt)
    for options in (None, g.Fp4Options(tile=256), g.Fp4Options(tile=128), g.Fp4Options(tile=128, cluster_k=2)):
        assert torch.equal(g.gemm_fp4_nt(a, b, dtype=F32, options=options).double(), va @ vb.T)


def test_alpha_and_exponents(g):
    check_product(g, 100, 300, 512, "nv", F32, alpha=-0.37)
    check_product(g, 300, 600, 512, "mx", F16, alpha=3.0, options=g.Fp4Options(tile=256))


# exponents of A and B and alpha whose product leaves fp32's range, at its edges and inside it
FACTORS = [(64, 64, 1.0), (64, 63, 1.9), (100, 100, 1.0), (100, -100, 0.3), (-100, 100, -1.0), (-100, -50, 1.0),
           (-60, -70, 1 / 3), (-63, -63, 0.7), (-100, -100, 1.0), (90, 90, 1e-40), (-90, -90, 3e39), (0, 3, -1e-41), (-3, 0, 1e300),
           (0, 0, float("inf"))]


def one_term(exponent, seed, n=192, K=512):
    """Rows of one element that is not zero, near 2**exponent; the first and the last row zeros."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros(n, K, dtype=torch.float64, device="cuda")
    at = torch.randint(0, K, (n,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    v = torch.randn(n, generator=gen, device="cuda").double() * torch.exp2(torch.randint(-6, 9, (n,), generator=gen, device="cuda").double())
    x[torch.arange(n), at] = v * 2.0 ** exponent
    x[0] = x[-1] = 0
    return x.float()


def same(d, want):
    return torch.equal(d.isnan(), want.isnan()) and torch.equal(torch.where(d.isnan(), 0, d), torch.where(want.isnan(), 0, want))


@pytest.mark.parametrize("options", [{}, dict(tile=256), dict(tile=128, cluster_k=2), dict(tile=128, swap=2)], ids=str)
@pytest.mark.parametrize("ea,eb,alpha", FACTORS)
def test_exponents_whose_sum_leaves_fp32(g, ea, eb, alpha, options):
    """One term a row: the sum is exact in fp32, so D is the one rounding of the exact value, and 0
    (NaN for an infinite alpha) where the sum is 0."""
    x, w = one_term(ea, 1), one_term(eb, 2)
    a, b = g.quantize_fp4(x, "nv", exponent=ea), g.quantize_fp4(w, "nv", exponent=eb)
    exact = ref.values(*ref.quantize(x, "nv", ea), "nv", ea) @ ref.values(*ref.quantize(w, "nv", eb), "nv", eb).T
    m, e = torch.frexp(torch.tensor(alpha, dtype=torch.float64))
    exact = exact * (float(m.float()) * 2.0 ** min(int(e), 900) if alpha != float("inf") else alpha)
    for dtype in (F32, BF16, F16):
        d = g.gemm_fp4_nt(a, b, dtype=dtype, alpha=alpha, options=g.Fp4Options(**options))
        assert same(d, exact.float().to(dtype)), dtype
        # the last row of B left out: rows of D that start anywhere
        d = g.gemm_fp4_nt(a, b._replace(data=b.data[:191]), dtype=dtype, alpha=alpha, options=g.Fp4Options(**options))
        assert same(d, exact[:, :191].float().to(dtype)), dtype


@pytest.mark.parametrize("ea,eb", [(64, 64), (100, -100), (-100, -50), (-80, -48), (-100, -100)])
def test_sums_with_extreme_exponents(g, ea, eb):
    """Values near 2**(exponent - 8) and 2**(exponent + 8), a padding row of zeros on each side."""
    for shift in (-8, 8):
        x, w = (normal(20, 90, 700).double() * 2.0 ** (ea + shift)).float(), (normal(21, 300, 700).double() * 2.0 ** (eb + shift)).float()
        x[7] = w[5] = 0
        a, b = g.quantize_fp4(x, "nv", exponent=ea), g.quantize_fp4(w, "nv", exponent=eb)
        va, vb = ref.values(*ref.quantize(x, "nv", ea), "nv", ea), ref.values(*ref.quantize(w, "nv", eb), "nv", eb)
        for options in (None, g.Fp4Options(tile=256)):
            for dtype in (F32, BF16, F16):
                d = g.gemm_fp4_nt(a, b, dtype=dtype, options=options)
                want, bound = ref.product_bound(va, vb, dtype)
                over = d.isinf() & (want.abs() + bound >= torch.finfo(dtype).max) & (torch.sign(d) == torch.sign(want))
                assert bool(((d.double() - want).abs() <= bound).logical_or(over).all())
                assert not d[7].any() and not d[:, 5].any()


def test_the_products_factor(g):
    """alpha and the option's exponent are one factor; out-of-range ones are refused."""
    a, b, va, vb = operands(g, 40, 72, 320, "nv", exponents=(0, 0))
    want = g.gemm_fp4_nt(a, b, dtype=F32, alpha=0.375)
    for alpha, exponent in ((3.0, -3), (0.375 * 2.0 ** -90, 90), (1.5 * 2.0 ** 100, -102)):
        assert torch.equal(g.gemm_fp4_nt(a, b, dtype=F32, alpha=alpha, options=g.Fp4Options(exponent=exponent)), want)
    m = g.quantize_fp4(normal(1, 40, 320), "mx")
    for bad in (lambda: g.gemm_fp4_nt(a, b, options=g.Fp4Options(exponent=2 ** 31 - 1)),
                lambda: g.gemm_fp4_nt(a, b, options=g.Fp4Options(exponent=-(2 ** 31))),
                lambda: g.gemm_fp4_nt(a, b, alpha=0.5, options=g.Fp4Options(exponent=1001)),
                lambda: g.gemm_fp4_nt(m, m, options=g.Fp4Options(exponent=1))):
        with pytest.raises(g.GemmError):
            bad()
    with pytest.raises(ValueError):
        g.gemm_fp4_nt(m, m, alpha=1e39)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_large_product_in_its_default_tile(g, fmt):
    check_product(g, 2304, 3840, 1056, fmt)


def test_random_shapes(g):
    import random

    rng = random.Random(11)
    for i in range(60):
        M, N, K = (max(1, int(2 ** rng.uniform(0, 10.5))) for _ in range(3))
        options = None
        if i % 3:
            tile = rng.choice([16, 32, 64, 128, 256])
            options = g.Fp4Options(tile=tile)
            if tile != 256:
                options.swap, options.cluster_k = rng.choice([1, 2]), rng.choice([0, 1, 2, 4, 8])
                if tile < 128:
                    M, N = (M, min(N, tile)) if options.swap == 1 else (min(M, tile), N)
            else:
                options.max_clusters = rng.choice([0, 1, 5])
        check_product(g, M, N, K, rng.choice(["mx", "nv"]), rng.choice([F16, BF16, F32]), options)


def test_streams_and_graphs(g):
    a, b, _, _ = operands(g, 64, 2048, 2048, "nv")
    want = g.gemm_fp4_nt(a, b)
    x = normal(9, 64, 2048, F16)
    q = g.quantize_fp4(x, "nv")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        d = g.gemm_fp4_nt(a, b, stream=side)
        q2 = g.quantize_fp4(x, "nv", stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(d, want) and torch.equal(q.data, q2.data) and torch.equal(q.scales, q2.scales)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        q3 = g.quantize_fp4(x, "nv")
        d3 = g.gemm_fp4_nt(q3, b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(d3, g.gemm_fp4_nt(q, b))


def test_refusals_on_a_stream(g):
    """What a call refuses it refuses with stream= as well, by the same error."""
    x, side = normal(1, 8, 64, F16), torch.cuda.Stream()
    q = g.quantize_fp4(x, "mx")
    for bad in (lambda: g.dequantize_fp4(x, stream=side), lambda: g.gemm_fp4_nt(x, x, stream=side), lambda: g.gemm_fp4_nt(q, x, stream=side),
                lambda: g.gemm_fp4_nt(3, q, stream=side), lambda: g.quantize_fp4(x, out=x, stream=side),
                lambda: g.gemm_fp4_nt(q, q, options=g.Options(), stream=side)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        g.quantize_fp4(x, "nv", out=q, stream=side)
    assert torch.equal(g.dequantize_fp4(q, stream=side), g.dequantize_fp4(q))


def test_chain_of_dependent_calls(g):
    """Each call reads what the one before wrote, with overlapped launches between them."""
    w = g.quantize_fp4(normal(1, 512, 512, scale=0.06), "mx")
    x = normal(2, 40, 512, F16)
    outs = []
    for wait in (True, False):
        y = x
        for _ in range(20):
            y = g.layer_norm(g.gemm_fp4_nt(g.quantize_fp4(y, "mx"), w))[0]
            if wait:
                torch.cuda.synchronize()
        outs.append(y)
    assert torch.equal(*outs) and torch.isfinite(outs[0].float()).all()


@pytest.mark.parametrize("options", [dict(tile=16, swap=2), dict(tile=64, swap=2, cluster_k=4), dict(tile=128), dict(tile=256)])
def test_waits_run_out_and_the_context_survives(g, options):
    a, b, va, vb = operands(g, 16, 512, 2048, "mx")
    g.gemm_fp4_nt(a, b, options=g.Fp4Options(debug_flags=1, timeout_ns=50_000_000, **options))
    status, info = g.fp4_device_status()
    assert status == TIMEOUT and info >> 56 in (1, 2, 3)
    assert g.fp4_device_status()[0] == 0
    d = g.gemm_fp4_nt(a, b, options=g.Fp4Options(**options))
    want, bound = ref.product_bound(va, vb, F16)
    assert bool(((d.double() - want).abs() <= bound).all()) and g.fp4_device_status()[0] == 0


def test_refusals(g):
    x = normal(1, 8, 64, F16)
    q, n = g.quantize_fp4(x, "mx"), g.quantize_fp4(x, "nv")
    for bad in (lambda: g.quantize_fp4(x, "e4m3"), lambda: g.quantize_fp4(x, "mx", exponent=1),
                lambda: g.quantize_fp4(x, "nv", exponent=101), lambda: g.quantize_fp4(x[0]), lambda: g.quantize_fp4(x.t()),
                lambda: g.quantize_fp4(x.cpu()), lambda: g.quantize_fp4(x, "nv", out=q), lambda: g.gemm_fp4_nt(q, n),
                lambda: g.gemm_fp4_nt(q, g.quantize_fp4(x[:, :32], "mx")), lambda: g.gemm_fp4_nt(q, q, torch.empty(8, 9, device="cuda")),
                lambda: g.gemm_fp4_nt(q._replace(cols=200), q), lambda: g.gemm_fp4_nt(q._replace(scales=n.scales[:0]), q),
                lambda: g.dequantize_fp4(q, out=torch.empty(8, 63, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: g.quantize_fp4(x.double()), lambda: g.gemm_fp4_nt(q, q, dtype=torch.int8),
                lambda: g.dequantize_fp4(q, torch.float64), lambda: g.gemm_fp4_nt(q._replace(data=q.data.view(torch.int8)), q)):
        with pytest.raises(TypeError):
            bad()
    wide = g.quantize_fp4(normal(1, 40, 64, F16))
    for options in (dict(tile=48), dict(cluster_k=3), dict(swap=3), dict(max_clusters=-1), dict(debug_flags=2), dict(timeout_ns=-1),
                    dict(tile=256, cluster_k=2), dict(tile=256, swap=1), dict(tile=16, swap=1)):
        with pytest.raises(g.GemmError):
            g.gemm_fp4_nt(wide, wide, options=g.Fp4Options(**options))
    with pytest.raises(g.GemmError):  # D over A
        buf = torch.zeros(8 * 32 + 512, dtype=torch.uint8, device="cuda")
        a = g.Fp4Tensor(buf[:256].view(8, 32), q.scales, 64)
        g.gemm_fp4_nt(a, q, buf[:128].view(F16).view(8, 8))
