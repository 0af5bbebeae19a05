"""Layer norm with 8-bit checkpoints on the GPU: what it keeps, its result and its gradient from that."""
import pytest

import checkpoint_reference as ref
import linear_reference as lref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g(gpu_lib):
    gpu_lib.load_linear()
    return gpu_lib


def normal(seed, shape, dtype, scale=1.0, offset=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale + offset).to(dtype)


def near(got, want, far, what=""):
    off = (got.double() - want).abs()
    assert bool((off <= far).all()), (what, float((off - far).max()), (off > far).nonzero()[:3].tolist())


def parameters(cols, wdtype, seed=5):
    if wdtype is None:
        return None, None
    return normal(seed, (cols,), wdtype, 0.2, 1.0), normal(seed + 1, (cols,), wdtype, 0.3)


def check_forward(g, x, weight, bias, eps=1e-5, **k):
    y, kept, rstd = g.layer_norm_checkpoint(x, weight, bias, eps, **k)
    rows = x.reshape(-1, x.shape[-1])
    want, _, want_rstd = lref.norm(rows, weight, bias, eps)
    far, _, far_rstd = lref.norm_bounds(rows, weight, bias, eps, x.dtype)
    near(y.reshape(rows.shape), want, far, "y")
    near(rstd.reshape(-1), want_rstd, far_rstd, "rstd")
    h, e = ref.h_bounds(rows, eps)
    assert kept.codes.shape == x.shape and kept.scales.shape == (*x.shape[:-1], -(-x.shape[-1] // 32))
    ref.check_kept(kept, h, e)
    return y, kept, rstd


def check_backward(g, dy, kept, weight, rstd, **k):
    dx, dweight, dbias = g.layer_norm_backward_checkpoint(dy, kept, weight, rstd, **k)
    wdtype = k.get("grad_dtype") or (dy.dtype if weight is None else weight.dtype)
    rows = dy.reshape(-1, dy.shape[-1])
    h, r = ref.values(kept).reshape(rows.shape), rstd.reshape(-1)
    want, far = ref.grad(rows, h, weight, r), ref.grad_bounds(rows, h, weight, r, dy.dtype, wdtype)
    near(dx.reshape(rows.shape), want[0], far[0], "dx")
    if dweight is not None:
        near(dweight, want[1], far[1], "dweight")
        near(dbias, want[2], far[2], "dbias")
    return dx, dweight, dbias


# widths on both sides of a block, of whole units, of each row shape and of the ring's end
WIDTHS = [1, 7, 8, 31, 32, 33, 64, 100, 255, 256, 257, 512, 760, 769, 1000, 1021, 1024, 1025, 2047, 2048, 3000, 4096, 5003,
          6144, 8192, 8193, 8200, 12288, 12300, 16384, 16392, 20001]


@pytest.mark.parametrize("dtype,wdtype", [(F16, F16), (BF16, F32), (F32, F32), (BF16, None)], ids=["f16", "bf16-f32", "f32", "bf16-none"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_widths(g, cols, dtype, wdtype):
    rows = 5 if cols > 4096 else 37
    x = normal(cols, (rows, cols), dtype, 2.0, 0.4)
    weight, bias = parameters(cols, wdtype)
    _, kept, rstd = check_forward(g, x, weight, bias)
    dy = normal(cols + 1, (rows, cols), dtype)
    check_backward(g, dy, kept, weight, rstd, grad_dtype=None if weight is not None else F32)
    for out in (F16, BF16, F32):
        if wdtype in (None, out, F32):
            near(g.layer_norm_restore(kept, weight, bias, out), *ref.restore(kept, weight, bias, out))


@pytest.mark.parametrize("rows", [1, 2, 3, 151, 152, 153, 1000, 5000])
@pytest.mark.parametrize("cols", [64, 69, 1024, 2056])
def test_rows(g, rows, cols):
    x = normal(rows, (rows, cols), BF16, 1.0, 0.2)
    weight, bias = parameters(cols, BF16)
    _, kept, rstd = check_forward(g, x, weight, bias)
    check_backward(g, normal(rows + 1, (rows, cols), BF16), kept, weight, rstd)
    near(g.layer_norm_restore(kept, weight, bias, BF16), *ref.restore(kept, weight, bias, BF16))


@pytest.mark.parametrize("dtype", [F16, F32], ids=["f16", "f32"])
@pytest.mark.parametrize("cols,gap,first", [(64, 8, 0), (64, 3, 0), (64, 8, 1), (100, 1, 5), (2048, 16, 8), (2048, 16, 3), (1021, 7, 1)])
def test_rows_inside_wider_ones(g, cols, gap, first, dtype):
    """Rows that lie apart and start anywhere, results into such rows: nothing beside them is written."""
    def inside(t, fill):
        big = torch.full((t.shape[0], t.shape[1] + gap + first), fill, dtype=t.dtype, device="cuda")
        view = big[:, first:first + t.shape[1]]
        view.copy_(t)
        return big, view
    rows = 19
    _, x = inside(normal(1, (rows, cols), dtype), float("nan"))
    _, dy = inside(normal(2, (rows, cols), dtype), float("nan"))
    weight, bias = parameters(cols, dtype)
    big, out = inside(torch.zeros(rows, cols, dtype=dtype, device="cuda"), 3.0)
    y, kept, rstd = check_forward(g, x, weight, bias, out=out)
    assert y.data_ptr() == out.data_ptr()
    out.fill_(3.0)
    assert bool((big == 3.0).all())
    check_backward(g, dy, kept, weight, rstd, dx=out)
    out.fill_(3.0)
    assert bool((big == 3.0).all())
    near(g.layer_norm_restore(kept, weight, bias, out=out), *ref.restore(kept, weight, bias, dtype))
    out.fill_(3.0)
    assert bool((big == 3.0).all())


def test_kept_rows_that_start_anywhere(g):
    """Kept rows from the middle of others: codes and scales at any byte."""
    for cols in (64, 100, 1021, 5003):
        whole = ref.keep(normal(cols, (12, cols), F32, 1.0))
        for first in (1, 2, 5):
            kept = g.Fp8Rows(whole[0][first:], whole[1][first:])
            dy, rstd = normal(7, (12 - first, cols), F16), normal(8, (12 - first,), F32).abs() + 0.1
            weight, bias = parameters(cols, F16)
            check_backward(g, dy, kept, weight, rstd)
            near(g.layer_norm_restore(kept, weight, bias, F16), *ref.restore(kept, weight, bias, F16))


def test_every_code_and_scale(g):
    """All codes under scales over fp32's range, in rows of whole units and others."""
    for cols in (256, 250):
        codes = torch.arange(cols, dtype=torch.uint8, device="cuda").repeat(6, 1)
        scales = torch.tensor([0, 1, 60, 127, 200, 255], dtype=torch.uint8, device="cuda")[:, None].repeat(1, 8)
        kept = g.Fp8Rows(codes.view(torch.float8_e4m3fn), scales)
        got, want = g.layer_norm_restore(kept, dtype=F32).double(), ref.values(kept)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got[~got.isnan()], want.float().double()[~want.isnan()])


@pytest.mark.parametrize("cols", [64, 100, 1024, 3001])
def test_blocks_of_any_size(g, cols):
    """Rows whose blocks differ by powers of two and hold zeros alone: each block has its own scale."""
    x = normal(3, (16, cols), F32)
    x *= torch.exp2(torch.randint(-12, 12, (16, -(-cols // 32)), device="cuda").float()).repeat_interleave(32, 1)[:, :cols]
    x[3] = 0
    x[5, 32:64] = x[5].mean()
    check_forward(g, x, None, None)
    check_forward(g, x.half(), None, None)


def test_zero_rows_and_constant_rows(g):
    x = torch.zeros(4, 96, dtype=BF16, device="cuda")
    x[1:3] = 7.0
    y, kept, rstd = check_forward(g, x, None, None)
    assert not bool(ref.values(kept).any()) and not bool(y.any()) and not bool(kept.scales.any())
    x[3, 5] = 1.0
    _, kept, _ = check_forward(g, x, None, None)
    assert bool(ref.values(kept)[3].any()) and not bool(ref.values(kept)[:3].any())


@pytest.mark.parametrize("cols", [96, 101, 2048, 20001])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_infinities_and_nan_stay_in_their_row(g, value, cols):
    x, dy = normal(1, (5, cols), BF16), normal(2, (5, cols), BF16)
    weight, bias = parameters(cols, BF16)
    x[2, cols // 2] = value
    y, kept, rstd = g.layer_norm_checkpoint(x, weight, bias)
    bad = torch.tensor([False, False, True, False, False], device="cuda")
    again = g.layer_norm_restore(kept, weight, bias, BF16)
    dx, dweight, dbias = g.layer_norm_backward_checkpoint(dy, kept, weight, rstd)
    for t in (y, again, dx):
        assert torch.equal(t.isnan().all(1), bad) and torch.equal(t.isfinite().all(1), ~bad)
    assert bool((kept.scales[2] == 255).all()) and bool((kept.scales[~bad] != 255).all())
    assert bool(dweight.isnan().all()) and bool(dbias.isfinite().all())


def test_shapes(g):
    """Leading axes, vectors, no rows."""
    weight, bias = parameters(40, F16)
    x = normal(1, (2, 3, 40), F16)
    y, kept, rstd = check_forward(g, x, weight, bias)
    assert y.shape == x.shape and rstd.shape == (2, 3)
    dx, _, _ = check_backward(g, normal(2, (2, 3, 40), F16), kept, weight, rstd)
    assert dx.shape == x.shape and g.layer_norm_restore(kept, weight).dtype == F16
    y, kept, rstd = g.layer_norm_checkpoint(x[0, 0], weight, bias)
    assert rstd.shape == () and g.layer_norm_restore(kept).dtype == F32
    y, kept, rstd = g.layer_norm_checkpoint(x[:0], weight, bias)
    assert kept.codes.shape == (0, 3, 40) and kept.scales.shape == (0, 3, 2)
    dx, dweight, dbias = g.layer_norm_backward_checkpoint(y, kept, weight, rstd)
    assert not bool(dweight.any() or dbias.any()) and g.layer_norm_restore(kept, weight).shape == x[:0].shape


def test_gradient_against_differences(g):
    """dx against differences of the norm at its own kept rows: with x = h (mean 0, variance 1 up to the
    codes' rounding) the loss sum(y * dy) is differenced in 64 bits along random directions."""
    cols, rows = 64, 6
    h = normal(4, (rows, cols), F32).double()
    h = (h - h.mean(1, keepdim=True)) / h.std(1, keepdim=True, unbiased=False)
    kept = g.Fp8Rows(*ref.keep(h))
    v = ref.values(kept)
    # the gradient's formula takes rows of mean 0 and variance 1: bring what the codes hold there in x
    x = (v - v.mean(1, keepdim=True)) / v.std(1, keepdim=True, unbiased=False)
    dy, step = normal(5, (rows, cols), F32), normal(6, (rows, cols), F32).double()
    dx, _, _ = g.layer_norm_backward_checkpoint(dy, kept, None, torch.ones(rows, device="cuda"))

    def loss(t):
        y = (t - t.mean(1, keepdim=True)) / t.std(1, keepdim=True, unbiased=False)
        return float((y * dy.double()).sum())

    got, want = float((dx.double() * step).sum()), (loss(x + 1e-5 * step) - loss(x - 1e-5 * step)) / 2e-5
    # v is within 2^-4 (half a step of E4M3) of rows with that mean and variance, relative
    assert abs(got - want) <= 2.0 ** -3 * float((dx.double().abs() * step.abs()).sum())


def test_same_bits_on_streams_and_in_graphs(g):
    x, dy = normal(1, (300, 1000), BF16), normal(2, (300, 1000), BF16)
    weight, bias = parameters(1000, F32)

    def run(stream=None):
        y, kept, rstd = g.layer_norm_checkpoint(x, weight, bias, stream=stream)
        grads = g.layer_norm_backward_checkpoint(dy, kept, weight, rstd, stream=stream)
        return y, kept.codes.view(torch.uint8), kept.scales, rstd, *grads, g.layer_norm_restore(kept, weight, bias, BF16, stream=stream)

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(want, run()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    x.mul_(-2), dy.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, run()))
