"""Layer norm and its gradient on the GPU against their definitions in 64 bits and differences."""
import pytest

import linear_reference as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g(gpu_lib):
    gpu_lib.load_linear()
    return gpu_lib


def rows_of(seed, rows, cols, dtype, gap=0, shift=0, offset=0.5):
    """rows x cols of normal values with an offset, `gap` elements between the rows, the first one
    `shift` elements into its memory."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn(rows * (cols + gap) + shift + 16, generator=gen, device="cuda").mul_(2).add_(offset).to(dtype)
    return buf[shift:shift + rows * (cols + gap)].view(rows, cols + gap)[:, :cols]


def weights_of(seed, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(cols, generator=gen, device="cuda").mul_(0.2).add_(1).to(dtype)
    b = torch.randn(cols, generator=gen, device="cuda").mul_(0.3).to(dtype)
    return w, b


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound).max())} bounds"


# one column to past what a CTA holds in registers, whole warps and odd ones, each side of the
# widths at which another number of threads, units or kernel is taken
COLS = [1, 2, 7, 31, 32, 64, 129, 255, 256, 512, 1000, 1021, 1024, 2056, 4096, 4099, 5003, 8192, 8200, 8320, 16384,
        16385, 32768, 33000]
TYPES = [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32), (F32, F32)]


def check_forward(g, x, w, b, eps):
    y, mean, rstd = g.layer_norm(x, w, b, eps)
    assert y.dtype == x.dtype and y.shape == x.shape and mean.dtype == rstd.dtype == F32
    want, wmean, wrstd = ref.norm(x, w, b, eps)
    ey, emean, erstd = ref.norm_bounds(x, w, b, eps, x.dtype)
    within(mean, wmean, emean, "mean")
    within(rstd, wrstd, erstd, "rstd")
    within(y, want, ey, "y")
    return y, mean, rstd


def check_backward(g, dy, x, w, mean, rstd):
    dx, dw, db = g.layer_norm_backward(dy, x, w, mean, rstd)
    wdtype = x.dtype if w is None else w.dtype
    want = ref.norm_grad(dy, x, w, mean, rstd)
    bound = ref.norm_grad_bounds(dy, x, w, mean, rstd, x.dtype, wdtype)
    within(dx, want[0], bound[0], "dx")
    if w is None:
        assert dw is None and db is None
    else:
        assert dw.dtype == db.dtype == wdtype
        within(dw, want[1], bound[1], "dweight")
        within(db, want[2], bound[2], "dbias")
    return dx, dw, db


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=lambda t: str(t).split(".")[-1])
def test_forward_and_gradient(g, cols, dtype, wdtype):
    for rows in (1, 5, 131):
        x = rows_of(cols + rows, rows, cols, dtype)
        w, b = weights_of(cols, cols, wdtype)
        _, mean, rstd = check_forward(g, x, w, b, 1e-5)
        check_backward(g, rows_of(7 * cols + rows, rows, cols, dtype, offset=0.0), x, w, mean, rstd)


@pytest.mark.parametrize("cols", [8193, 9001, 12280, 12288, 12289, 12296, 16376, 16383])
@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=lambda t: str(t).split(".")[-1])
def test_wide_rows(g, cols, dtype, wdtype):
    """Each side of the widths at which 384 and 512 threads take a row, aligned and not; more rows
    than CTAs fit at once."""
    for rows in (2, 309):
        x = rows_of(cols + rows, rows, cols, dtype)
        w, b = weights_of(cols, cols, wdtype)
        _, mean, rstd = check_forward(g, x, w, b, 1e-5)
        check_backward(g, rows_of(7 * cols + rows, rows, cols, dtype, offset=0.0), x, w, mean, rstd)


@pytest.mark.parametrize("rows", [303, 304, 305, 1000, 4001])
@pytest.mark.parametrize("cols", [48, 1024, 4096])
def test_many_rows(g, rows, cols):
    """More rows than the gradient has parts: each part sums several."""
    x, dy = rows_of(rows, rows, cols, BF16), rows_of(rows + 1, rows, cols, BF16)
    w, b = weights_of(3, cols, F32)
    _, mean, rstd = check_forward(g, x, w, b, 1e-6)
    check_backward(g, dy, x, w, mean, rstd)


# one row a CTA on 152 SMs, and as many as a CTA takes: 16, 12 and 3 of these widths
@pytest.mark.parametrize("cols,rows", [(cols, rows + d) for cols, most in ((48, 16), (1024, 12), (4096, 3), (4099, 1))
                                       for rows in sorted({152, 152 * 2, 152 * most}) for d in (-1, 0, 1)])
def test_rows_around_the_parts(g, cols, rows):
    """Each side of the row counts at which a CTA of the gradient takes a second row, or a row of its
    threads does."""
    x, dy = rows_of(rows, rows, cols, F16), rows_of(rows + 1, rows, cols, F16)
    w, b = weights_of(3, cols, F32)
    _, mean, rstd = check_forward(g, x, w, b, 1e-5)
    check_backward(g, dy, x, w, mean, rstd)


@pytest.mark.parametrize("gap,shift", [(8, 0), (6, 0), (0, 1), (8, 8), (3, 5)])
@pytest.mark.parametrize("dtype", [F16, F32], ids=["f16", "f32"])
def test_strides_and_alignment(g, gap, shift, dtype):
    x, dy = rows_of(1, 37, 1000, dtype, gap, shift), rows_of(2, 37, 1000, dtype, gap + 8, shift)
    w, b = weights_of(3, 1001, F32)
    for wv, bv in ((w[:1000], b[:1000]), (w[1:], b[1:])):
        _, mean, rstd = check_forward(g, x, wv, bv, 1e-5)
        check_backward(g, dy, x, wv, mean, rstd)
        # into rows with a gap (of another alignment, so perhaps another order of the sums): the
        # gap keeps what it held
        buf = torch.full((37, 1000 + gap + 1), -7.0, dtype=dtype, device="cuda")
        out = g.layer_norm(x, wv, bv, out=buf[:, :1000])[0]
        assert out.data_ptr() == buf.data_ptr() and bool((buf[:, 1000:] == -7).all())
        within(out, ref.norm(x, wv, bv, 1e-5)[0], ref.norm_bounds(x, wv, bv, 1e-5, dtype)[0], "y with a gap")
        buf.fill_(-7)
        out = g.layer_norm_backward(dy, x, wv, mean, rstd, dx=buf[:, :1000])[0]
        assert out.data_ptr() == buf.data_ptr() and bool((buf[:, 1000:] == -7).all())
        within(out, ref.norm_grad(dy, x, wv, mean, rstd)[0],
               ref.norm_grad_bounds(dy, x, wv, mean, rstd, dtype, F32)[0], "dx with a gap")


@pytest.mark.parametrize("dtype", [F16, F32], ids=["f16", "f32"])
@pytest.mark.parametrize("cols,gap", [(1000, 0), (1024, 0), (333, 0), (1021, 3), (16400, 0)])
def test_slices_of_one_matrix(g, cols, gap, dtype):
    """Input and output beside each other in the rows of one buffer: the bits of separate tensors,
    and the rest of the buffer as it was."""
    rows, width = 200, cols + gap
    buf = rows_of(1, rows, 4 * width, dtype).contiguous()
    x, dy, y, dx = (buf[:, i * width:i * width + cols] for i in range(4))
    w, b = weights_of(3, cols, F32)
    kept = buf.clone()
    xs, dys = (kept[:, i * width:i * width + cols] for i in range(2))
    # the same rows elsewhere, so that the kernels are the same
    want = g.layer_norm(xs, w, b, out=torch.empty_like(kept)[:, 2 * width:2 * width + cols])
    grads = g.layer_norm_backward(dys, xs, w, *want[1:], dx=torch.empty_like(kept)[:, 3 * width:3 * width + cols])
    got = g.layer_norm(x, w, b, out=y)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all(torch.equal(p, q) for p, q in zip(g.layer_norm_backward(dy, x, w, *got[1:], dx=dx), grads))
    kept[:, 2 * width:2 * width + cols], kept[:, 3 * width:3 * width + cols] = want[0], grads[0]
    assert torch.equal(buf, kept)
    with pytest.raises(g.GemmError):
        g.layer_norm(x, w, b, out=buf[:, 1:1 + cols])


def test_one_row_read_many_times(g):
    """An expanded row (stride 0): every output row is its norm, the gradients sum over all."""
    x = rows_of(5, 1, 768, F16).expand(50, 768)
    w, b = weights_of(6, 768, F16)
    y, mean, rstd = check_forward(g, x, w, b, 1e-5)
    assert torch.equal(y, y[:1].expand_as(y))
    check_backward(g, rows_of(8, 50, 768, F16), x, w, mean, rstd)


@pytest.mark.parametrize("w_on,b_on", [(False, False), (True, False), (False, True)])
def test_without_weight_or_bias(g, w_on, b_on):
    x = rows_of(5, 9, 1000, BF16)
    w, b = weights_of(6, 1000, BF16)
    w, b = w if w_on else None, b if b_on else None
    _, mean, rstd = check_forward(g, x, w, b, 1e-5)
    check_backward(g, rows_of(6, 9, 1000, BF16), x, w, mean, rstd)


@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=lambda t: str(t).split(".")[-1])
@pytest.mark.parametrize("cols", [1, 1000, 1021, 16385, 20480])
def test_gradient_of_a_bias_alone(g, cols, dtype, wdtype):
    """Without a weight dbias (and dweight, that of a weight of ones) comes when it is asked for."""
    x, dy = rows_of(5, 200, cols, dtype), rows_of(6, 200, cols, dtype)
    b = weights_of(6, cols, wdtype)[1]
    _, mean, rstd = check_forward(g, x, None, b, 1e-5)
    want = ref.norm_grad(dy, x, None, mean, rstd)
    bound = ref.norm_grad_bounds(dy, x, None, mean, rstd, dtype, wdtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        got = g.layer_norm_backward(dy, x, None, mean, rstd, grad_dtype=wdtype, stream=stream)
        side.synchronize()
        assert got[0].dtype == dtype and got[1].dtype == got[2].dtype == wdtype
        for t, w, e, what in zip(got, want, bound, ("dx", "dweight", "dbias")):
            within(t, w, e, what)
    assert torch.equal(got[0], g.layer_norm_backward(dy, x, None, mean, rstd)[0])
    none = g.layer_norm_backward(dy[:0], x[:0], None, mean[:0], rstd[:0], grad_dtype=wdtype)
    assert none[2].shape == (cols,) and not none[2].any()


def test_gradient_dtype_refusals(g):
    x = rows_of(5, 9, 64, BF16)
    w, _ = weights_of(6, 64, BF16)
    _, mean, rstd = g.layer_norm(x, w)
    for weight, dtype in ((w, F32), (None, F16), (None, torch.float64), (None, 3)):
        with pytest.raises(TypeError):
            g.layer_norm_backward(x, x, weight, mean, rstd, grad_dtype=dtype)
    assert g.layer_norm_backward(x, x, w, mean, rstd, grad_dtype=BF16)[1].dtype == BF16


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cols", [3, 8, 255, 1000, 1021, 2056, 5003, 12304, 16385, 20479, 20480])
def test_gradient_where_mean_times_rstd_leaves_fp32(g, cols, dtype):
    """Constant rows of 2**110 (h = 0) with rstd = 2**22 among ordinary ones and one of NaN: threads
    that hold columns past the row's end see mean * rstd there, which is no number of fp32."""
    x, dy = rows_of(5, 300, cols, dtype), rows_of(6, 300, cols, dtype)
    w, b = weights_of(6, cols, F32)
    x[::3] = 2.0 ** 110
    x[4, cols // 2] = float("nan")
    _, mean, rstd = g.layer_norm(x, w, b, 1e-5)
    mean[::3], rstd[::3] = 2.0 ** 110, 2.0 ** 22
    for weight in (w, None):
        dx = g.layer_norm_backward(dy, x, weight, mean, rstd)[0]
        assert dx[4].isnan().all()
        keep = torch.arange(300, device="cuda") != 4
        within(dx[keep], ref.norm_grad(dy, x, weight, mean, rstd)[0][keep],
               ref.norm_grad_bounds(dy, x, weight, mean, rstd, dtype, F32)[0][keep], "dx")
    x[4], mean[4], rstd[4] = 0, 0, 1
    check_backward(g, dy, x, w, mean, rstd)


def test_leading_axes(g):
    x = rows_of(5, 24, 512, F16).view(2, 3, 4, 512)
    w, b = weights_of(6, 512, F16)
    y, mean, rstd = g.layer_norm(x, w, b)
    flat = g.layer_norm(x.view(24, 512), w, b)
    assert mean.shape == rstd.shape == (2, 3, 4) and torch.equal(y.view(24, 512), flat[0])
    dx, dw, db = g.layer_norm_backward(x, x, w, mean, rstd)
    dx2, dw2, db2 = g.layer_norm_backward(x.view(24, 512), x.view(24, 512), w, flat[1], flat[2])
    assert torch.equal(dx.view(24, 512), dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
    one = g.layer_norm(x[0, 0, 0], w, b)
    assert one[1].shape == () and torch.equal(one[0], y[0, 0, 0])


def test_no_rows(g):
    x = torch.empty(0, 512, dtype=F16, device="cuda")
    w, b = weights_of(6, 512, F16)
    y, mean, rstd = g.layer_norm(x, w, b)
    assert y.shape == (0, 512) and mean.shape == (0,)
    dx, dw, db = g.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 512) and not dw.any() and not db.any()


def test_constant_rows_and_a_large_offset(g):
    """No variance: y is the bias where the mean is exact; an offset of 1000 deviations keeps its bound."""
    x = torch.full((3, 4096), 2.5, dtype=F32, device="cuda")
    w, b = weights_of(6, 4096, F32)
    y, mean, rstd = g.layer_norm(x, w, b, 1e-5)
    assert torch.equal(y, b.expand_as(y)) and torch.equal(mean, torch.full_like(mean, 2.5))
    check_forward(g, rows_of(3, 20, 4096, F32, offset=2000.0), w, b, 1e-5)
    check_forward(g, rows_of(3, 20, 70000, F32, offset=-2000.0), *weights_of(6, 70000, F32), 1e-5)


def test_infinities_and_nan_stay_in_their_row(g):
    x = rows_of(9, 6, 1024, F16)
    x[1, 3], x[2, 1000], x[4, 0] = float("nan"), float("inf"), float("-inf")
    w, b = weights_of(6, 1024, F16)
    y, mean, rstd = g.layer_norm(x, w, b)
    for r in (1, 2, 4):
        assert y[r].isnan().all() and rstd[r].isnan()
    keep = [0, 3, 5]
    assert torch.equal(y[keep], g.layer_norm(x[keep].contiguous(), w, b)[0])
    dx, dw, _ = g.layer_norm_backward(x, x, w, mean, rstd)
    assert dx[1].isnan().all() and torch.isfinite(dx[keep].float()).all() and dw.isnan().all()


def test_gradient_against_differences(g):
    """Central differences of L = sum(y * r) in 64 bits: their own error is h^2 times a third
    derivative (bounded here by 1e-6 of the gradient's scale at h = 1e-4), so the gradient's fp32
    result has to agree to 2e-5 of that scale."""
    x = rows_of(1, 3, 24, F32)
    w, b = weights_of(2, 24, F32)
    r = rows_of(3, 3, 24, F32, offset=0.0)
    _, mean, rstd = g.layer_norm(x, w, b, 1e-5)
    dx, dw, db = g.layer_norm_backward(r, x, w, mean, rstd)

    def loss(x, w, b):
        return float((ref.norm(x, w, b, 1e-5)[0] * r.double()).sum())

    h = 1e-4
    for t, grad in ((x, dx), (w, dw), (b, db)):
        want = torch.empty_like(t, dtype=torch.float64)
        for i in range(t.numel()):
            d = torch.zeros(t.numel(), dtype=torch.float64, device="cuda")
            d[i] = h
            d = d.view(t.shape)
            args = [v.double() for v in (x, w, b)]
            k = [x, w, b].index(t) if t.dim() == 2 else (1 if t is w else 2)
            up, down = list(args), list(args)
            up[k], down[k] = args[k] + d, args[k] - d
            want.view(-1)[i] = (loss(*up) - loss(*down)) / (2 * h)
        assert float((grad.double() - want).abs().max()) <= 2e-5 * float(want.abs().max())


def test_same_bits_every_time_and_on_another_stream(g):
    x, dy = rows_of(1, 2000, 1024, BF16), rows_of(2, 2000, 1024, BF16)
    w, b = weights_of(2, 1024, F32)
    y, mean, rstd = g.layer_norm(x, w, b)
    first = g.layer_norm_backward(dy, x, w, mean, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        again = g.layer_norm_backward(dy, x, w, mean, rstd, stream=side)
        y2 = g.layer_norm(x, w, b, stream=side.cuda_stream)[0]
    side.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(p, q) for p, q in zip(first, again))


def test_in_a_graph(g):
    x, dy = rows_of(1, 300, 1024, F16), rows_of(2, 300, 1024, F16)
    w, b = weights_of(2, 1024, F16)
    y, mean, rstd = g.layer_norm(x, w, b)
    want = g.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        y2, mean2, rstd2 = g.layer_norm(x, w, b)
        got = g.layer_norm_backward(dy, x, w, mean2, rstd2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(p, q) for p, q in zip(want, got))


def test_refusals(g):
    x = rows_of(1, 4, 64, F16)
    w, b = weights_of(2, 64, F16)
    y, mean, rstd = g.layer_norm(x, w, b)
    with pytest.raises(TypeError):
        g.layer_norm(x.double())
    with pytest.raises(TypeError):
        g.layer_norm(x, w.bfloat16(), b)
    with pytest.raises(TypeError):
        g.layer_norm(x, w, b.float())
    with pytest.raises(ValueError):
        g.layer_norm(x, w[:63], b)
    with pytest.raises(ValueError):
        g.layer_norm(x.cpu())
    with pytest.raises(ValueError):
        g.layer_norm(x.t())
    with pytest.raises(ValueError):
        g.layer_norm(x[:, :0])
    with pytest.raises(ValueError):
        g.layer_norm(x, w, b, out=y[:, :32])
    for eps in (-1.0, float("inf"), float("nan")):
        with pytest.raises(g.GemmError):
            g.layer_norm(x, w, b, eps)
    with pytest.raises(g.GemmError):
        g.layer_norm(x, w, b, out=x)
    with pytest.raises(ValueError):
        g.layer_norm_backward(x, x, w, mean[:3], rstd)
    with pytest.raises(ValueError):
        g.layer_norm_backward(x[:3], x, w, mean, rstd)
    with pytest.raises(ValueError):
        g.layer_norm_backward(x, x, w, mean.double(), rstd)
    with pytest.raises(g.GemmError):
        g.layer_norm_backward(x, y, w, mean, rstd, dx=y)
