"""Operands and results as column slices of one wider matrix: rows that lie between each other's."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g(gpu_lib):
    gpu_lib.load_linear()
    return gpu_lib


def normal(seed, shape, dtype, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("dtype", [F16, F32], ids=["f16", "f32"])
@pytest.mark.parametrize("cols,gap", [(1000, 0), (1024, 0), (333, 0), (1021, 3), (16400, 0)])
def test_checkpoints(g, cols, gap, dtype):
    """x, dy and both results in the rows of one buffer: the bits of separate tensors, and the rest as it was."""
    rows, width = 200, cols + gap
    buf = normal(1, (rows, 4 * width), dtype)
    x, dy, y, dx = (buf[:, i * width:i * width + cols] for i in range(4))
    w, b = normal(2, (cols,), F32), normal(3, (cols,), F32)
    whole = buf.clone()
    xs, dys = (whole[:, i * width:i * width + cols] for i in range(2))
    # the same rows elsewhere, so that the kernels are the same
    want, kept, rstd = g.layer_norm_checkpoint(xs, w, b, out=torch.empty_like(whole)[:, 2 * width:2 * width + cols])
    grads = g.layer_norm_backward_checkpoint(dys, kept, w, rstd, dx=torch.empty_like(whole)[:, 3 * width:3 * width + cols])
    got, kept2, rstd2 = g.layer_norm_checkpoint(x, w, b, out=y)
    assert torch.equal(got, want) and torch.equal(rstd, rstd2)
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(kept, kept2))
    assert all(torch.equal(p, q) for p, q in zip(g.layer_norm_backward_checkpoint(dy, kept, w, rstd, dx=dx), grads))
    whole[:, 2 * width:2 * width + cols], whole[:, 3 * width:3 * width + cols] = want, grads[0]
    assert torch.equal(buf, whole)
    for off in (1, cols - 1):
        with pytest.raises(g.GemmError):
            g.layer_norm_checkpoint(x, w, b, out=buf[:, off:off + cols])
        with pytest.raises(g.GemmError):
            g.layer_norm_backward_checkpoint(x, kept, w, rstd, dx=buf[:, off:off + cols])


@pytest.mark.parametrize("tile", [0, 32, 128, 256])
def test_grouped_products_and_adapters(g, tile):
    """The rows in and out as slices of one buffer: the bits of separate tensors, and the rest as it was."""
    rows, N, K = 150, 136, 200
    counts = [0, 3, 60, 60, 141]
    offsets = torch.tensor(counts, dtype=torch.int32, device="cuda")
    B, buf = normal(1, (4, N, K), BF16, 0.1), normal(2, (rows, 2 * (N + K)), BF16)
    A, D, dD, dA = buf[:, :K], buf[:, K:K + N], buf[:, K + N:K + 2 * N], buf[:, K + 2 * N:]
    o = g.GroupedOptions(tile=tile)
    whole = buf.clone()
    whole[:141, K:K + N] = g.grouped_gemm_nt(A, B, offsets, options=o)[:141]
    whole[:141, K + 2 * N:] = g.grouped_gemm_nn(dD, B, offsets, options=o)[:141]
    assert g.grouped_gemm_nt(A, B, offsets, D, options=o).data_ptr() == D.data_ptr()
    assert g.grouped_gemm_nn(dD, B, offsets, dA, options=o).data_ptr() == dA.data_ptr()
    assert torch.equal(buf, whole)
    down, up = normal(3, (3, 16, K), BF16, K ** -0.5), normal(4, (3, N, 16), BF16)
    adapters = torch.tensor([0, 2, -1, 1], dtype=torch.int32, device="cuda")
    whole[:, K:K + N] = g.gemm_lora_nt(A, B[0], down, up, offsets, adapters, options=o)
    g.gemm_lora_nt(A, B[0], down, up, offsets, adapters, D, options=o)
    assert torch.equal(buf, whole)
    for call in (lambda: g.grouped_gemm_nt(A, B, offsets, buf[:, K - 8:K + N - 8], options=o),
                 lambda: g.gemm_lora_nt(A, B[0], down, up, offsets, adapters, buf[:, K - 8:K + N - 8], options=o),
                 lambda: g.grouped_gemm_nn(dD, B, offsets, buf[:, K + N + 8:2 * K + N + 8], options=o)):
        with pytest.raises(g.GemmError):
            call()
    assert g.grouped_device_status()[0] == 0
