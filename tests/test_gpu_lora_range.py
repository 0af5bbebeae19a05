"""fp16 adapters whose intermediate, h = scale * x * down^T, lies far outside fp16's range, on the GPU
against 64 bits."""
import pytest

import grouped_reference as ref
from linear_reference import TINY, UNIT

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F16 = torch.float16


@pytest.fixture(scope="module")
def g(gpu_lib):
    gpu_lib.load_linear()
    return gpu_lib


def normal(gen, shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).half()


def want(x, W, down, up, offsets, chosen, scales):
    """(D, bound).  x·Wᵀ and h are off as fp32 sums (``grouped_reference.adapters``), h by a rounding more
    for the scale, and it is held to 2^-22 of its row's largest: two numbers of 11 bits each, the second's
    least step 2^-25 where the largest is at least 2^-3 times their power of two."""
    rows, K = x.shape
    a64 = x.double()
    D = a64 @ W.double().t()
    far = (K / 64 + 64) * 2.0 ** -23 * (a64.abs() @ W.double().abs().t())
    for e, (i, j) in enumerate(ref.spans(offsets, rows)):
        a = chosen[e]
        if a < 0 or i == j:
            continue
        s, d, u, xs = float(scales[a]), down[a].double(), up[a].double(), a64[i:j]
        h = s * (xs @ d.t())
        eh = (K / 64 + 64) * 2.0 ** -23 * s * (xs.abs() @ d.abs().t()) + 2.0 ** -23 * h.abs() + 2.0 ** -22 * h.abs().amax(1, keepdim=True)
        D[i:j] += h @ u.t()
        far[i:j] += eh @ u.abs().t() + (K / 64 + 64) * 2.0 ** -23 * ((h.abs() + eh) @ u.abs().t())
    return D, far + UNIT[F16] * (D.abs() + far) + TINY[F16]


PATHS = [dict(), dict(tile=16), dict(tile=32, split=2), dict(tile=64, split=1), dict(tile=128, split=8), dict(tile=256)]
PATH_IDS = ["chosen", "16", "32-2", "64-1", "128-8", "256"]


@pytest.mark.parametrize("path", PATHS, ids=PATH_IDS)
@pytest.mark.parametrize("rank", [8, 24, 64, 72, 128])
@pytest.mark.parametrize("counts", [[1], [70, 1, 1, 33, 20], [300, 5, 0, 129, 260]], ids=["1", "125", "694"])
def test_far_sizes(g, counts, rank, path):
    """Requests whose adapters leave h near 1, 2^17, 2^-18, 2^70 and 2^-40, in one batch, and rows of
    one request that differ by up to 2^11."""
    gen = torch.Generator(device="cuda").manual_seed(rank)
    N, K, many = 200, 328, 5
    offsets = [2]
    for c in counts:
        offsets.append(offsets[-1] + c)
    rows = offsets[-1] + 3
    x = normal(gen, (rows, K)) * torch.exp2(-(torch.arange(rows, device="cuda") % 12))[:, None].half()
    W = normal(gen, (N, K), 0.01)
    down, up = normal(gen, (many, rank, K), K ** -0.5), normal(gen, (many, N, rank), 0.3)
    scales = 2.0 ** torch.tensor([0, 17, -18, 70, -40], dtype=torch.float32, device="cuda")
    up[1] *= 2.0 ** -14  # what h is large by
    up[2] *= 2.0 ** 13
    up[3] = 0            # infinite h would be NaN
    up[4] *= 2.0 ** 13   # nothing is left of it
    o, chosen = torch.tensor(offsets, dtype=torch.int32, device="cuda"), [1, 0, 2, 3, 4]
    for turn in range(5 if len(counts) == 1 else 2):
        adapters = torch.tensor(chosen[:len(counts)], dtype=torch.int32, device="cuda")
        got = g.gemm_lora_nt(x, W, down, up, o, adapters, scales=scales, options=g.GroupedOptions(**path, timeout_ns=2_000_000_000))
        value, far = want(x, W, down, up, offsets, chosen, scales)
        off = (got.double() - value).abs()
        assert bool((off <= far).all()), (float((off / far).nan_to_num(nan=float("inf")).max()), (~(off <= far)).nonzero()[:3].tolist())
        chosen = chosen[1:] + chosen[:1]
    assert g.grouped_device_status()[0] == 0


@pytest.mark.parametrize("path", PATHS, ids=PATH_IDS)
@pytest.mark.parametrize("rows", [1, 200, 1600])
def test_values_past_the_largest(g, rows, path):
    """x of ones, down of 16 and up of 2^-8, K 4096: h is 65536, and its contribution 256; columns of up
    that are 0 get 0."""
    x, W = torch.ones(rows, 4096, device="cuda").half(), torch.zeros(24, 4096, device="cuda").half()
    down, up = torch.zeros(1, 8, 4096, device="cuda").half(), torch.zeros(1, 24, 8, device="cuda").half()
    down[0, 0] = 16.0
    up[0, ::2, 0] = 2.0 ** -8
    o, adapters = torch.tensor([0, rows], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = g.gemm_lora_nt(x, W, down, up, o, adapters, options=g.GroupedOptions(**path))
    assert bool((got[:, ::2] == 256.0).all()) and not bool(got[:, 1::2].any())


@pytest.mark.parametrize("path", PATHS, ids=PATH_IDS)
def test_infinite_ranks(g, path):
    """One rank past fp32 (an infinity), another at 2^120 with the other sign: the sum is the
    infinity; a row of another request is what it is alone."""
    x, W = torch.ones(140, 8, device="cuda").half(), torch.zeros(8, 8, device="cuda").half()
    down, up = torch.zeros(2, 8, 8, device="cuda").half(), torch.zeros(2, 8, 8, device="cuda").half()
    down[0, 0, 0], down[0, 1, 0], up[0, :, 0], up[0, :, 1] = 4.0, -(2.0 ** -7), 1.0, 1.0
    down[1, 0, 0], up[1, :, 0] = 3.0, 2.0
    o = torch.tensor([0, 70, 71, 140], device="cuda")
    adapters = torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda")
    scales = torch.tensor([2.0 ** 127, 1.0], device="cuda")
    got = g.gemm_lora_nt(x, W, down, up, o, adapters, scales=scales, options=g.GroupedOptions(**path))
    assert bool((got[70] == 6.0).all())
    assert bool((got[:70] == float("inf")).all()) and bool((got[71:] == float("inf")).all())


@pytest.mark.parametrize("value", [1, 257, 65793])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_large_intermediate_values_of_both_types(g, dtype, value):
    """h of 1, 257 and 65793 = 256² + 256 + 1, of which the shared product takes the largest part away:
    fp16 holds 22 bits of each and gives the difference; bf16 16 bits, so 65792 of the last (a tie between it
    and 65794 in the second number's steps of 1, and no tie: 65793 - 65536 = 257 is 256 or 258 of 8 bits)."""
    for path in PATHS:
        x, W = torch.zeros(130, 16, device="cuda", dtype=dtype), torch.zeros(8, 16, device="cuda", dtype=dtype)
        down, up = torch.zeros(1, 8, 16, device="cuda", dtype=dtype), torch.zeros(1, 8, 8, device="cuda", dtype=dtype)
        x[:, 0], x[:, 1], x[:, 2] = 256.0, 16.0, 1.0
        parts = {1: (0, 0, 1), 257: (0, 16, 1), 65793: (256, 16, 1)}[value]
        for i, v in enumerate(parts):
            down[0, 0, i] = v
        up[0, 0, 0] = 1.0
        W[0, 0] = -parts[0]
        o, adapters = torch.tensor([0, 130], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        got = g.gemm_lora_nt(x, W, down, up, o, adapters, options=g.GroupedOptions(**path))
        right = value - parts[0] * 256.0
        if dtype == torch.bfloat16 and value > 257:
            assert bool(((got[:, 0] == 256.0) | (got[:, 0] == 258.0)).all())
        elif dtype == torch.bfloat16 and value == 257:
            assert bool((got[:, 0] == 256.0).all())  # 257 rounded to 8 bits, ties to even
        else:
            assert bool((got[:, 0] == right).all())
        assert not bool(got[:, 1:].any())


@pytest.mark.parametrize("path", PATHS, ids=PATH_IDS)
@pytest.mark.parametrize("rows", [1, 130, 1700])
def test_the_last_fp32_numbers_in_bf16(g, rows, path):
    """h between bf16's largest and fp32's, which rounds to no bf16: 2^128 - 2^106; up takes 2^121 of it away, and D is off by a rounding (2^-8) and h's two (2^-16)."""
    bf = torch.bfloat16
    x, W = torch.ones(rows, 16, device="cuda", dtype=bf), torch.zeros(8, 16, device="cuda", dtype=bf)
    down, up = torch.zeros(2, 8, 16, device="cuda", dtype=bf), torch.zeros(2, 8, 8, device="cuda", dtype=bf)
    down[:, 0, 0], up[0, ::2, 0], up[1, ::2, 0] = 1.0, 2.0 ** -121, -(2.0 ** -121)
    scales = torch.tensor([3.4e38, -3.4e38], device="cuda")
    o, adapters = torch.tensor([0, rows // 2, rows], device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    got = g.gemm_lora_nt(x, W, down, up, o, adapters, scales=scales, options=g.GroupedOptions(**path)).double()
    value = float(scales[0].double()) * 2.0 ** -121
    assert bool(((got[:, ::2] - value).abs() <= 2.0 ** -7 * value).all()) and not bool(got[:, 1::2].any())
