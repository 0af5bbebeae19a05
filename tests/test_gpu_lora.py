"""Low-rank adapters of many requests beside a shared product, on the GPU against 64 bits."""
import pytest

import grouped_reference as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
TIMEOUT = -7


@pytest.fixture(scope="module")
def g(gpu_lib):
    gpu_lib.load_linear()
    return gpu_lib


def normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


class Batch:
    """Requests of the given lengths with adapters `chosen`, after `first` rows and before `spare`
    that belong to none."""

    def __init__(self, counts, chosen, many, rank, N, K, dtype, first=0, spare=0, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rows = first + sum(counts) + spare
        o = [first]
        for c in counts:
            o.append(o[-1] + c)
        self.x, self.W = normal(gen, (rows, K), dtype), normal(gen, (N, K), dtype, 0.05)
        self.down, self.up = normal(gen, (many, rank, K), dtype, K ** -0.5), normal(gen, (many, N, rank), dtype, 0.3)
        self.scales = torch.rand(many, generator=gen, device="cuda") + 0.5
        self.offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
        self.adapters = torch.tensor(chosen, dtype=torch.int32, device="cuda")

    def args(self):
        return self.x, self.W, self.down, self.up, self.offsets, self.adapters

    def want(self):
        return ref.adapters(self.x, self.W, self.down, self.up, self.offsets.tolist(), self.adapters.tolist(), self.scales)


def near(got, want):
    value, far = want
    off = (got.double() - value).abs()
    assert bool((off <= far).all()), (float((off - far).max()), (off > far).nonzero()[:3].tolist())


def check(g, b, **options):
    near(g.gemm_lora_nt(*b.args(), scales=b.scales, options=g.GroupedOptions(**options, timeout_ns=2_000_000_000)), b.want())
    assert g.grouped_device_status()[0] == 0


PATHS = [dict(), dict(tile=16), dict(tile=32, split=2), dict(tile=64, split=1), dict(tile=128, split=8), dict(tile=256)]
BATCHES = [([1], [0]), ([1] * 40, [e % 5 - 1 for e in range(40)]), ([3, 0, 1, 17, 64], [2, 2, 9, 0, -1]),
           ([300, 5, 129], [1, 1, 0]), ([260], [3])]


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(f"{k}{v}" for k, v in p.items()) or "chosen")
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("batch", BATCHES, ids=lambda b: f"{len(b[0])}of{sum(b[0])}")
def test_batches(g, batch, dtype, path):
    check(g, Batch(*batch, 4, 16, 200, 328, dtype, 2, 5), **path)


@pytest.mark.parametrize("rank", [8, 16, 24, 64, 72, 128])
@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(f"{k}{v}" for k, v in p.items()) or "chosen")
@pytest.mark.parametrize("N,K", [(8, 8), (136, 1024), (520, 72)])
def test_ranks_and_widths(g, N, K, rank, path):
    check(g, Batch([1, 30, 1, 150], [1, 0, 2, 1], 3, rank, N, K, BF16), **path)


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(f"{k}{v}" for k, v in p.items()) or "chosen")
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_an_adapter_reaches_its_own_rows_only(g, path, value):
    """Adapters that hold NaN or infinities, in use or not, a scale or a row that is NaN: the other
    rows are what they are without."""
    b = Batch([2, 1, 9, 1, 20], [0, 1, 2, -1, 0], 5, 24, 136, 200, F16, 1, 3)
    want, far = b.want()
    b.up[1] = value                       # of row 3
    b.down[2, 3] = value                  # of rows 4 to 12
    b.up[3], b.down[3], b.scales[4] = value, value, value  # of none
    b.x[0], b.x[14] = value, value        # a row without a request, the first of the last one
    got = g.gemm_lora_nt(*b.args(), scales=b.scales, options=g.GroupedOptions(**path))
    touched = [0, *range(3, 13), 14]
    sound = [r for r in range(b.x.shape[0]) if r not in touched]
    near(got[sound], (want[sound], far[sound]))
    assert not bool(got[touched].isfinite().all(1).any())


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(f"{k}{v}" for k, v in p.items()) or "chosen")
def test_strides_given_result_and_offsets(g, path):
    b = Batch([40, 9, 70], [1, 0, 1], 2, 16, 72, 136, BF16, 3, 2)
    def inside(t, fill):  # the same values inside a larger tensor
        big = torch.full([s + 8 for s in t.shape], fill, dtype=t.dtype, device="cuda")
        view = big[tuple(slice(0, s) for s in t.shape)]
        view.copy_(t)
        return big, view
    nan = float("nan")
    x, W, down, up = (inside(t, nan)[1] for t in (b.x, b.W, b.down, b.up))
    out, D = inside(torch.zeros(124, 72, dtype=BF16, device="cuda"), 3.0)
    got = g.gemm_lora_nt(x, W, down, up, b.offsets, b.adapters, D, scales=b.scales, options=g.GroupedOptions(**path))
    assert got.data_ptr() == D.data_ptr()
    near(got, b.want())
    D.fill_(3.0)
    assert bool((out == 3.0).all())
    for host in ([-4, 40, 30, 10 ** 12], [50, 20, 100, 90], [200, 0, 0, 0], [7, 7, 7, 7]):
        b.offsets = torch.tensor(host, dtype=torch.int64, device="cuda")
        check(g, b, **path)


def test_without_adapters(g):
    """No requests, no adapters, no scales, and nothing at all."""
    b = Batch([5, 30], [0, 1], 2, 16, 72, 136, BF16)
    b.scales = None
    check(g, b)
    for tile in (0, 256):
        o = g.GroupedOptions(tile=tile)
        none = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = g.gemm_lora_nt(b.x, b.W, b.down, b.up, none, none[:0], options=o)
        b.adapters = torch.tensor([-1, 2], dtype=torch.int32, device="cuda")
        near(got, b.want())
        check(g, b, tile=tile)
        assert torch.equal(got, g.gemm_lora_nt(b.x, b.W, b.down[:0], b.up[:0], b.offsets, b.adapters, options=o))
    assert g.gemm_lora_nt(b.x[:0], b.W, b.down, b.up, b.offsets, b.adapters).shape == (0, 72)
    assert not bool(g.gemm_lora_nt(b.x[:, :0], b.W[:, :0], b.down[:, :, :0], b.up, b.offsets, b.adapters).any())


def test_many_requests(g):
    check(g, Batch([e % 3 for e in range(1024)], [e % 7 - 1 for e in range(1024)], 6, 8, 64, 136, BF16, 4, 4))
    check(g, Batch([e % 3 for e in range(1024)], [e % 7 - 1 for e in range(1024)], 6, 8, 64, 136, BF16, 4, 4), tile=256)


def test_large_intermediate_values(g):
    """x·downᵀ far outside bf16's 8 bits: 1, 257 and 65793 are held by the two 16-bit numbers, or fp32."""
    for path in PATHS:
        b = Batch([130], [0], 1, 8, 8, 8, BF16)
        b.x.fill_(0), b.W.fill_(0), b.down.fill_(0), b.up.fill_(0)
        b.x[:, 0], b.x[:, 1], b.down[0, 0, 0], b.down[0, 0, 1] = 1.0, 1.0, 256.0, 1.0  # h = 257
        b.up[0, 0, 0], b.W[0, 0] = 1.0, -256.0
        b.scales.fill_(1.0)
        got = g.gemm_lora_nt(*b.args(), scales=b.scales, options=g.GroupedOptions(**path))
        assert bool((got[:, 0] == 1.0).all()) and not bool(got[:, 1:].any())


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(f"{k}{v}" for k, v in p.items()) or "chosen")
def test_dependent_calls(g, path):
    """Each call reads what the one before has just written; its first launch may start before that
    one has ended, its second before its first.  40 rounds give the bits of the first, alone and
    from a graph."""
    b = Batch([30, 1, 1, 99], [1, 0, -1, 1], 2, 16, 136, 136, BF16, 1, 2)
    o = g.GroupedOptions(**path)

    def chain():
        x = b.x
        for _ in range(3):
            x = g.gemm_lora_nt(x, b.W, b.down, b.up, b.offsets, b.adapters, scales=b.scales, options=o)
        return x

    want = chain()
    first = g.gemm_lora_nt(*b.args(), scales=b.scales, options=o)
    near(first, b.want())
    for _ in range(40):
        assert torch.equal(want, chain())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(first, g.gemm_lora_nt(*b.args(), scales=b.scales, options=o, stream=side).cpu().cuda())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    b.adapters.copy_(torch.tensor([0, 0, 1, -1], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, chain()) and not torch.equal(got, want)
    assert g.grouped_device_status()[0] == 0


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(f"{k}{v}" for k, v in p.items()) or "chosen")
def test_a_wait_that_runs_out(g, path):
    b = Batch([30, 40], [1, 0], 2, 16, 264, 520, F16)
    bad = g.GroupedOptions(**path, debug_flags=1, timeout_ns=100_000_000)
    g.gemm_lora_nt(*b.args(), scales=b.scales, options=bad)
    assert g.grouped_device_status()[0] == TIMEOUT
    check(g, b, **path)


@pytest.mark.parametrize("rank", [8, 16, 24, 40, 96])
@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(f"{k}{v}" for k, v in p.items()) or "chosen")
def test_both_ways_to_the_ranks(g, rank, path):
    """x·downᵀ by either of its kernels: rows x rank below 12288, at it (rank 8, 16, 24, 96) and past it."""
    for rows in (12288 // rank - 1, 12288 // rank, 12288 // rank + 8):
        check(g, Batch([rows - 40, 3, 0, 30], [1, -1, 0, 2], 3, rank, 72, 136, F16, 2, 5), **path)
