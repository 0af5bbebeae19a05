"""Products grouped by rows on the GPU, all three directions against 64 bits."""
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


def normal(seed, shape, dtype, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def offsets_of(counts, first=0, dtype=torch.int32):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=dtype, device="cuda")


def inputs(counts, N, K, dtype, spare=0, first=0, seed=0):
    rows = first + sum(counts) + spare
    return (normal(seed + 1, (rows, K), dtype), normal(seed + 2, (len(counts), N, K), dtype, 0.1),
            normal(seed + 3, (rows, N), dtype), offsets_of(counts, first))


def near(got, want):
    value, far = want
    off = (got.double() - value).abs()
    assert bool((off <= far).all()), (float((off - far).max()), (off > far).nonzero()[:3].tolist())


def check_all(g, A, B, dD, offsets, tile=0):
    o = g.GroupedOptions(tile=tile, timeout_ns=2_000_000_000)
    host = offsets.tolist()
    near(g.grouped_gemm_nt(A, B, offsets, options=o), ref.product(A, B, host, True))
    near(g.grouped_gemm_nn(dD, B, offsets, options=o), ref.product(dD, B, host, False))
    if tile != 32:
        near(g.grouped_gemm_tn(dD, A, offsets, options=o), ref.matrices(dD, A, host))
    assert g.grouped_device_status()[0] == 0


# one group and many, groups of none, one and around a tile's 16, 32, 64, 128 and 256 rows
COUNTS = [[1], [0, 0, 3], [64], [257], [15, 16, 17, 0, 1, 31, 32, 33], [128, 0, 127, 129, 255, 256, 65], [5] * 40, [700, 1, 2]]


@pytest.mark.parametrize("tile", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c[:8])))
def test_groups(g, counts, dtype, tile):
    check_all(g, *inputs(counts, 200, 136, dtype), tile)


@pytest.mark.parametrize("N,K", [(8, 8), (8, 512), (512, 8), (16, 72), (128, 64), (136, 1024), (1000, 56), (264, 2056), (2048, 264)])
@pytest.mark.parametrize("tile", [0, 64, 128, 256])
def test_widths(g, N, K, tile):
    check_all(g, *inputs([70, 0, 9, 300], N, K, BF16), tile)


@pytest.mark.parametrize("tile", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_other_rows_hold_counts_for_nothing(g, tile, value):
    """Rows without a group, before and behind, hold infinities and NaN, and one group's rows too:
    no other result has any."""
    counts, first, spare = [19, 3, 50, 1], 5, 30
    A, B, dD, offsets = inputs(counts, 136, 72, F16, spare, first)
    rows = A.shape[0]
    bad = list(range(first)) + list(range(first + 19, first + 22)) + list(range(first + 73, rows))
    for t in (A, dD):
        t[bad] = value
    good = [r for r in range(first, first + 73) if r not in bad]
    o = g.GroupedOptions(tile=tile)
    D, dA, dB = g.grouped_gemm_nt(A, B, offsets, options=o), g.grouped_gemm_nn(dD, B, offsets, options=o), g.grouped_gemm_tn(dD, A, offsets, options=o)
    for t in (A, dD):
        t[bad] = 0
    for got, (want, far) in ((D, ref.product(A, B, offsets.tolist(), True)), (dA, ref.product(dD, B, offsets.tolist(), False))):
        near(got[good], (want[good], far[good]))
        none = list(range(first)) + list(range(first + 73, rows))
        assert bool((got[none] == 0).all()) and not bool(got[first + 19:first + 22].isfinite().any())
    want, far = ref.matrices(dD, A, offsets.tolist())
    sound = [0, 2, 3]
    near(dB[sound], (want[sound], far[sound]))
    assert not bool(dB[1].isfinite().any())


def test_nan_in_another_groups_matrix(g):
    A, B, dD, offsets = inputs([20, 7, 40], 200, 136, BF16)
    B[1] = float("nan")
    D, dA = g.grouped_gemm_nt(A, B, offsets), g.grouped_gemm_nn(dD, B, offsets)
    assert bool(D[20:27].isnan().all()) and bool(dA[20:27].isnan().all())
    assert bool(D[:20].isfinite().all() and D[27:].isfinite().all() and dA[:20].isfinite().all() and dA[27:].isfinite().all())


@pytest.mark.parametrize("tile", [32, 64, 128, 256])
def test_given_results_keep_the_rows_without_a_group(g, tile):
    """Into a slice of a wider matrix: rows without a group and columns beside the slice stay."""
    counts, first, spare = [10, 33, 0, 100], 3, 9
    A, B, dD, offsets = inputs(counts, 136, 200, BF16, spare, first)
    o = g.GroupedOptions(tile=tile)
    for call, x, nt, width in ((g.grouped_gemm_nt, A, True, 136), (g.grouped_gemm_nn, dD, False, 200)):
        whole = normal(9, (A.shape[0], width + 24), BF16)
        kept = whole.clone()
        got = call(x, B, offsets, whole[:, 8:8 + width], options=o)
        assert got.data_ptr() == whole[:, 8:].data_ptr()
        want, far = ref.product(x, B, offsets.tolist(), nt)
        near(got[first:first + 143], (want[first:first + 143], far[first:first + 143]))
        kept[first:first + 143, 8:8 + width] = whole[first:first + 143, 8:8 + width]
        assert torch.equal(kept, whole)


def test_strides(g):
    """Operands that are slices: rows further apart than their width, matrices than their extent."""
    A, B, dD, offsets = inputs([40, 0, 90], 72, 136, F16)
    wide = [torch.full((t.shape[0], t.shape[1] + 40), float("nan"), dtype=F16, device="cuda") for t in (A, dD)]
    for t, w in zip((A, dD), wide):
        w[:, 16:16 + t.shape[1]] = t
    A2, dD2 = wide[0][:, 16:16 + 136], wide[1][:, 16:16 + 72]
    Bw = torch.full((3, 80, 144), float("nan"), dtype=F16, device="cuda")
    Bw[:, :72, :136] = B
    check_all(g, A2, Bw[:, :72, :136], dD2, offsets)
    dBw = torch.zeros(3, 80, 144, dtype=F16, device="cuda")
    got = g.grouped_gemm_tn(dD2, A2, offsets, dBw[:, :72, :136])
    near(got, ref.matrices(dD, A, offsets.tolist()))
    dBw[:, :72, :136] = 0
    assert not bool(dBw.any())


def test_offsets_of_64_bits_and_out_of_order(g):
    """Values are taken as at least 0, at most the rows, and at least the one before."""
    A, B, dD, _ = inputs([100, 100, 100], 72, 136, BF16)
    for host in ([0, 100, 200, 300], [-5, 40, 40, 10 ** 12], [50, 20, 250, 100], [400, 0, 0, 0], [10, 10, 10, 10]):
        offsets = torch.tensor(host, dtype=torch.int64, device="cuda")
        check_all(g, A, B, dD, offsets)
        if max(host) < 2 ** 31:
            check_all(g, A, B, dD, offsets.int())


def test_many_groups(g):
    counts = [(7 * e) % 5 for e in range(1024)]
    check_all(g, *inputs(counts, 64, 40, BF16))


def test_nothing_to_do(g):
    A, B, dD, offsets = inputs([0, 0], 64, 40, F16)
    assert g.grouped_gemm_nt(A, B, offsets).shape == (0, 64) and g.grouped_gemm_nn(dD, B, offsets).shape == (0, 40)
    assert not bool(g.grouped_gemm_tn(dD, A, offsets).any())
    A, B, dD, offsets = inputs([5, 9], 64, 0, F16)
    assert not bool(g.grouped_gemm_nt(A, B, offsets).any()) and g.grouped_gemm_tn(dD, A, offsets).shape == (2, 64, 0)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    A = normal(1, (9, 40), F16)
    assert not bool(g.grouped_gemm_nt(A, torch.empty(0, 64, 40, dtype=F16, device="cuda"), none).any())
    assert g.grouped_gemm_tn(normal(2, (9, 64), F16), A, none).shape == (0, 64, 40)
    assert g.grouped_device_status()[0] == 0


def test_gradients_against_differences(g):
    """Sum(D * dD) changes by <dA, step> for a small step of A, and by <dB, step> for one of B; D is
    exact here (small whole numbers), so the differences are too."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    counts, N, K = [6, 0, 11], 24, 16
    offsets = offsets_of(counts)
    A, B, dD, sA, sB = (torch.randint(-2, 3, s, generator=gen, device="cuda").to(BF16)
                        for s in ((17, K), (3, N, K), (17, N), (17, K), (3, N, K)))

    def loss(a, b):
        return (g.grouped_gemm_nt(a, b, offsets).double() * dD.double()).sum()

    dA, dB = g.grouped_gemm_nn(dD, B, offsets), g.grouped_gemm_tn(dD, A, offsets)
    # |D| <= 4 * 16 and |dA| <= 4 * 24, |dB| <= 4 * 11 are whole numbers that bf16 holds
    assert float((loss(A + sA, B) - loss(A - sA, B)) / 2) == float((dA.double() * sA.double()).sum())
    assert float((loss(A, B + sB) - loss(A, B - sB)) / 2) == float((dB.double() * sB.double()).sum())


def test_same_bits_on_streams_and_in_graphs(g):
    A, B, dD, offsets = inputs([30, 0, 200, 41], 264, 136, BF16, 12)
    calls = (lambda **k: g.grouped_gemm_nt(A, B, offsets, **k), lambda **k: g.grouped_gemm_nn(dD, B, offsets, **k),
             lambda **k: g.grouped_gemm_tn(dD, A, offsets, **k))
    want = [c() for c in calls]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [c(stream=side) for c in calls]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [c() for c in calls]
    # the graph reads offsets and operands anew with each replay
    A.mul_(0.5)
    offsets.copy_(offsets_of([0, 100, 71, 100]))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, [c() for c in calls]))


def test_a_chain_of_dependent_calls(g):
    """Each call reads what the one before has just written; 30 rounds give the bits of the first."""
    A, B, _, offsets = inputs([30, 5, 200, 41], 136, 136, BF16)
    B = B * 0.5

    def chain():
        D = A
        for _ in range(4):
            D = g.grouped_gemm_nt(D, B, offsets)
        return D, g.grouped_gemm_tn(D, A, offsets)

    want = chain()
    for _ in range(30):
        assert all(torch.equal(a, b) for a, b in zip(want, chain()))


@pytest.mark.parametrize("tile", [32, 64, 128, 256])
@pytest.mark.parametrize("mode", ["nt", "nn", "tn"])
def test_a_wait_that_runs_out(g, tile, mode):
    """Every wait gives up after 0.1 s; the status says so, and the next calls are right."""
    if mode == "tn" and tile == 32:
        pytest.skip("not a tile of this direction")
    A, B, dD, offsets = inputs([40, 90], 264, 136, F16)
    bad = g.GroupedOptions(tile=tile, debug_flags=1, timeout_ns=100_000_000)
    if mode == "tn":
        g.grouped_gemm_tn(dD, A, offsets, options=bad)
    else:
        (g.grouped_gemm_nt if mode == "nt" else g.grouped_gemm_nn)(A if mode == "nt" else dD, B, offsets, options=bad)
    assert g.grouped_device_status()[0] == TIMEOUT
    check_all(g, A, B, dD, offsets, tile)


@pytest.mark.parametrize("tile", [16, 32, 64, 128])
@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_sums_shared_by_a_cluster(g, tile, split):
    """Tiles of 16 to 128 rows whose sum 1 to 8 CTAs share: odd groups, rows without one, given results."""
    for counts, N, K, first, spare in (([1, 0, 2], 200, 1032, 0, 0), ([15, 33, 0, 130], 136, 520, 3, 4), ([5], 8, 8, 0, 1)):
        A, B, dD, offsets = inputs(counts, N, K, BF16, spare, first)
        o = g.GroupedOptions(tile=tile, split=split, timeout_ns=2_000_000_000)
        for call, x, nt in ((g.grouped_gemm_nt, A, True), (g.grouped_gemm_nn, dD, False)):
            want = ref.product(x, B, offsets.tolist(), nt)
            near(call(x, B, offsets, options=o), want)
            given = torch.full(want[0].shape, 7.0, dtype=BF16, device="cuda")
            call(x, B, offsets, given, options=o)
            last = first + sum(counts)
            near(given[first:last], (want[0][first:last], want[1][first:last]))
            assert bool((given[:first] == 7.0).all() and (given[last:] == 7.0).all())
        bad = g.GroupedOptions(tile=tile, split=split, debug_flags=1, timeout_ns=50_000_000)
        assert g.grouped_device_status()[0] == 0
        g.grouped_gemm_nt(A, B, offsets, options=bad)
        assert g.grouped_device_status()[0] == TIMEOUT


def test_capped_grids(g):
    A, B, dD, offsets = inputs([300, 5, 77], 520, 136, BF16)
    want = g.grouped_gemm_nt(A, B, offsets), g.grouped_gemm_tn(dD, A, offsets)
    for n in (1, 3):
        o = g.GroupedOptions(max_clusters=n)
        assert torch.equal(g.grouped_gemm_nt(A, B, offsets, options=o), want[0])
        assert torch.equal(g.grouped_gemm_tn(dD, A, offsets, options=o), want[1])


@pytest.mark.parametrize("tile", [64, 128])
@pytest.mark.parametrize("split", [1, 2, 4, 8])
@pytest.mark.parametrize("counts", [[1], [0, 5], [64], [130, 0, 17, 1], [1000], [512, 515, 3]], ids=lambda c: "-".join(map(str, c)))
def test_sums_over_rows_shared_by_a_cluster(g, counts, tile, split):
    """The matrices' gradient with its rows split over a cluster: sums shorter than the cluster's K tiles, of
    no whole number of steps, of none; what rows of no group hold counts for nothing; a given result's other columns stay."""
    for N, K, dtype in ((8, 8, F16), (136, 72, BF16), (264, 320, F16)):
        A, B, dD, offsets = inputs(counts, N, K, dtype, 9, 3)
        for t in (A, dD):
            t[:3] = float("nan")
            t[3 + sum(counts):] = float("inf")
        o = g.GroupedOptions(tile=tile, split=split, timeout_ns=2_000_000_000)
        whole = torch.full((len(counts), N + 8, K + 16), 7.0, dtype=dtype, device="cuda")
        got = g.grouped_gemm_tn(dD, A, offsets, whole[:, :N, 8:8 + K], options=o)
        near(got, ref.matrices(dD, A, offsets.tolist()))
        whole[:, :N, 8:8 + K] = 7.0
        assert bool((whole == 7.0).all())
    assert g.grouped_device_status()[0] == 0


@pytest.mark.parametrize("rows,groups,N,K", [(3855, 1, 208, 208), (8192, 1, 64, 64), (3000, 2, 520, 136), (700, 1, 1032, 264), (5000, 12, 200, 104)])
def test_long_sums_of_small_matrices(g, rows, groups, N, K):
    """As the library chooses: few tiles and long sums, groups of unlike lengths, twice with the same bits."""
    cuts = [rows * e * e // (groups * groups) for e in range(groups + 1)]
    A, _, dD, _ = inputs([rows], N, K, BF16)
    offsets = torch.tensor(cuts, device="cuda")
    got = g.grouped_gemm_tn(dD, A, offsets)
    near(got, ref.matrices(dD, A, cuts))
    assert torch.equal(got, g.grouped_gemm_tn(dD, A, offsets)) and g.grouped_device_status()[0] == 0


def test_shared_sums_over_rows_that_time_out(g):
    A, B, dD, offsets = inputs([300, 200], 136, 72, F16)
    o = g.GroupedOptions(tile=64, split=4, debug_flags=1, timeout_ns=50_000_000)
    g.grouped_gemm_tn(dD, A, offsets, options=o)
    assert g.grouped_device_status()[0] == TIMEOUT
    near(g.grouped_gemm_tn(dD, A, offsets), ref.matrices(dD, A, offsets.tolist()))
