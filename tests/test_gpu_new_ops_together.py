"""Grouped products, adapters and checkpoints from several host threads, on two streams at once with
workspaces of their own, in two graphs of one pool, and from rows that are read again and again."""
import threading

import pytest

import checkpoint_reference as cref
import grouped_reference as gref

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


class Step:
    """One use of every operator for `rows` rows; the adapters' h of some fp16 rows lies outside fp16."""

    def __init__(self, rows, dtype, seed):
        self.x, self.dy = normal(seed, (rows, 264), dtype, 1.5), normal(seed + 1, (rows, 136), dtype)
        self.w, self.b = normal(seed + 2, (264,), dtype), normal(seed + 3, (264,), dtype)
        self.B = normal(seed + 4, (3, 136, 264), dtype, 0.06)
        ends = [0, rows // 3, rows // 2, rows]
        self.offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
        self.down, self.up = normal(seed + 5, (2, 24, 264), dtype, 0.06), normal(seed + 6, (2, 136, 24), dtype, 0.2)
        self.adapters = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
        self.scales = torch.tensor([1.0, 2.0 ** -14], device="cuda")
        if dtype == F16:
            self.up[1] *= 2.0 ** 10

    def run(self, g, stream=None):
        y, kept, rstd = g.layer_norm_checkpoint(self.x, self.w, self.b, stream=stream)
        D = g.grouped_gemm_nt(y, self.B, self.offsets, stream=stream)
        E = g.gemm_lora_nt(y, self.B[0], self.down, self.up, self.offsets, self.adapters, scales=self.scales, stream=stream)
        dh = g.grouped_gemm_nn(self.dy, self.B, self.offsets, stream=stream)
        again = g.layer_norm_restore(kept, self.w, self.b, y.dtype, stream=stream)
        dB = g.grouped_gemm_tn(self.dy, again, self.offsets, stream=stream)
        return (y, D, E, dh, again, dB, *g.layer_norm_backward_checkpoint(dh, kept, self.w, rstd, stream=stream))


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


SIZES = [(1, F16), (9, BF16), (130, F16), (600, F16), (1500, BF16)]


def test_several_threads(g):
    """Threads with streams of their own, each the first to launch some shape: one thread's results."""
    steps = [Step(rows, dtype, 10 * i) for i, (rows, dtype) in enumerate(SIZES)]
    results, failures = {}, []

    def work(i):
        try:
            side = torch.cuda.Stream()
            for _ in range(20):
                results[i] = steps[i % len(steps)].run(g, side)
            side.synchronize()
        except Exception as e:  # seen by the test below
            failures.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(10)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures and len(results) == 10, failures
    for i, got in results.items():
        assert same(got, steps[i % len(steps)].run(g)), i
    assert g.grouped_device_status()[0] == 0


def test_two_streams_at_once(g):
    """Calls that run beside each other have workspaces of their own."""
    steps = [Step(130, F16, 1), Step(600, BF16, 2)]
    want = [s.run(g) for s in steps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [[], []]
        for _ in range(4):
            for i in range(2):
                got[i].append(steps[i].run(g, streams[i]))
        torch.cuda.synchronize()
        assert all(same(r, want[i]) for i in range(2) for r in got[i])


def test_two_graphs_of_one_pool(g):
    """Captured one after the other into one pool of memory and replayed in turn, with new inputs."""
    steps = [Step(130, F16, 3), Step(9, BF16, 4)]
    for s in steps:
        s.run(g)
    graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for i, s in enumerate(steps):
        with torch.cuda.graph(graphs[i], pool=graphs[0].pool() if i else None):
            got.append(s.run(g))
    for scale in (0.5, -2.0, 1.0):
        for s in steps:
            s.x.mul_(scale)
        for i in (0, 1):
            graphs[i].replay()
            torch.cuda.synchronize()
            kept = [t.clone() for t in got[i]]
            assert same(kept, steps[i].run(g))
    assert g.grouped_device_status()[0] == 0


@pytest.mark.parametrize("cols", [64, 333, 1024, 20001])
def test_rows_read_again_and_again(g, cols):
    """Expanded rows (stride 0) of x and dy: each result is that of the row written out."""
    x, dy = normal(1, (1, cols), F16), normal(2, (1, cols), F16)
    w, b = normal(3, (cols,), F16), normal(4, (cols,), F16)
    want = g.layer_norm_checkpoint(x.repeat(40, 1), w, b)
    got = g.layer_norm_checkpoint(x.expand(40, cols), w, b)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got[1], want[1]))
    grads = g.layer_norm_backward_checkpoint(dy.repeat(40, 1), want[1], w, want[2])
    assert same(g.layer_norm_backward_checkpoint(dy.expand(40, cols), want[1], w, want[2]), grads)
    h, far = cref.values(want[1]), cref.grad_bounds(dy.expand(40, cols), cref.values(want[1]), w, want[2], F16, F16)
    for t, right, e in zip(grads, cref.grad(dy.expand(40, cols), h, w, want[2]), far):
        assert bool(((t.double() - right).abs() <= e).all())


def test_expanded_operands_are_refused(g):
    """The grouped products and adapters take rows at least a row apart, and matrices at least a matrix."""
    s = Step(9, F16, 5)
    row = s.x[:1].expand(9, 264)
    for bad in (lambda: g.grouped_gemm_nt(row, s.B, s.offsets), lambda: g.grouped_gemm_nt(s.x, s.B[:1].expand(3, 136, 264), s.offsets),
                lambda: g.grouped_gemm_tn(s.dy, row, s.offsets),
                lambda: g.gemm_lora_nt(row, s.B[0], s.down, s.up, s.offsets, s.adapters),
                lambda: g.gemm_lora_nt(s.x, s.B[0], s.down[:1].expand(2, 24, 264), s.up, s.offsets, s.adapters)):
        with pytest.raises(g.GemmError):
            bad()
    assert gref.clamp(s.offsets.tolist(), 9) == [0, 3, 4, 9]


def test_first_calls_in_a_graph():
    """A process whose first call of each operator is captured: tiles, clusters' sizes and shared memory are
    asked for then, and the graph gives what eager calls do."""
    import os
    import subprocess
    import sys

    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import torch, blackwell_tensor_core_02_gb300 as g\n"
            "from test_gpu_new_ops_together import Step, same, F16, BF16\n"
            "steps = [Step(1, F16, 1), Step(600, BF16, 2), Step(130, F16, 3)]\n"
            "torch.cuda.synchronize()\n"
            "graph = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(graph):\n"
            "    got = [s.run(g) for s in steps]\n"
            "graph.replay(); torch.cuda.synchronize()\n"
            "kept = [[t.clone() for t in r] for r in got]\n"
            "assert all(same(k, s.run(g)) for k, s in zip(kept, steps)) and g.grouped_device_status()[0] == 0\n"
            % (os.path.dirname(here), here))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
