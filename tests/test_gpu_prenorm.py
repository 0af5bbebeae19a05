"""The pre-norm linear layer of prenorm.py: its training step against 64-bit autograd and its served
result against the product of the quantised values."""
import json

import pytest

import linear_reference as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer(gpu_lib):
    from blackwell_tensor_core_02_gb300 import prenorm

    return prenorm.make_layer(512, 384, seed=5)


def _x(tokens, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(tokens, 512, generator=gen, device="cuda") * 1.5 + 0.2).half()


def test_training_step_against_64_bit_autograd(layer):
    """Each result is rounded to fp16 (2^-11 of its size) from inputs that were: y from h (one
    rounding of h), dweight from h and dy, dx and the norm's gradients from dh.  Relative in the
    2-norm that is at most 3 roundings, 3 * 2^-11, and a product's fp32 sums beside."""
    x, dy = _x(64, 1), _x(64, 2)[:, :384].contiguous()
    y, kept = layer.forward(x)
    dx, dweight, dscale, dshift = layer.backward(dy, kept)
    leaves = [t.double().requires_grad_() for t in (x, layer.weight, layer.scale, layer.shift)]
    x64, w64, s64, b64 = leaves
    mean = x64.mean(1, keepdim=True)
    h = (x64 - mean) / ((x64 - mean).square().mean(1, keepdim=True) + layer.eps).sqrt() * s64 + b64
    y64 = h @ w64.t()
    y64.backward(dy.double())
    for got, want, what in ((y, y64, "y"), (dx, x64.grad, "dx"), (dweight, w64.grad, "dweight"),
                            (dscale, s64.grad, "dscale"), (dshift, b64.grad, "dshift")):
        off = float((got.double() - want.detach()).norm() / want.detach().norm())
        assert off <= 3 * 2.0 ** -11, (what, off)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("tokens", [1, 5, 200])
def test_served_result_is_the_quantised_product(gpu_lib, layer, fmt, tokens):
    layer.quantize(fmt)
    x = _x(tokens, 10 + tokens)
    served = layer.serve(x)
    h = gpu_lib.layer_norm(x, layer.scale, layer.shift, layer.eps)[0]
    e = layer.weight4.exponent
    a = ref.values(*ref.quantize(h, fmt), fmt)
    b = ref.values(*ref.quantize(layer.weight, fmt, e), fmt, e)
    want, bound = ref.product_bound(a, b, torch.float16)
    assert bool(((served.double() - want).abs() <= bound).all())
    # 4 bits keep a few per cent of noise on each side; the layer's result stays near the fp16 one
    y = layer.forward(x)[0].double()
    assert float((served.double() - y).norm() / y.norm()) < 0.25
    assert gpu_lib.fp4_device_status()[0] == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("value", [0.0, float("inf"), float("nan")])
def test_weights_without_a_size(gpu_lib, fmt, value):
    """A layer whose weights are zeros gives zeros; one infinity or NaN among them gives its output."""
    from blackwell_tensor_core_02_gb300 import prenorm

    layer = prenorm.make_layer(128, 48, seed=2)
    if value == 0.0:
        layer.weight.zero_()
    else:
        layer.weight[5, 7] = value
    layer.quantize(fmt)
    assert layer.weight4.exponent == 0
    served = layer.serve(_x(9, 3)[:, :128].contiguous())
    want = torch.zeros(9, 48, dtype=torch.bool, device="cuda")
    want[:, 5] = value != 0.0
    assert torch.equal(served.isnan(), want)
    assert bool((served != 0).any()) == (value != 0.0) and gpu_lib.fp4_device_status()[0] == 0


def test_calls_from_several_threads(gpu_lib, layer):
    """Threads with streams of their own, each the first to launch some shape: the results are those
    of one thread alone."""
    import threading

    g = gpu_lib
    layer.quantize("nv")
    inputs = [(_x(tokens, tokens), _x(tokens, tokens + 1)) for tokens in (3, 40, 129, 700)]

    def work(x, dy, stream=None):
        y, mean, rstd = g.layer_norm(x, layer.scale, layer.shift, stream=stream)
        grads = g.layer_norm_backward(dy, x, layer.scale, mean, rstd, stream=stream)
        q = g.quantize_fp4(y, "nv", stream=stream)
        return (y, *grads, g.gemm_fp4_nt(q, layer.weight4, stream=stream), g.dequantize_fp4(q, stream=stream))

    results, failures = {}, []

    def run(i):
        try:
            side = torch.cuda.Stream()
            for _ in range(20):
                results[i] = work(*inputs[i % len(inputs)], stream=side)
            side.synchronize()
        except Exception as e:  # seen by the test below
            failures.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures and len(results) == 8, failures
    for i, got in results.items():
        assert all(torch.equal(a, b) for a, b in zip(got, work(*inputs[i % len(inputs)])))
    assert g.fp4_device_status()[0] == 0


def test_command(capsys, gpu_lib):
    from blackwell_tensor_core_02_gb300 import prenorm

    prenorm.main(["--tokens", "1", "16", "--width", "256", "--out", "512", "--format", "nv", "--steps", "3"])
    lines = [json.loads(s) for s in capsys.readouterr().out.splitlines()]
    assert [d["tokens"] for d in lines] == [1, 16] and all(d["status"] == 0 and d["serve_us"] > 0 for d in lines)
    assert "step_us" not in lines[0] and lines[1]["step_us"] > 0
