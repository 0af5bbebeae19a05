"""The layers of prenorm.py on the grouped products, the adapters and the 8-bit checkpoints: training
steps and served results against the same in 64 bits, and against differences."""
import json

import pytest

import checkpoint_reference as cref
from linear_reference import UNIT

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def _randn(*shape, seed, dtype, size=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * size).to(dtype)


def _routes(tokens, top, experts, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    chosen = torch.rand(tokens, experts, generator=gen, device="cuda").topk(top).indices
    return chosen, torch.rand(tokens, top, generator=gen, device="cuda").softmax(1)


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


def _norm(x, eps):
    mean = x.mean(1, keepdim=True)
    return (x - mean) / ((x - mean).square().mean(1, keepdim=True) + eps).sqrt()


def _mix(h, weights, chosen, gates):
    """Σ_j gates[t, j]·h[t]·W[chosen[t, j]]ᵀ; an expert out of range gives nothing."""
    out = 0.0
    for e in range(weights.shape[0]):
        out = out + ((chosen == e) * gates).sum(1, keepdim=True) * (h @ weights[e].t())
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,top,experts", [(1, 1, 3), (40, 2, 8), (301, 3, 5)])
def test_experts_training_step(gpu_lib, dtype, tokens, top, experts):
    """y against 64-bit autograd: h, each expert's row and y are rounded, 3 units relative in the 2-norm.
    The gradients against autograd from the rows that were kept (their derivative is the norm's, so the
    norm's own gradient is written out): restored h and the gated dy are rounded, dh, its sum and each result, at
    most 4 units relative in the 2-norm (dgates: by element, below)."""
    from blackwell_tensor_core_02_gb300 import prenorm

    width, out, unit = 512, 384, UNIT[dtype]
    layer = prenorm.make_experts(width, out, experts, seed=3, dtype=dtype)
    x = _randn(tokens, width, seed=1, dtype=dtype, size=1.5) + 0.25
    dy = _randn(tokens, out, seed=2, dtype=dtype)
    chosen, gates = _routes(tokens, top, experts, seed=4)
    if tokens > 8:  # experts that do not exist give nothing
        chosen[3, 0], chosen[5, 1] = -1, experts + 2
    y, kept = layer.forward(x, chosen, gates)
    dx, dweights, dscale, dshift, dgates = layer.backward(dy, kept)
    assert [t.dtype for t in (y, dx, dweights)] == [dtype] * 3

    w64, s64, b64, g64 = (t.double().requires_grad_() for t in (layer.weights, layer.scale, layer.shift, gates))
    y64 = _mix(_norm(x.double(), layer.eps) * s64 + b64, w64, chosen, g64).detach()
    assert _off(y, y64) <= 3 * unit
    h64 = cref.values(kept[0])
    h = (h64 * s64 + b64).detach().requires_grad_()
    _mix(h, w64, chosen, g64).backward(dy.double())
    want_dx, want_dscale, want_dshift = cref.grad(h.grad, h64, s64.detach(), kept[1])
    for got, want, what in ((dx, want_dx, "dx"), (dweights, w64.grad, "dweights"), (dscale, want_dscale, "dscale"),
                            (dshift, want_dshift, "dshift")):
        assert _off(got, want) <= 4 * unit, what
    # a gate's gradient is the sum of width products of dh and h, which may cancel: with a rounding of
    # each factor it is off by 2 units of the magnitudes' sum, and the sums' 2^-23 a term are below a third
    magnitude = torch.zeros_like(gates, dtype=torch.float64)
    for e in range(experts):
        dh = (dy.double() @ layer.weights[e].double()).abs()
        magnitude += (chosen == e) * (dh * h.detach().abs()).sum(1, keepdim=True)
    assert bool(((dgates.double() - g64.grad).abs() <= 3 * unit * magnitude).all())
    assert gpu_lib.grouped_device_status()[0] == 0


def test_experts_gradient_against_differences(gpu_lib):
    """The gradient for x along a direction against the 64-bit function's central difference.  The kept
    rows are off by half a step of E4M3, 2^-4 of an element, at most (448 to 512 of a block's scale: an
    eighth), rounded to nearest, so independent: over 64 x 512 elements and as many of the products' sums
    the directional derivative, alike to dx in direction (cosine 1), is off by far less than an eighth."""
    from blackwell_tensor_core_02_gb300 import prenorm

    layer = prenorm.make_experts(512, 256, 4, seed=7, dtype=torch.float16)
    x, dy = _randn(64, 512, seed=8, dtype=torch.float16), _randn(64, 256, seed=9, dtype=torch.float16)
    chosen, gates = _routes(64, 2, 4, seed=10)
    dx = layer.backward(dy, layer.forward(x, chosen, gates)[1])[0].double()

    def f(x):
        h = _norm(x, layer.eps) * layer.scale.double() + layer.shift.double()
        return float((_mix(h, layer.weights.double(), chosen, gates.double()) * dy.double()).sum())

    step = 1e-4
    want = (f(x.double() + step * dx) - f(x.double() - step * dx)) / (2 * step)
    assert abs(float((dx * dx).sum()) - want) <= want / 8


def test_experts_step_in_a_graph(gpu_lib):
    """Forward and backward captured in two graphs with new inputs between replays; no call reads on the host."""
    from blackwell_tensor_core_02_gb300 import prenorm

    layer = prenorm.make_experts(256, 128, 4, seed=11)
    inputs = [(_randn(70, 256, seed=s, dtype=torch.bfloat16), _randn(70, 128, seed=s + 1, dtype=torch.bfloat16),
               *_routes(70, 2, 4, seed=s + 2)) for s in (20, 30)]
    want = []
    for x, dy, chosen, gates in inputs:
        y, kept = layer.forward(x, chosen, gates)
        want.append((y, *layer.backward(dy, kept)))
    held = [t.clone() for t in inputs[0]]
    forward, backward = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(forward):
        y, kept = layer.forward(held[0], held[2], held[3])
    with torch.cuda.graph(backward, pool=forward.pool()):
        grads = layer.backward(held[1], kept)
    for i in (1, 0, 1):
        for t, new in zip(held, inputs[i]):
            t.copy_(new)
        forward.replay()
        backward.replay()
        assert all(torch.equal(a, b) for a, b in zip((y, *grads), want[i]))


def test_linear_layer_with_checkpoints(gpu_lib):
    """The layer that keeps 8 bits: the same y as without, and gradients of the kept rows: dh, the
    restored h and each result are rounded, at most 3 units."""
    from blackwell_tensor_core_02_gb300 import prenorm

    layer, plain = (prenorm.make_layer(512, 384, seed=5, checkpoint=c) for c in (True, False))
    x, dy = _randn(64, 512, seed=1, dtype=torch.float16, size=1.5), _randn(64, 384, seed=2, dtype=torch.float16)
    y, kept = layer.forward(x)
    assert torch.equal(y, plain.forward(x)[0])
    dx, dweight, dscale, dshift = layer.backward(dy, kept)
    h64, dh64 = cref.values(kept[0]), dy.double() @ layer.weight.double()
    want = cref.grad(dh64, h64, layer.scale.double(), kept[1])
    dw64 = dy.double().t() @ (h64 * layer.scale.double() + layer.shift.double())
    for got, right, what in ((dx, want[0], "dx"), (dscale, want[1], "dscale"), (dshift, want[2], "dshift"), (dweight, dw64, "dweight")):
        assert _off(got, right) <= 3 * 2.0 ** -11, what


@pytest.mark.parametrize("tokens,requests,rank", [(1, 1, 8), (5, 8, 16), (64, 16, 64), (700, 3, 24)])
def test_served_adapters(gpu_lib, tokens, requests, rank):
    """y = h·Wᵀ and each request's adapter, from h as the norm rounds it: one rounding of y beside."""
    from blackwell_tensor_core_02_gb300 import prenorm

    layer = prenorm.make_layer(512, 384, seed=5)
    down, up, scales = prenorm.make_adapters(layer, requests, rank, seed=6)
    x, offsets = _randn(tokens, 512, seed=7, dtype=torch.float16), prenorm.even_offsets(tokens, requests)
    adapters = torch.arange(requests, device="cuda", dtype=torch.int32).flip(0)
    adapters[0] = -1
    y = layer.serve_adapted(x, down, up, offsets, adapters, scales)
    h64 = _norm(x.double(), layer.eps) * layer.scale.double() + layer.shift.double()
    want = h64 @ layer.weight.double().t()
    ends = offsets.tolist()
    for i, j, a in zip(ends, ends[1:], adapters.tolist()):
        if a >= 0:
            want[i:j] += scales[a].double() * (h64[i:j] @ down[a].double().t()) @ up[a].double().t()
    assert _off(y, want) <= 2 * 2.0 ** -11
    assert gpu_lib.grouped_device_status()[0] == 0


def test_command(capsys, gpu_lib):
    from blackwell_tensor_core_02_gb300 import prenorm

    prenorm.main(["--tokens", "1", "16", "--width", "256", "--out", "512", "--steps", "3", "--checkpoint", "--adapters", "4",
                  "--rank", "8", "--experts", "4", "--top", "2"])
    lines = [json.loads(s) for s in capsys.readouterr().out.splitlines()]
    assert [d["tokens"] for d in lines] == [1, 16] and all(d["status"] == 0 for d in lines)
    assert all(d[k] > 0 for d in lines for k in ("serve_us", "adapted_us", "experts_forward_us", "experts_step_us"))
