"""The layers of prenorm.py at their edges."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def _randn(*shape, seed, dtype, size=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * size).to(dtype)


def _inputs(tokens, top, experts, seed=4, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    chosen = torch.rand(tokens, experts, generator=gen, device="cuda").topk(top).indices
    gates = torch.rand(tokens, top, generator=gen, device="cuda").softmax(1)
    return _randn(tokens, 256, seed=1, dtype=dtype), _randn(tokens, 128, seed=2, dtype=dtype), chosen, gates


def _step(layer, x, dy, chosen, gates):
    y, kept = layer.forward(x, chosen, gates)
    return (y, *layer.backward(dy, kept))


def test_experts_without_tokens(gpu_lib):
    """No tokens, or no expert for any: results of those shapes, gradients of the parameters 0."""
    from blackwell_tensor_core_02_gb300 import prenorm

    layer = prenorm.make_experts(256, 128, 4, seed=3)
    for tokens, top in ((0, 2), (5, 0)):
        x, dy, _, _ = _inputs(tokens, 2, 4)
        chosen = torch.zeros(tokens, top, dtype=torch.int64, device="cuda")
        y, dx, dweights, dscale, dshift, dgates = _step(layer, x, dy, chosen, torch.zeros(tokens, top, device="cuda"))
        assert y.shape == (tokens, 128) and dx.shape == x.shape and dgates.shape == (tokens, top)
        assert dweights.shape == layer.weights.shape
        assert not any(bool(t.any()) for t in (y, dx, dweights, dscale, dshift, dgates))


def test_gates_and_choices_of_any_layout(gpu_lib):
    """Transposed, sliced and expanded gates and choices: the results of contiguous ones."""
    from blackwell_tensor_core_02_gb300 import prenorm

    layer = prenorm.make_experts(256, 128, 4, seed=3)
    x, dy, chosen, gates = _inputs(40, 2, 4)
    want = _step(layer, x, dy, chosen, gates)
    wide = torch.full((40, 5), 7.0, device="cuda")
    wide[:, 1:3] = gates
    for c, w in ((chosen.t().contiguous().t(), gates), (chosen, gates.t().contiguous().t()), (chosen, wide[:, 1:3])):
        assert all(torch.equal(a, b) for a, b in zip(_step(layer, x, dy, c, w), want))
    even = torch.full((1, 1), 0.5, device="cuda")
    got, want = (_step(layer, x, dy, chosen, w) for w in (even.expand(40, 2), even.repeat(40, 2)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.int8, torch.uint8, torch.int16, torch.int32])
def test_choices_of_any_whole_type(gpu_lib, dtype):
    """Numbers of experts that the choices' type just holds, or does not: 127 is the last of 128."""
    from blackwell_tensor_core_02_gb300 import prenorm

    for experts in (128, 256):
        layer = prenorm.make_experts(256, 16, experts, seed=3)
        x, dy, chosen, gates = _inputs(40, 2, 128)
        dy = dy[:, :16].contiguous()
        chosen[7, 0] = 127
        want = _step(layer, x, dy, chosen, gates)
        assert all(torch.equal(a, b) for a, b in zip(_step(layer, x, dy, chosen.to(dtype), gates), want))
