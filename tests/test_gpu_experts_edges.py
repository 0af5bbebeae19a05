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


@pytest.mark.parametrize("parameters", ["float32", "none"])
def test_checkpoints_with_other_parameters(gpu_lib, parameters):
    """Scale and shift in 32 bits, or none, as the layer without checkpoints takes them: the step runs, its
    matrices' gradients are those of the restored rows, and the rest is near the layer's without."""
    from blackwell_tensor_core_02_gb300 import prenorm

    def change(layer):
        if parameters == "none":
            layer.scale = layer.shift = None
        else:
            layer.scale, layer.shift = layer.scale.float(), layer.shift.float()
        return layer

    layer, plain = (change(prenorm.make_layer(256, 128, seed=5, checkpoint=c)) for c in (True, False))
    x, dy = _randn(64, 256, seed=1, dtype=torch.float16, size=1.5), _randn(64, 128, seed=2, dtype=torch.float16)
    y, kept = layer.forward(x)
    assert torch.equal(y, plain.forward(x)[0])
    dx, dweight, dscale, dshift = layer.backward(dy, kept)
    h = gpu_lib.layer_norm_restore(kept[0], layer.scale, layer.shift, torch.float16)
    assert torch.equal(dweight, gpu_lib.gemm_f16_nt(dy.t().contiguous(), h.t().contiguous()))
    # the kept rows' elements are off by 2^-4 of themselves at most (an eighth in the top binade)
    for got, want in zip((dx, dscale, dshift), plain.backward(dy, plain.forward(x)[1])[:1] + plain.backward(dy, plain.forward(x)[1])[2:]):
        assert (got is None) == (want is None)
        if got is not None:
            assert got.dtype == want.dtype
            assert float((got.double() - want.double()).norm()) <= 0.125 * float(want.double().norm())
    experts = change(prenorm.make_experts(256, 128, 4, seed=3))
    x, dy, chosen, gates = _inputs(40, 2, 4)
    y, kept = experts.forward(x, chosen, gates)
    dx, dweights, dscale, dshift, dgates = experts.backward(dy, kept)
    assert dx.dtype == dweights.dtype == torch.bfloat16 and bool(dweights.isfinite().all())
    rows, _, token, _, offsets, _ = kept
    h = gpu_lib.layer_norm_restore(rows, experts.scale, experts.shift, torch.bfloat16)
    order = chosen.reshape(-1).argsort(stable=True)
    weighed = (dy[token].float() * gates.reshape(-1)[order][:, None]).to(torch.bfloat16)
    assert torch.equal(dweights, gpu_lib.grouped_gemm_tn(weighed, h[token], offsets))
