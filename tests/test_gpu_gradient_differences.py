"""The gradients from kept rows against differences, at rows that 8 bits hold exactly."""
import pytest

torch = pytest.importorskip("torch")

import checkpoint_reference as ref
import gradient_differences as diff

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [64, 96, 1008, 1024, 8208, 20000])
def test_norm(gpu_lib, cols):
    """The forward pass keeps such rows exactly, and the gradient from them is the differences' along each
    direction (``gradient_differences.off``; what it sees is held on the CPU)."""
    g = gpu_lib
    h = diff.rows(6, cols, 1)
    y, kept, rstd = g.layer_norm_checkpoint(h.float().cuda(), None, None, 0.0)
    # 1 / cols, the variance and its root are rounded in 32 bits
    assert torch.equal(ref.values(kept).cpu(), h) and bool(((rstd - 1).abs() <= 2.0 ** -22).all())
    assert bool(((y.cpu().double() - h).abs() <= 2.0 ** -21 * h.abs()).all())
    dy, w = diff.upstream(h, 2), diff.weight(cols, 3)
    dx, dweight, dbias = g.layer_norm_backward_checkpoint(dy.cuda(), kept, w.cuda(), torch.ones_like(rstd))
    for name, (off, bound) in diff.off(h, dy, w, dx.cpu().double(), diff.bound(h, dy, w)).items():
        assert bool((off <= bound).all()), (name, float((off / bound).max()))
    # the parameters': the loss is linear in them, 6 rows' sums
    for got, want in ((dweight, (dy.double() * h).sum(0)), (dbias, dy.double().sum(0))):
        assert bool(((got.cpu().double() - want).abs() <= 8 * 2.0 ** -24 * (dy.double().abs() * (1 + h.abs())).sum(0)).all())


def test_experts(gpu_lib):
    """A layer's whole backward pass for the loss |y|^2 / 2 in fp16.  Along ones and along the rows its derivative
    is 0: of dx's own rounding 2^-11 an element is left, and of the restored rows' and dh's nothing that the
    norm's gradient does not take away, beside its fp32 sums (a thousandth of that).  Along dx it is the
    difference: h, each expert's row, y, dh, its sum and dx are rounded, so 6 units relative."""
    from blackwell_tensor_core_02_gb300 import prenorm

    unit, tokens, width, out, experts = 2.0 ** -11, 48, 512, 256, 4
    layer = prenorm.make_experts(width, out, experts, seed=7, dtype=torch.float16)
    layer.eps = 0.0
    layer.weights += 0.03  # so that dh has a mean
    x = diff.rows(tokens, width, 5).cuda()
    gen = torch.Generator(device="cuda").manual_seed(10)
    chosen = torch.rand(tokens, experts, generator=gen, device="cuda").topk(2).indices
    gates = torch.rand(tokens, 2, generator=gen, device="cuda").softmax(1)
    w64, s64, b64 = layer.weights.double(), layer.scale.double(), layer.shift.double()

    def forward(t):
        c = t - t.mean(1, keepdim=True)
        h = c / c.square().mean(1, keepdim=True).sqrt() * s64 + b64
        return sum(((chosen == e) * gates.double()).sum(1, keepdim=True) * (h @ w64[e].t()) for e in range(experts))

    y, kept = layer.forward(x.half(), chosen, gates)
    assert torch.equal(ref.values(kept[0]), x)
    dx = layer.backward(y, kept)[0].double()
    y64 = forward(x)
    dh = sum(((chosen == e) * gates.double()).sum(1, keepdim=True) * (y64 @ w64[e]) for e in range(experts)) * s64
    for u in (torch.ones_like(x), x):
        bound = 1.01 * unit * (dx.abs() * u.abs()).sum(1) + unit / 256 * (dh.abs() * u.abs()).sum(1)
        assert bool(((dx * u).sum(1).abs() <= bound).all())
        assert bool(((dh * u).sum(1).abs() > 4 * bound).float().mean() > 0.9)  # the terms that make it so are large
    step = 1e-5
    u = dx / dx.abs().max()
    loss = lambda t: float((y64 * forward(t)).sum())  # its derivative at x is the loss's
    want = (loss(x + step * u) - loss(x - step * u)) / (2 * step)
    assert abs(float((dx * u).sum()) - want) <= 6 * unit * abs(want)
    assert gpu_lib.grouped_device_status()[0] == 0
