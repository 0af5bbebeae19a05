"""The differences that the kept rows' gradient is held against: the formula passes, and fails without either of
its terms or a hundredth off (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

import checkpoint_reference as ref
import gradient_differences as diff


@pytest.mark.parametrize("cols", [64, 1008])
def test_what_the_differences_see(cols):
    h = diff.rows(6, cols, 1)
    assert bool((h.sum(1) == 0).all()) and bool((h.square().mean(1) == 1).all())
    codes, scales = ref.keep(h)
    assert torch.equal(ref.values((codes, scales)), h)
    dy, w = diff.upstream(h, 2), diff.weight(cols, 3)
    far = diff.bound(h, dy, w)
    g = dy.double() * w.double()
    dx = ref.grad(dy, h, w, torch.ones(6))[0]
    for name, (off, bound) in diff.off(h, dy, w, dx, far).items():
        assert bool((off <= bound).all()), name
    mean, along = g.mean(1, keepdim=True), h * (g * h).mean(1, keepdim=True)
    for what, wrong in (("no mean", g - along), ("no part along h", g - mean), ("neither", g), ("too large", 1.01 * dx),
                        ("too small", 0.99 * dx), ("negated", -dx), ("h of the mean", g - mean - h * g.mean(1, keepdim=True))):
        seen = diff.off(h, dy, w, wrong, far)
        assert any(bool((off > 10 * bound).all()) for off, bound in seen.values()), what
