"""Host-side tests of layer norm with 8-bit checkpoints (no GPU, no compute call): the C ABI of
include/checkpoint_ops.h, its refusals, and the tests' reference."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import blackwell_tensor_core_02_gb300 as g
import checkpoint_reference as ref

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED, SCRATCH = 0, -1, -2, -3, -9
P = 1 << 20  # an aligned address that is never read: the calls below are refused first


@pytest.fixture(scope="module")
def lib():
    lib = g.load_linear()
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    lib.norm_checkpoint_forward.argtypes = [vp, i64, vp, vp, vp, i64, vp, vp, vp, i64, i64, f32, i32, i32, vp]
    lib.norm_checkpoint_restore.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp]
    lib.norm_checkpoint_backward.argtypes = [vp, i64, vp, vp, vp, vp, vp, i64, vp, vp, i64, i64, i32, i32, vp, i64, vp]
    return lib


def test_library_exports_every_declared_function(lib, tmp_path):
    header = os.path.join(ROOT, "include", "checkpoint_ops.h")
    with open(header) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(norm_checkpoint_\w+)\s*\(", text))
    assert names == {"norm_checkpoint_forward", "norm_checkpoint_restore", "norm_checkpoint_backward"}
    for name in names:
        assert hasattr(lib, name), name
    if shutil.which("gcc"):
        src = tmp_path / "abi.c"
        src.write_text('#include "checkpoint_ops.h"\nint main(void) { return 0; }\n')
        subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                        str(src), "-o", str(tmp_path / "abi")], check=True)


def test_refusals(lib):
    def keep(x=P, xs=64, w=None, b=None, y=2 * P, ys=64, c=3 * P, s=4 * P, r=5 * P, rows=4, cols=64, eps=1e-5, t=0, wt=0):
        return lib.norm_checkpoint_forward(x, xs, w, b, y, ys, c, s, r, rows, cols, eps, t, wt, None)

    assert keep(cols=0) == keep(rows=-1) == keep(t=3) == keep(wt=1) == keep(eps=-1.0) == keep(xs=-1) == INVALID
    assert keep(eps=float("inf")) == keep(eps=float("nan")) == keep(x=None) == keep(c=None) == keep(s=None) == keep(r=None) == INVALID
    assert keep(ys=63) == keep(y=P) == keep(c=P) == keep(s=3 * P + 255) == keep(r=2 * P) == keep(w=3 * P) == INVALID
    assert keep(rows=1 << 31) == keep(cols=1 << 31) == UNSUPPORTED
    assert keep(x=P + 1) == keep(y=2 * P + 1) == keep(r=5 * P + 2) == keep(w=8 * P + 2, wt=2) == MISALIGNED
    assert keep(rows=0, x=None, y=None, c=None) == OK

    def restore(c=P, s=2 * P, w=None, b=None, y=3 * P, ys=64, rows=4, cols=64, t=0, wt=0):
        return lib.norm_checkpoint_restore(c, s, w, b, y, ys, rows, cols, t, wt, None)

    assert restore(c=None) == restore(s=None) == restore(y=None) == restore(ys=63) == restore(t=3) == restore(wt=1) == INVALID
    assert restore(y=P) == restore(y=2 * P) == restore(w=3 * P) == INVALID
    assert restore(y=3 * P + 1) == restore(b=8 * P + 1) == MISALIGNED
    assert restore(rows=0, y=None) == OK

    def grad(dy=P, ds=64, c=2 * P, s=3 * P, w=None, r=4 * P, dx=5 * P, dxs=64, dw=6 * P, db=7 * P, rows=4, cols=64, t=0, wt=0,
             ws=8 * P, nb=1 << 20):
        return lib.norm_checkpoint_backward(dy, ds, c, s, w, r, dx, dxs, dw, db, rows, cols, t, wt, ws, nb, None)

    assert grad(dw=None) == grad(dx=None) == grad(c=None) == grad(r=None) == grad(ws=None) == grad(dxs=63) == grad(nb=-1) == INVALID
    assert grad(dx=P) == grad(dw=2 * P) == grad(db=6 * P + 2) == grad(ws=5 * P) == grad(dx=3 * P) == INVALID
    assert grad(dw=6 * P + 1) == grad(ws=8 * P + 8) == grad(r=4 * P + 2) == MISALIGNED
    need = lib.layer_norm_backward_workspace_size(4, 64)
    assert grad(nb=need - 1) == SCRATCH


@pytest.mark.parametrize("kwargs", [{}, dict(stream=0)], ids=["here", "stream"])
def test_tensors_that_are_refused(kwargs):
    x = torch.zeros(4, 64)
    kept = g.Fp8Rows(torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8))
    for bad in (lambda: g.layer_norm_checkpoint(3, **kwargs), lambda: g.layer_norm_checkpoint(x.int(), **kwargs),
                lambda: g.layer_norm_restore(x, **kwargs), lambda: g.layer_norm_restore(3, **kwargs),
                lambda: g.layer_norm_restore(g.Fp8Rows(x, x), **kwargs),
                lambda: g.layer_norm_backward_checkpoint("x", kept, None, x, **kwargs)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: g.layer_norm_checkpoint(x, **kwargs), lambda: g.layer_norm_restore(kept, **kwargs),
                lambda: g.layer_norm_restore(g.Fp8Rows(kept.codes, kept.scales[:, :1]), **kwargs),
                lambda: g.layer_norm_backward_checkpoint(x, kept, None, x[:, 0], **kwargs)):
        with pytest.raises(ValueError):
            bad()


def test_reference_by_hand():
    # amax 448 -> floor(log2) 8, scale 1; amax 1 -> scale 2^-8; 500 past 448
    h = torch.zeros(1, 70)
    h[0, 0], h[0, 1], h[0, 32], h[0, 33], h[0, 64] = 500.0, 17.0, 1.0, -0.3, 0.0
    codes, scales = ref.keep(h)
    assert scales.tolist() == [[127, 119, 0]]
    v = ref.values((codes, scales))[0]
    # 17 lies between 16 and 18: a tie, to the even code; 0.3 * 256 = 76.8 between 72 and 80
    assert v[[0, 1, 32, 33, 64]].tolist() == [448.0, 16.0, 1.0, -80 / 256, 0.0]
    assert torch.equal(codes.float(), (ref.nearest(ref.blocks(h.double()) / torch.exp2(scales.double() - 127)[:, :, None]).view(1, -1)[:, :70]).float())
    ref.check_kept((codes, scales), h.double(), torch.zeros(1, 70, dtype=torch.float64))
    with pytest.raises(AssertionError):
        ref.check_kept((codes, scales + 1), h.double(), torch.zeros(1, 70, dtype=torch.float64))


def test_reference_gradient_against_autograd():
    x = torch.randn(5, 33, dtype=torch.float64, requires_grad=True)
    w = torch.randn(33, dtype=torch.float64, requires_grad=True)
    b = torch.zeros(33, dtype=torch.float64, requires_grad=True)
    y = torch.nn.functional.layer_norm(x, (33,), w, b, 1e-3)
    dy = torch.randn(5, 33, dtype=torch.float64)
    y.backward(dy)
    rstd = (x.var(1, unbiased=False) + 1e-3).rsqrt().detach()
    h = ((x - x.mean(1, keepdim=True)) * rstd[:, None]).detach()
    for got, want in zip(ref.grad(dy, h, w.detach(), rstd), (x.grad, w.grad, b.grad)):
        assert torch.allclose(got, want, rtol=1e-10, atol=1e-10)
