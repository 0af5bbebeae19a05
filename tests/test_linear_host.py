"""Host-side tests of the linear layer's operators (no GPU, no compute call): the C ABI of
include/linear_ops.h, its refusals, the choice of a product's tile, and the reference the GPU tests
use, pinned on values worked out by hand."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import blackwell_tensor_core_02_gb300 as g
import linear_reference as ref

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED, SCRATCH = 0, -1, -2, -3, -9
P = 1 << 20  # an aligned address that is never read: the calls below are refused first


def test_library_exports_every_declared_function():
    with open(os.path.join(ROOT, "include", "linear_ops.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = sorted(set(re.findall(r"\b((?:layer_norm|fp4|gemm_fp4)_\w+)\s*\(", text)))
    assert len(names) == 10
    for name in names:
        assert hasattr(g.load_linear(), name), name


def test_header_is_c99_and_the_binding_matches_its_layouts(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    from blackwell_tensor_core_02_gb300 import linear

    structs = {"gemm_fp4_options": linear.Fp4Options, "gemm_fp4_launch_info": linear.Fp4LaunchInfo}
    lines = ['#include "linear_ops.h"', "#include <stddef.h>", "#include <stdio.h>", "int main(void) {"]
    for cname, py in structs.items():
        lines.append(f'    printf("{cname} size %d\\n", (int)sizeof({cname}));')
        lines += [f'    printf("{cname} {f} %d\\n", (int)offsetof({cname}, {f}));' for f, _ in py._fields_]
    lines += ['    printf("bytes %d\\n", (int)fp4_scale_bytes(129, 64, FP4_NV));', "    return 0;", "}"]
    src, exe = tmp_path / "abi.c", tmp_path / "abi"
    src.write_text("\n".join(lines) + "\n")
    lib_dir = os.path.dirname(g.load_linear()._name)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-L", lib_dir, "-l:liblinear_ops.so", f"-Wl,-rpath,{lib_dir}", "-o", str(exe)], check=True)
    got = dict(s.rsplit(" ", 1) for s in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for cname, py in structs.items():
        assert int(got[f"{cname} size"]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(got[f"{cname} {f}"]) == getattr(py, f).offset
    assert int(got["bytes"]) == 2 * 512


def norm(x=P, xs=64, w=None, b=None, y=2 * P, ys=64, mean=3 * P, rstd=4 * P, rows=4, cols=64, eps=1e-5, t=0, wt=0):
    return g.load_linear().layer_norm_forward(x, xs, w, b, y, ys, mean, rstd, rows, cols, eps, t, wt, None)


def grad(dy=P, ds=64, x=2 * P, xs=64, w=None, mean=3 * P, rstd=4 * P, dx=5 * P, dxs=64, dw=6 * P, db=7 * P, rows=4, cols=64,
         t=0, wt=0, ws=8 * P, nb=1 << 20):
    return g.load_linear().layer_norm_backward(dy, ds, x, xs, w, mean, rstd, dx, dxs, dw, db, rows, cols, t, wt, ws, nb, None)


def test_layer_norm_refusals():
    assert norm(cols=0) == norm(rows=-1) == norm(t=3) == norm(wt=1) == norm(eps=-1.0) == INVALID
    assert norm(eps=float("inf")) == norm(eps=float("nan")) == norm(mean=None) == norm(x=None) == norm(y=None) == INVALID
    assert norm(ys=63) == norm(xs=-1) == norm(y=P) == norm(y=P + 256) == norm(w=2 * P) == INVALID
    assert norm(rows=1 << 31) == norm(cols=1 << 31) == UNSUPPORTED
    assert norm(x=P + 1) == norm(y=2 * P + 1) == norm(w=8 * P + 2, wt=2) == norm(mean=3 * P + 2) == MISALIGNED
    assert norm(mean=P + 64) == norm(rstd=3 * P + 12) == norm(mean=2 * P) == norm(w=8 * P, rstd=8 * P) == INVALID
    assert norm(rows=0, x=None, y=None) == OK
    assert grad(dw=None) == grad(db=None) == grad(dx=None) == grad(ws=None) == grad(dxs=63) == grad(nb=-1) == INVALID
    assert grad(dx=P) == grad(dw=2 * P) == grad(db=6 * P + 2) == grad(ws=5 * P) == INVALID
    assert grad(dw=6 * P + 1) == grad(ws=8 * P + 8) == MISALIGNED
    need = g.load_linear().layer_norm_backward_workspace_size(4, 64)
    assert need == 4 * 2 * 64 * 4 and grad(nb=need - 1) == SCRATCH
    assert g.load_linear().layer_norm_backward_workspace_size(10 ** 6, 1021) == 152 * 2 * 1024 * 4
    assert g.load_linear().layer_norm_backward_workspace_size(-1, 64) == INVALID


def test_layer_norm_rows_between_each_others():
    """Slices of one wider matrix share no memory unless their columns do; 4 rows of 64 halves, 256
    bytes apart.  (Where nothing is refused the calls end at the missing device.)"""
    import torch

    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    for y, refused in ((P + 128, False), (P + 126, True), (P + 2, True), (P + 130, True), (P - 128, False), (P - 126, True),
                       (P + 3 * 256 + 128, False), (P + 2 * 256, True), (P + 4 * 256, False), (P - 3 * 256 - 128, False)):
        assert (norm(x=P, xs=128, y=y, ys=128) == INVALID) == refused, y - P
        assert (grad(dy=P, ds=128, dx=y, dxs=128) == INVALID) == refused, y - P
        assert (grad(x=P, xs=128, dy=9 * P, dx=y, dxs=128) == INVALID) == refused, y - P
    assert norm(x=P, xs=128, y=P + 128, ys=136) == norm(x=P, xs=0, y=P - 128, ys=128) == INVALID
    assert norm(x=P, xs=64, y=P + 128, ys=64) == norm(rows=1, xs=128, y=P + 64, ys=128) == INVALID
    assert norm(x=P, xs=128, y=P + 128, ys=128, mean=P + 128) == grad(dy=P, ds=128, dx=P + 128, dxs=128, dw=P) == INVALID


def test_fp4_sizes_and_refusals():
    lib = g.load_linear()
    for rows, cols, data, mx, nv in ((1, 1, 16, 512, 512), (128, 128, 128 * 64, 512, 1024), (129, 129, 129 * 80, 2 * 1024, 2 * 1536),
                                     (0, 64, 0, 0, 0), (5, 0, 0, 0, 0)):
        assert (lib.fp4_data_bytes(rows, cols), lib.fp4_scale_bytes(rows, cols, 0), lib.fp4_scale_bytes(rows, cols, 1)) == (data, mx, nv)
    assert lib.fp4_data_bytes(-1, 4) == lib.fp4_scale_bytes(1, 1, 2) == INVALID
    assert lib.fp4_data_bytes(1, 65535 * 4096 + 1) == UNSUPPORTED
    q = lib.fp4_quantize
    assert q(P, 64, 4, 64, 0, 0, 1, 2 * P, 3 * P, None) == q(P, 64, 4, 64, 0, 1, 101, 2 * P, 3 * P, None) == INVALID
    assert q(P, 64, 4, 64, 4, 0, 0, 2 * P, 3 * P, None) == q(None, 64, 4, 64, 0, 0, 0, 2 * P, 3 * P, None) == INVALID
    assert q(P, 64, 4, 64, 0, 0, 0, P + 128, 3 * P, None) == q(P, 64, 4, 64, 0, 0, 0, 2 * P, 2 * P + 64, None) == INVALID
    assert q(P + 1, 64, 4, 64, 0, 0, 0, 2 * P, 3 * P, None) == q(P, 64, 4, 64, 0, 0, 0, 2 * P + 8, 3 * P, None) == MISALIGNED
    d = lib.fp4_dequantize
    assert d(P, 2 * P, 4, 64, 0, 0, 3 * P, 63, 0, None) == d(P, 2 * P, 4, 64, 0, 0, P, 64, 0, None) == INVALID
    assert d(P, 2 * P, 4, 64, 0, 0, 3 * P + 2, 64, 2, None) == MISALIGNED

    def gemm(a=P, sa=2 * P, b=3 * P, sb=4 * P, dd=5 * P, M=8, N=8, K=64, fmt=0, t=0, **o):
        return lib.gemm_fp4_nt(a, sa, b, sb, dd, M, N, K, fmt, t, 1.0, None, g.Fp4Options(**o))

    assert gemm(M=-1) == gemm(fmt=2) == gemm(t=3) == gemm(a=None) == gemm(dd=None) == gemm(dd=P) == gemm(dd=2 * P) == INVALID
    assert gemm(tile=24) == gemm(cluster_k=3) == gemm(swap=3) == gemm(tile=256, swap=1) == gemm(debug_flags=2) == INVALID
    assert gemm(K=1 << 31) == gemm(N=1 << 31) == gemm(K=65535 * 4096 + 32) == UNSUPPORTED
    assert gemm(a=P + 8) == gemm(sb=4 * P + 4) == gemm(dd=5 * P + 1) == MISALIGNED
    assert gemm(M=0, a=None, dd=None) == OK


def test_product_exponent_refusals():
    def gemm(fmt, exponent):
        return g.load_linear().gemm_fp4_nt(P, 2 * P, 3 * P, 4 * P, 5 * P, 8, 8, 64, fmt, 0, 1.0, None, g.Fp4Options(exponent=exponent))

    assert gemm(1, 1001) == gemm(1, -1001) == gemm(0, 1) == gemm(0, -1) == INVALID


def test_choice_of_tile():
    for (M, N, K), tile, ks, swap, ctas in (
            ((1, 8192, 8192), 16, 4, 2, 256),        # a token: the weights' rows on the 128-row side
            ((8192, 1, 8192), 16, 4, 1, 256),
            ((1, 28672, 4096), 16, 1, 2, 224),       # tiles for a wave: no K split
            ((1, 4096, 14336), 16, 8, 2, 256),
            ((32, 32, 8192), 32, 8, 1, 8),
            ((64, 4096, 4096), 64, 4, 2, 128),
            ((64, 4096, 512), 64, 1, 2, 32),         # two K tiles: no split
            ((100, 4096, 4096), 128, 4, 2, 128),
            ((300, 300, 8192), 128, 8, 1, 72),
            ((512, 4096, 4096), 256, 1, 1, 64),      # CTA pairs from an eighth of the SMs' tiles on
            ((8192, 8192, 8192), 256, 1, 1, 152)):
        d = g.describe_fp4(M, N, K)
        assert (d["tile"], d["cluster_k"], d["swap"], d["ctas"]) == (tile, ks, swap, ctas), (M, N, K, d)
    assert g.describe_fp4(1000, 600, 4096, options=g.Fp4Options(tile=256, max_clusters=3))["ctas"] == 6
    assert g.describe_fp4(1000, 600, 256, options=g.Fp4Options(tile=128, cluster_k=8))["cluster_k"] == 1  # one K tile
    for options in (g.Fp4Options(tile=16, swap=1), g.Fp4Options(tile=64, swap=2)):
        with pytest.raises(g.GemmError):
            g.describe_fp4(100, 100, 512, options=options)
    assert set(g.describe_fp4(0, 5, 5).values()) == {0}
    with pytest.raises(ValueError):
        g.describe_fp4(1, 1, 1, "int4")


def test_import_builds_nothing():
    """`import *` brings the operators' names without torch, a build or a compiler; the first call
    builds."""
    code = """
import sys
sys.modules["torch"] = None
import blackwell_tensor_core_02_gb300.build as build
def refuse(*args, **kwargs):
    raise SystemExit("built")
build.build_many = build.build_binding = refuse
from blackwell_tensor_core_02_gb300 import *
q = Fp4Tensor(None, None, 64, "nv", 3)
assert q.exponent == 3 and gemm_fp4_nt and Fp4Options(tile=16).tile == 16
print("imported")
layer_norm(3)
"""
    import sys

    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.stdout == "imported\n" and r.returncode == 1 and "built" in r.stderr, r.stderr


def test_first_calls_from_several_threads():
    """The binding is loaded once, whoever calls first."""
    code = """
import threading
import torch
import blackwell_tensor_core_02_gb300 as g
from blackwell_tensor_core_02_gb300 import linear
loads, load, errors = [], linear._load_binding, []
linear._load_binding = lambda: loads.append(0) or load()
def call():
    try:
        g.layer_norm(torch.zeros(2, 8))
    except ValueError as e:
        errors.append(e)
threads = [threading.Thread(target=call) for _ in range(8)]
[t.start() for t in threads], [t.join() for t in threads]
assert len(loads) == 1 and len(errors) == 8, (len(loads), len(errors))
"""
    import sys

    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_cpu_tensors_and_wrong_types_are_refused():
    x = torch.zeros(4, 64)
    for bad in (lambda: g.layer_norm(x), lambda: g.layer_norm(x, stream=0), lambda: g.quantize_fp4(x),
                lambda: g.gemm_fp4_nt(g.Fp4Tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), 64),
                                      g.Fp4Tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), 64))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: g.layer_norm(3), lambda: g.layer_norm(x.int()), lambda: g.dequantize_fp4(x), lambda: g.quantize_fp4(x, "nv", exponent="a")):
        with pytest.raises(TypeError):
            bad()


@pytest.mark.parametrize("kwargs", [{}, dict(stream=0)], ids=["here", "stream"])
def test_refusals_are_the_same_on_a_stream(kwargs):
    x, q = torch.zeros(4, 64), g.Fp4Tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), 64)
    for bad in (lambda: g.layer_norm(3, **kwargs), lambda: g.layer_norm(None, **kwargs), lambda: g.layer_norm_backward(1, 2, 3, 4, 5, **kwargs),
                lambda: g.quantize_fp4("x", **kwargs), lambda: g.dequantize_fp4(x, **kwargs), lambda: g.dequantize_fp4(None, **kwargs),
                lambda: g.gemm_fp4_nt(x, q, **kwargs), lambda: g.gemm_fp4_nt(3, 4, **kwargs),
                lambda: g.gemm_fp4_nt((), (), **kwargs), lambda: g.quantize_fp4(3, out=4, **kwargs)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: g.layer_norm(x, **kwargs), lambda: g.quantize_fp4(x, **kwargs), lambda: g.dequantize_fp4(q, **kwargs),
                lambda: g.gemm_fp4_nt(q, q, **kwargs)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("options", [g.Options(), 0, {}, (16, 0, 0, 0, 0, 0, 0)], ids=["f16", "int", "dict", "tuple"])
def test_options_of_another_type_are_refused(options):
    q = g.Fp4Tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), 64)
    with pytest.raises(TypeError):
        g.gemm_fp4_nt(q, q, options=options)


# ------------------------------------------------------------ the reference --

def test_reference_formats_by_hand():
    assert ref.e4m3_values()[:3] == [0.0, 2.0 ** -9, 2.0 ** -8] and ref.e4m3_values()[126] == 448.0
    assert ref.e4m3_values()[8] == 2.0 ** -6 and ref.e4m3_values()[56] == 1.0
    v = torch.tensor([0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 100.0], dtype=torch.float64)
    assert ref.nearest(v, ref.E2M1).tolist() == [0, 1, 2, 2, 4, 4, 6, 6, 7, 7]
    # amax 6 -> scale 1; amax 8 -> floor(log2) - 2 = 1, scale 2
    x = torch.zeros(1, 64)
    x[0, 0], x[0, 1], x[0, 32], x[0, 33] = 6.0, -1.6, 8.0, 7.0
    codes, scales = ref.quantize(x, "mx")
    assert scales.tolist() == [[127, 128]] and codes[0, [0, 1, 32, 33]].tolist() == [7, 11, 6, 6]
    assert ref.values(codes, scales, "mx")[0, [0, 1, 32, 33]].tolist() == [6.0, -1.5, 8.0, 8.0]
    codes, scales = ref.quantize(x, "nv")
    assert scales.tolist() == [[56, 1, 59, 1]]  # 1, the least, 8 / 6 = 1.333 -> 1.375, the least
    tiled = ref.tile(scales)
    assert tiled.shape == (1, 1, 32, 4, 4) and tiled[0, 0, 0, 0].tolist() == [56, 1, 59, 1] and int(tiled.sum()) == 117
    assert ref.pack(torch.tensor([[1, 2, 15, 0]])).tolist() == [[0x21, 0x0F]]


def test_reference_norm_against_torch():
    x = torch.randn(5, 33, dtype=torch.float64, requires_grad=True)
    w, b = torch.randn(33, dtype=torch.float64, requires_grad=True), torch.randn(33, dtype=torch.float64, requires_grad=True)
    y, mean, rstd = ref.norm(x, w, b, 1e-3)
    assert torch.allclose(y, torch.nn.functional.layer_norm(x, (33,), w, b, 1e-3), rtol=1e-12, atol=1e-12)
    dy = torch.randn(5, 33, dtype=torch.float64)
    y.backward(dy)
    dx, dw, db = ref.norm_grad(dy, x.detach(), w.detach(), mean.detach(), rstd.detach())
    for got, want in ((dx, x.grad), (dw, w.grad), (db, b.grad)):
        assert torch.allclose(got, want, rtol=1e-10, atol=1e-10)
