"""Host-side tests of the products grouped by rows (no GPU, no compute call): the C ABI of
include/grouped_ops.h and its refusals, and the tests' reference."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import blackwell_tensor_core_02_gb300 as g
import grouped_reference as ref

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, -1, -2, -3
P = 1 << 20  # an aligned address that is never read: the calls below are refused first


@pytest.fixture(scope="module")
def lib():
    from blackwell_tensor_core_02_gb300 import grouped

    return grouped.load_grouped()


def test_library_exports_every_declared_function(lib):
    with open(os.path.join(ROOT, "include", "grouped_ops.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b((?:grouped|gemm_lora)_\w+)\s*\(", text))
    assert {"grouped_gemm_nt", "grouped_gemm_nn", "grouped_gemm_tn", "grouped_last_device_status"} <= names
    for name in names:
        assert hasattr(lib, name), name


def test_header_is_c99_and_the_binding_matches_its_layouts(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    fields = [f for f, _ in g.GroupedOptions._fields_]
    lines = ['#include "grouped_ops.h"', "#include <stddef.h>", "#include <stdio.h>", "int main(void) {",
             '    printf("size %d\\n", (int)sizeof(grouped_options));',
             *(f'    printf("{f} %d\\n", (int)offsetof(grouped_options, {f}));' for f in fields), "    return 0;", "}"]
    src, exe = tmp_path / "abi.c", tmp_path / "abi"
    src.write_text("\n".join(lines) + "\n")
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = dict(s.split() for s in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(g.GroupedOptions)
    for f in fields:
        assert int(got[f]) == getattr(g.GroupedOptions, f).offset


def test_refusals(lib):
    def nt(a=P, lda=64, b=2 * P, ldb=64, bs=32 * 64, off=3 * P, ot=0, d=4 * P, ldd=32, rows=16, groups=3, N=32, K=64, t=0, o=None):
        return lib.grouped_gemm_nt(a, lda, b, ldb, bs, off, ot, d, ldd, rows, groups, N, K, t, 1, None, o)

    assert nt(rows=-1) == nt(groups=-1) == nt(N=-8) == nt(K=-8) == nt(t=2) == nt(ot=2) == INVALID
    assert nt(a=None) == nt(b=None) == nt(off=None) == nt(d=None) == INVALID
    assert nt(lda=56) == nt(ldb=56) == nt(ldd=24) == nt(bs=31 * 64) == INVALID
    assert nt(N=36) == nt(K=60) == nt(groups=1025) == nt(rows=1 << 31) == nt(N=1 << 31) == UNSUPPORTED
    assert nt(a=P + 8) == nt(b=2 * P + 2) == nt(d=4 * P + 8) == nt(lda=68) == nt(bs=32 * 64 + 4) == nt(off=3 * P + 2) == MISALIGNED
    assert nt(off=3 * P + 4, ot=1) == MISALIGNED
    assert nt(d=P) == nt(d=2 * P + 16) == nt(d=3 * P) == nt(d=P + 16 * 64 * 2 - 16) == INVALID
    for bad in (dict(tile=8), dict(split=3), dict(split=2, tile=256), dict(split=-1, tile=16), dict(max_clusters=-1), dict(debug_flags=2), dict(timeout_ns=-1)):
        assert nt(o=g.GroupedOptions(**bad)) == INVALID, bad
    assert nt(rows=0, a=None, d=None) == nt(N=0, b=None, d=None) == OK

    def tn(dd=P, ldd=32, a=2 * P, lda=64, off=3 * P, ot=0, db=4 * P, ldb=64, bs=32 * 64, rows=16, groups=3, N=32, K=64, t=1, o=None):
        return lib.grouped_gemm_tn(dd, ldd, a, lda, off, ot, db, ldb, bs, rows, groups, N, K, t, None, o)

    assert tn(t=2) == tn(dd=None) == tn(a=None) == tn(db=None) == tn(db=P) == tn(bs=31 * 64) == tn(ldb=56) == INVALID
    assert tn(o=g.GroupedOptions(tile=32)) == tn(o=g.GroupedOptions(tile=16, split=2)) == INVALID
    assert tn(dd=P + 8) == tn(db=4 * P + 8) == tn(ldd=36) == MISALIGNED
    assert tn(groups=0) == tn(N=0) == tn(K=0) == OK


@pytest.mark.parametrize("kwargs", [{}, dict(stream=0)], ids=["here", "stream"])
def test_tensors_that_are_refused(kwargs):
    a, b, o = torch.zeros(4, 64, dtype=torch.float16), torch.zeros(2, 32, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    for bad in (lambda: g.grouped_gemm_nt(3, b, o, **kwargs), lambda: g.grouped_gemm_nt(a.float(), b, o, **kwargs),
                lambda: g.grouped_gemm_nn(None, b, o, **kwargs), lambda: g.grouped_gemm_tn(a, "x", o, **kwargs),
                lambda: g.grouped_gemm_nt(a, b, o, options=3, **kwargs)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: g.grouped_gemm_nt(a, b, o, **kwargs), lambda: g.grouped_gemm_nn(a, b, o, **kwargs),
                lambda: g.grouped_gemm_tn(a, a, o, **kwargs)):
        with pytest.raises(ValueError):
            bad()


def test_reference_by_hand():
    assert ref.clamp([-3, 5, 2, 99], 10) == [0, 5, 5, 10] and ref.spans([2, 3, 3], 9) == [(2, 3), (3, 3)]
    A, B = torch.tensor([[1.0, 2], [3, 4], [5, 6]]).half(), torch.tensor([[[1.0, 0], [1, 1]], [[2.0, 1], [0, 1]]]).half()
    assert ref.product(A, B, [0, 1, 2], True)[0].tolist() == [[1, 3], [10, 4], [0, 0]]
    assert ref.product(A, B, [0, 1, 2], False)[0].tolist() == [[3, 2], [6, 7], [0, 0]]
    assert ref.matrices(A, A, [0, 2, 2])[0].tolist() == [[[10, 14], [14, 20]], [[0, 0], [0, 0]]]
