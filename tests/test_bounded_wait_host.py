"""The bounded waits of the linear layer's kernels: two translation units may have them (no GPU)."""
import os
import subprocess

from blackwell_tensor_core_02_gb300 import build


def test_two_translation_units(tmp_path):
    """Each has a status word of its own, so they link as relocatable device code too (compiled whole, as
    the library is, nvcc makes such words each file's own by itself)."""
    files = []
    for name in ("a", "b"):
        path = tmp_path / f"{name}.cu"
        path.write_text('#include "bounded_wait.cuh"\n'
                        f"__global__ void {name}(uint32_t bar) {{ linear_ops::wait_bounded(bar, 0, nullptr, 1, 1, 0); }}\n")
        files.append(str(path))
    out = str(tmp_path / "both.so")
    r = subprocess.run([build.nvcc_path(), *build.ARCH_FLAGS, "-std=c++17", "-rdc=true", "-shared", "-Xcompiler", "-fPIC", "--threads", "0",
                        "-I", build.INCLUDE, "-I", build.LINEAR_CSRC, *files, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0 and os.path.exists(out), r.stderr[-2000:]
