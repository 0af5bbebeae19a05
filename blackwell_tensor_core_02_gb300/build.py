"""Build the sm_103a CUDA library in-tree (nvcc, one translation unit).

The result is ``blackwell_tensor_core_02_gb300/_build/libgemm_f16.so``; it
exports exactly the C ABI declared in ``include/gemm_f16.h``.  A second build
of the same source with the device range checks compiled in
(``-DGEMM_F16_DEVICE_CHECKS=1``), ``libgemm_f16_checked.so``, is for tests.  The
operators around a linear layer's product (``csrc/linear/``) are a library of
their own, ``liblinear_ops.so``, with the C ABI of ``include/linear_ops.h``.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_NAME = "libgemm_f16.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
CHECKED_LIB_PATH = os.path.join(BUILD_DIR, "libgemm_f16_checked.so")
LINEAR_LIB_PATH = os.path.join(BUILD_DIR, "liblinear_ops.so")
LINEAR_CSRC = os.path.join(CSRC, "linear")
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the sm_103a library cannot be built")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "gemm_f16.h")])


def linear_sources() -> list[str]:
    return sorted(glob.glob(os.path.join(LINEAR_CSRC, "*.cu")) + glob.glob(os.path.join(LINEAR_CSRC, "*.cuh")) +
                  glob.glob(os.path.join(LINEAR_CSRC, "*.h")) +
                  glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def is_stale(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return True
    built = os.path.getmtime(path)
    return any(os.path.getmtime(s) > built for s in (linear_sources() if path == LINEAR_LIB_PATH else sources()))


def _command(path: str, checked: bool, verbose: bool, target: str = LIB_PATH) -> list[str]:
    if target == LINEAR_LIB_PATH:
        return [nvcc_path(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "--threads", "0",
                *(["-Xptxas", "-v"] if verbose else []), "-I", INCLUDE, "-I", LINEAR_CSRC,
                *sorted(glob.glob(os.path.join(LINEAR_CSRC, "*.cu"))), "-o", path]
    return [nvcc_path(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
            *(["-DGEMM_F16_DEVICE_CHECKS=1"] if checked else []), *(["-Xptxas", "-v"] if verbose else []),
            "-I", INCLUDE, "-I", CSRC, os.path.join(CSRC, "gemm_f16.cu"), "-o", path]


def binding_path() -> str:
    """The Python binding of the linear layer's operators, for this torch."""
    from importlib.metadata import version

    return os.path.join(BUILD_DIR, f"_linear_binding.torch{version('torch')}.so")


def _binding_command(path: str) -> list[str]:
    import importlib.util
    import sysconfig

    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    system = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
              os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return [shutil.which("g++") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
            *(a for d in system for a in ("-isystem", d)), "-I", INCLUDE, os.path.join(LINEAR_CSRC, "binding.cpp"), "-o", path,
            "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10",
            "-lc10_cuda", "-L", BUILD_DIR, "-l:" + os.path.basename(LINEAR_LIB_PATH), "-Wl,-rpath,$ORIGIN",
            "-Wl,-rpath," + os.path.join(torch_dir, "lib")]


def build_binding(force: bool = False) -> str:
    """Compile the Python binding if missing or older than its sources; return its path.  (It links
    the operators' library, which is built first.)"""
    build_linear()
    path = binding_path()
    sources = [os.path.join(LINEAR_CSRC, "binding.cpp"), *glob.glob(os.path.join(INCLUDE, "*.h"))]
    if force or not os.path.exists(path) or any(os.path.getmtime(s) > os.path.getmtime(path) for s in sources):
        tmp = f"{path}.{os.getpid()}.tmp"
        r = subprocess.run(_binding_command(tmp), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, path)
    return path


def build_many(targets: list[tuple[str, bool]], force: bool = False, verbose: bool = False) -> None:
    """Compile the (path, checked) targets that are missing or stale, in parallel."""
    todo = [(path, checked) for path, checked in targets if force or is_stale(path)]
    if not todo:
        return
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = []
    for path, checked in todo:
        tmp = f"{path}.{os.getpid()}.tmp"
        cmd = _command(tmp, checked, verbose, path)
        procs.append((path, tmp, cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
    errors = []
    for path, tmp, cmd, proc in procs:
        out, err = proc.communicate()
        if proc.returncode != 0:
            errors.append(f"nvcc failed ({proc.returncode}):\n{' '.join(cmd)}\n{out}\n{err}")
            continue
        if verbose:
            print(out + err)
        os.replace(tmp, path)
    if errors:
        raise RuntimeError("\n".join(errors))


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    """Compile the library (or its checked build) if missing or older than its sources; return its path."""
    path = CHECKED_LIB_PATH if checked else LIB_PATH
    build_many([(path, checked)], force=force, verbose=verbose)
    return path


def build_linear(force: bool = False, verbose: bool = False) -> str:
    """Compile the linear layer's operators if missing or older than their sources; return the path."""
    build_many([(LINEAR_LIB_PATH, False)], force=force, verbose=verbose)
    return LINEAR_LIB_PATH


def build_all(force: bool = False, verbose: bool = False) -> None:
    """Every library, compiled side by side."""
    build_many([(LIB_PATH, False), (CHECKED_LIB_PATH, True), (LINEAR_LIB_PATH, False)], force=force, verbose=verbose)
    build_binding(force=force)


if __name__ == "__main__":
    build_all(force=True, verbose=True)
    print(LIB_PATH)
    print(CHECKED_LIB_PATH)
    print(LINEAR_LIB_PATH)
