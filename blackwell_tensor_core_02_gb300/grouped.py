"""Products grouped by rows: each group (an expert's tokens) is multiplied with a matrix of its own,
or (a request's tokens) goes through its own low-rank adapter beside a shared matrix.

Over the C ABI of ``include/grouped_ops.h`` (library ``_build/liblinear_ops.so``), by the binding and
in the manner of ``linear.py``: float16 and bfloat16, fp32 sums, one rounding; ``stream=`` as there.

    D = g.grouped_gemm_nt(A, B, offsets)       # D[r] = A[r]·B[e]ᵀ for the rows r of group e
    dA = g.grouped_gemm_nn(dD, B, offsets)     # dA[r] = dD[r]·B[e]
    dB = g.grouped_gemm_tn(dD, A, offsets)     # dB[e] = dD_eᵀ·A_e
    D = g.gemm_lora_nt(x, W, down, up, offsets, adapters, scales=scales)
                                               # D[r] = x[r]·Wᵀ + scales[a]·(x[r]·down[a]ᵀ)·up[a]ᵀ, a = adapters[e]

``offsets`` (int32 or int64, groups + 1 of them on the device): group e has the rows offsets[e] to
offsets[e + 1] - 1.  No call reads them on the host.  Values are taken as at least 0, at most the
number of rows and at least the one before.  Rows before the first offset and from the last on have no
group.  N and K are multiples of 8, rows 16-byte aligned (any number of them) and at least a row apart, so
expanded operands are refused; results may lie between the operands' rows (slices of one matrix).  Up to
1024 groups.
"""
from __future__ import annotations

import ctypes

from . import build as _build
from . import linear as _linear

__all__ = ["grouped_gemm_nt", "grouped_gemm_nn", "grouped_gemm_tn", "gemm_lora_nt", "GroupedOptions", "grouped_device_status"]


class GroupedOptions(ctypes.Structure):
    """Mirror of ``grouped_options`` (zero fields mean defaults)."""
    _fields_ = [("tile", ctypes.c_int32), ("split", ctypes.c_int32), ("max_clusters", ctypes.c_int32), ("debug_flags", ctypes.c_int32),
                ("timeout_ns", ctypes.c_int64)]


_lib: ctypes.CDLL | None = None


def load_grouped() -> ctypes.CDLL:
    """Build (if stale) and load the library, with the types of its functions here."""
    global _lib
    if _lib is None:
        vp, i64, i32, opts = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.POINTER(GroupedOptions)
        lib = ctypes.CDLL(_build.build_linear())
        rows = [vp, i64, vp, i64, i64, vp, i32, vp, i64, i64, i64, i64, i64, i32, i32, vp, opts]
        for name, args in (("grouped_gemm_nt", rows), ("grouped_gemm_nn", rows),
                           ("grouped_gemm_tn", [vp, i64, vp, i64, vp, i32, vp, i64, i64, i64, i64, i64, i64, i32, vp, opts]),
                           ("gemm_lora_nt", [vp, i64, vp, i64, vp, i64, i64, vp, i64, i64, vp, vp, i32, vp, vp, i64, i64, i64, i64, i64,
                                             i64, i64, i32, vp, i64, vp, opts]),
                           ("grouped_last_device_status", [vp, ctypes.POINTER(ctypes.c_uint64)])):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        lib.gemm_lora_workspace_size.argtypes, lib.gemm_lora_workspace_size.restype = [i64, i64], i64
        _lib = lib
    return _lib


def _address(options) -> int:
    if options is not None and not isinstance(options, GroupedOptions):
        raise TypeError("options must be a GroupedOptions")
    return 0 if options is None else ctypes.addressof(options)


def _call(name, args, stream, options):
    args = (*args, _address(options))
    call = getattr(_linear._native, name)
    return call(*args) if stream is None else _linear._on(stream, call, args, args[:-1])


# The calls below go to the binding at once where neither a stream nor options are given: the
# smallest take less time on the GPU than the way through _call.


def grouped_gemm_nt(A, B, offsets, D=None, *, stream=None, options: GroupedOptions | None = None):
    """D[r] = A[r]·B[e]ᵀ for the rows r of group e; A rows x K, B groups x N x K, D rows x N.

    Rows without a group are 0 in a D that the call makes, and left as they are in a given one.
    """
    if stream is None and options is None:
        return _linear._native.grouped_gemm_nt(A, B, offsets, D, 0)
    return _call("grouped_gemm_nt", (A, B, offsets, D), stream, options)


def grouped_gemm_nn(dD, B, offsets, dA=None, *, stream=None, options: GroupedOptions | None = None):
    """The gradient of ``grouped_gemm_nt`` for A: dA[r] = dD[r]·B[e]; rows without a group as there."""
    if stream is None and options is None:
        return _linear._native.grouped_gemm_nn(dD, B, offsets, dA, 0)
    return _call("grouped_gemm_nn", (dD, B, offsets, dA), stream, options)


def grouped_gemm_tn(dD, A, offsets, dB=None, *, stream=None, options: GroupedOptions | None = None):
    """The gradient of ``grouped_gemm_nt`` for B: dB[e] = dD_eᵀ·A_e, 0 for a group without rows.

    Rows without a group count for nothing, whatever they hold.
    """
    if stream is None and options is None:
        return _linear._native.grouped_gemm_tn(dD, A, offsets, dB, 0)
    return _call("grouped_gemm_tn", (dD, A, offsets, dB), stream, options)


def gemm_lora_nt(x, W, down, up, offsets, adapters, D=None, *, scales=None, stream=None,
                 options: GroupedOptions | None = None):
    """D[r] = x[r]·Wᵀ + scales[a]·(x[r]·down[a]ᵀ)·up[a]ᵀ for the rows r of request e, a = adapters[e].

    x rows x K, W N x K, down adapters x rank x K, up adapters x N x rank, D rows x N; rank a multiple
    of 8 up to 128; ``adapters`` int32, ``scales`` float32 (None: 1), both on the device, one for each
    request and each adapter.  An adapter out of range (-1) and rows without a request have the
    shared product alone.  No row's result depends on another row's adapter.  Between its two products
    scales[a]·x[r]·down[a]ᵀ is held, whatever its size, to 2⁻¹⁶ of itself (bfloat16) or 2⁻²² of the row's
    largest (float16); the sum is fp32.
    """
    if stream is None and options is None:
        return _linear._native.gemm_lora_nt(x, W, down, up, offsets, adapters, D, scales, 0)
    return _call("gemm_lora_nt", (x, W, down, up, offsets, adapters, D, scales), stream, options)


def grouped_device_status(stream=None) -> tuple[int, int]:
    """(status, info) of these products' device status word, after synchronising `stream`; clears it."""
    import torch

    handle = torch.cuda.current_stream().cuda_stream if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
    info = ctypes.c_uint64(0)
    rc = load_grouped().grouped_last_device_status(handle, ctypes.byref(info))
    return rc, info.value
