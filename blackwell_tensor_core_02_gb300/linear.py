"""The operators around a linear layer's product: layer norm and its gradient, quantisation to
microscaled 4-bit floats, and the product of two such matrices.

Argument marshalling over the C ABI of ``include/linear_ops.h`` (library ``_build/liblinear_ops.so``),
as the package's ``gemm_f16_nt`` is over its own, here by a compiled binding (``csrc/linear/binding.cpp``):
PyTorch supplies memory and streams, every step of the computation runs in the library, and there is
no fallback.  The first call builds what is stale and loads it (importing this module does neither).

    y, mean, rstd = g.layer_norm(x, weight, bias)
    dx, dweight, dbias = g.layer_norm_backward(dy, x, weight, mean, rstd)
    W = g.quantize_fp4(w)                       # once
    D = g.gemm_fp4_nt(g.quantize_fp4(y), W)     # = y @ w.T of the quantised values

With ``stream=`` a call runs on that stream; what it allocates belongs to that stream, and the
inputs' memory is kept from reuse until the call has run.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import threading
from typing import TYPE_CHECKING, NamedTuple

from . import build as _build

if TYPE_CHECKING:
    import torch

__all__ = ["layer_norm", "layer_norm_backward", "Fp4Tensor", "quantize_fp4", "dequantize_fp4", "gemm_fp4_nt",
           "Fp4Options", "describe_fp4", "fp4_device_status"]

_FORMATS = {"mx": 0, "nv": 1}


class Fp4Options(ctypes.Structure):
    """Mirror of ``gemm_fp4_options`` (zero fields mean defaults)."""
    _fields_ = [("tile", ctypes.c_int32), ("cluster_k", ctypes.c_int32), ("swap", ctypes.c_int32),
                ("max_clusters", ctypes.c_int32), ("debug_flags", ctypes.c_int32), ("timeout_ns", ctypes.c_int64),
                ("exponent", ctypes.c_int32)]


class Fp4LaunchInfo(ctypes.Structure):
    """Mirror of ``gemm_fp4_launch_info``."""
    _fields_ = [("tile", ctypes.c_int32), ("cluster_k", ctypes.c_int32), ("swap", ctypes.c_int32),
                ("ctas", ctypes.c_int64)]


class Fp4Tensor(NamedTuple):
    """A matrix of microscaled 4-bit floats, rows x cols.

    ``data``: uint8 [rows, ceil(cols / 32) * 16], two E2M1 codes a byte, the even column in the low
    nibble, code 0 from column `cols` on.  ``scales``: uint8 [ceil(rows / 128), ceil(blocks / 4), 32,
    4, 4]: the scale code of row 128 i + 32 g + l and block 4 j + k at [i, j, l, g, k].  ``format``
    "mx": blocks of 32, E8M0 scales; "nv": blocks of 16, E4M3 scales times 2**exponent.
    """
    data: torch.Tensor
    scales: torch.Tensor
    cols: int
    format: str = "mx"
    exponent: int = 0

    @property
    def rows(self) -> int:
        return self.data.shape[0]


_lock = threading.Lock()
_lib: ctypes.CDLL | None = None


def load_linear() -> ctypes.CDLL:
    """Build (if stale) and load the library and its binding; raise if that is impossible."""
    global _lib
    _native.layer_norm  # loads the binding
    if _lib is None:
        with _lock:
            if _lib is None:
                vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
                lib = ctypes.CDLL(_build.build_linear())
                opts = ctypes.POINTER(Fp4Options)
                for name, args, res in (
                        ("layer_norm_forward", [vp, i64, vp, vp, vp, i64, vp, vp, i64, i64, f32, i32, i32, vp], ctypes.c_int),
                        ("layer_norm_backward", [vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, vp, i64, i64, i32, i32, vp, i64, vp],
                         ctypes.c_int),
                        ("layer_norm_backward_workspace_size", [i64, i64], i64),
                        ("fp4_data_bytes", [i64, i64], i64),
                        ("fp4_scale_bytes", [i64, i64, i32], i64),
                        ("fp4_quantize", [vp, i64, i64, i64, i32, i32, i32, vp, vp, vp], ctypes.c_int),
                        ("fp4_dequantize", [vp, vp, i64, i64, i32, i32, vp, i64, i32, vp], ctypes.c_int),
                        ("gemm_fp4_nt", [vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, f32, vp, opts], ctypes.c_int),
                        ("gemm_fp4_nt_describe", [i64, i64, i64, i32, opts, i32, ctypes.POINTER(Fp4LaunchInfo)], ctypes.c_int),
                        ("gemm_fp4_last_device_status", [vp, ctypes.POINTER(ctypes.c_uint64)], ctypes.c_int)):
                    fn = getattr(lib, name)
                    fn.argtypes, fn.restype = args, res
                _lib = lib
    return _lib


def _load_binding():
    from . import GemmError

    path = _build.build_binding()
    loader = importlib.machinery.ExtensionFileLoader("_linear_binding", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_linear_binding", loader, origin=path))
    loader.exec_module(module)
    module.set_error(GemmError)
    return module


class _Unloaded:
    """The binding before its first use, which puts the loaded one in its place."""

    def __getattr__(self, name):
        global _native
        with _lock:
            if _native is self:
                _native = _load_binding()
        return getattr(_native, name)


_native = _Unloaded()


def _on(stream, call, args, tensors):
    """call(*args) on `stream` (a torch stream or a handle), the tensors' memory kept until it has run."""
    import torch

    device = next((t.device for t in tensors if isinstance(t, torch.Tensor)), None)
    if device is None or device.type != "cuda":
        return call(*args)  # refused there
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        result = call(*args)
    for t in tensors:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return result


def _parts(q) -> tuple:
    """The tensors of an Fp4Tensor; of anything else, which the call refuses, itself."""
    return q[:2] if isinstance(q, tuple) else (q,)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, *, out=None, stream=None):
    """(y, mean, rstd) of layer norm over the last axis of x (float16, bfloat16 or float32).

    mean = sum(x) / n, rstd = 1 / sqrt(sum((x - mean)^2) / n + eps), y = (x - mean) * rstd * weight
    + bias.  weight and bias (x's dtype or float32; None: 1 and 0) are vectors of the last axis;
    mean and rstd are float32 of the leading axes' shape, as ``layer_norm_backward`` takes them.
    Sums are fp32, y is rounded once.  The last axis is contiguous and the others step evenly (any
    alignment).  ``out``: y's memory, which must not overlap x.
    """
    if stream is not None:
        return _on(stream, _native.layer_norm, (x, weight, bias, eps, out), (x, weight, bias, out))
    return _native.layer_norm(x, weight, bias, eps, out)


def layer_norm_backward(dy, x, weight, mean, rstd, *, dx=None, grad_dtype=None, stream=None):
    """(dx, dweight, dbias): the gradient of ``layer_norm`` at x, from its mean and rstd.

    dx has x's dtype and shape; dweight and dbias have weight's dtype.  Without a weight they are
    None unless ``grad_dtype`` (x's or float32) asks for them, as a norm with a bias alone does.  Sums over rows are fp32 in a fixed order: the same inputs give the same bits.  ``dx``:
    the memory for dx, which must not overlap the inputs.
    """
    if stream is not None:
        return _on(stream, _native.layer_norm_backward, (dy, x, weight, mean, rstd, dx, grad_dtype),
                   (dy, x, weight, mean, rstd, dx))
    return _native.layer_norm_backward(dy, x, weight, mean, rstd, dx, grad_dtype)


def quantize_fp4(x, format: str = "mx", *, exponent: int = 0, out: Fp4Tensor | None = None, stream=None) -> Fp4Tensor:
    """x (a matrix of float16, bfloat16 or float32) as microscaled 4-bit floats.

    With amax a block's largest magnitude, its scale is 2**(floor(log2(amax)) - 2) for "mx", and
    amax / 6 / 2**exponent rounded to E4M3 within [2**-9, 448], times 2**exponent, for "nv"; each
    element is x / scale rounded to E2M1, ties to the even code, magnitudes past 6 to 6.  A block
    that holds an infinity or NaN becomes NaN.  ``out``: the Fp4Tensor whose memory is written.
    """
    if stream is not None:
        data, scales = _on(stream, _native.quantize_fp4, (x, format, exponent, out),
                           (x, *_parts(out)))
    else:
        data, scales = _native.quantize_fp4(x, format, exponent, out)
    return Fp4Tensor(data, scales, x.shape[1], format, exponent) if out is None else out


def dequantize_fp4(q: Fp4Tensor, dtype=None, *, out=None, stream=None):
    """The values of q as a rows x cols matrix of `dtype` (None: torch.float32; it and, short of its
    range, bfloat16 hold every one exactly)."""
    if stream is not None:
        return _on(stream, _native.dequantize_fp4, (q, dtype, out), (*_parts(q), out))
    return _native.dequantize_fp4(q, dtype, out)


def gemm_fp4_nt(A: Fp4Tensor, B: Fp4Tensor, D=None, *, dtype=None, alpha: float = 1.0, stream=None,
                options: Fp4Options | None = None):
    """D = alpha * A·Bᵀ of the values of A (M×K) and B (N×K), both of one format; returns D (M×N; of
    `dtype` if none is given, None: torch.float16).

    The sum is fp32 on the tensor cores, D (float16, bfloat16 or float32) is rounded once.  "nv"
    matrices' exponents are brought in whatever their sum; alpha and they together may leave fp32's
    range.
    """
    if options is not None and not isinstance(options, Fp4Options):
        raise TypeError("options must be an Fp4Options")
    address = 0 if options is None else ctypes.addressof(options)
    if stream is not None:
        return _on(stream, _native.gemm_fp4_nt, (A, B, D, dtype, alpha, address), (*_parts(A), *_parts(B), D))
    return _native.gemm_fp4_nt(A, B, D, dtype, alpha, address)


def describe_fp4(M: int, N: int, K: int, format: str = "mx", options: Fp4Options | None = None, sms: int = 152) -> dict:
    """The tile, K split, side and CTAs that ``gemm_fp4_nt`` would launch on a device of `sms` SMs."""
    from . import GemmError

    if format not in _FORMATS:
        raise ValueError(f'format must be "mx" or "nv", not {format!r}')
    info = Fp4LaunchInfo()
    rc = load_linear().gemm_fp4_nt_describe(M, N, K, _FORMATS[format], options, sms, ctypes.byref(info))
    if rc != 0:
        raise GemmError(rc, "gemm_fp4_nt_describe")
    return {f: getattr(info, f) for f, _ in Fp4LaunchInfo._fields_}


def fp4_device_status(stream=None) -> tuple[int, int]:
    """(status, info) of the products' device status word, after synchronising `stream`; clears it."""
    import torch

    handle = torch.cuda.current_stream().cuda_stream if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
    info = ctypes.c_uint64(0)
    rc = load_linear().gemm_fp4_last_device_status(handle, ctypes.byref(info))
    return rc, info.value
