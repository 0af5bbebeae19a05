"""The operators around a linear layer's product: layer norm and its gradient, quantisation to
microscaled 4-bit floats, and the product of two such matrices.

Argument marshalling over the C ABI of ``include/linear_ops.h`` (library ``_build/liblinear_ops.so``),
as the package's ``gemm_f16_nt`` is over its own: PyTorch supplies memory and streams, every step of
the computation runs in the library, and there is no fallback.

    y, mean, rstd = g.layer_norm(x, weight, bias)
    dx, dweight, dbias = g.layer_norm_backward(dy, x, weight, mean, rstd)
    W = g.quantize_fp4(w)                       # once
    D = g.gemm_fp4_nt(g.quantize_fp4(y), W)     # = y @ w.T of the quantised values

With ``stream=`` a call runs on that stream; what it allocates belongs to that stream, and the
inputs' memory is kept from reuse until the call has run.
"""
from __future__ import annotations

import ctypes
import threading
from typing import NamedTuple

import torch

from . import build as _build

__all__ = ["layer_norm", "layer_norm_backward", "Fp4Tensor", "quantize_fp4", "dequantize_fp4", "gemm_fp4_nt",
           "Fp4Options", "describe_fp4", "fp4_device_status"]

_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_FORMATS = {"mx": 0, "nv": 1}


class Fp4Options(ctypes.Structure):
    """Mirror of ``gemm_fp4_options`` (zero fields mean defaults)."""
    _fields_ = [("tile", ctypes.c_int32), ("cluster_k", ctypes.c_int32), ("swap", ctypes.c_int32),
                ("max_clusters", ctypes.c_int32), ("debug_flags", ctypes.c_int32), ("timeout_ns", ctypes.c_int64)]


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
    """Build (if stale) and load the library; raise if that is impossible."""
    global _lib
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


# The stream's handle of a device, without building a Stream object for it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _raise(code: int, where: str):
    from . import GemmError

    raise GemmError(code, where)


def _enqueue(body, device, stream, inputs):
    """body(stream handle) with `device` current; on `stream` if one is given (a torch stream or a
    handle), with the inputs' memory kept until it has run."""
    index = device.index
    if stream is None:
        if torch.cuda.current_device() == index:
            return body(_raw_stream(index))
        with torch.cuda.device(index):
            return body(_raw_stream(index))
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        result = body(stream.cuda_stream)
    for t in inputs:
        if t is not None:
            t.record_stream(stream)
    return result


def _dtype(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float16, bfloat16 or float32, not {t.dtype}")
    return code


def _rows(t, name):
    """(rows, cols, row stride) of a CUDA tensor whose last axis is contiguous and whose other axes
    step evenly (a matrix, or what views as one)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError(f"{name} must have at least one axis")
        cols = t.shape[-1]
        rows = 1
        for n in t.shape[:-1]:
            rows *= n
        try:
            t = t.view(rows, cols)
        except RuntimeError as e:
            raise ValueError(f"{name}: its rows do not step evenly; make it contiguous") from e
    rows, cols = t.shape
    step, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name}: its last axis must be contiguous")
    return rows, cols, step


def _vector(t, name, cols, device, dtype=None):
    if t.dim() != 1 or t.shape[0] != cols or (cols > 1 and t.stride(0) != 1) or t.device != device:
        raise ValueError(f"{name} must be a contiguous vector of {cols} elements on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    return t.data_ptr()


def _weight_dtype(x, *named):
    """The dtype of the weights given (all the same, x's or float32), x's if there is none."""
    dtype = None
    for name, t in named:
        if t is not None:
            if t.dtype != x.dtype and t.dtype != torch.float32:
                raise TypeError(f"{name} must be {x.dtype} or float32, not {t.dtype}")
            if dtype is not None and t.dtype != dtype:
                raise TypeError("weight and bias must have one dtype")
            dtype = t.dtype
    return dtype or x.dtype


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, *, out=None, stream=None):
    """(y, mean, rstd) of layer norm over the last axis of x (float16, bfloat16 or float32).

    mean = sum(x) / n, rstd = 1 / sqrt(sum((x - mean)^2) / n + eps), y = (x - mean) * rstd * weight
    + bias.  weight and bias (x's dtype or float32; None: 1 and 0) are vectors of the last axis;
    mean and rstd are float32 of the leading axes' shape, as ``layer_norm_backward`` takes them.
    Sums are fp32, y is rounded once.  ``out``: y's memory, which must not overlap x.
    """
    code = _dtype(x, "x")
    rows, cols, step = _rows(x, "x")
    if cols == 0:
        raise ValueError("x: rows of no elements have no norm")
    device = x.device
    wcode = _DTYPES[_weight_dtype(x, ("weight", weight), ("bias", bias))]
    w = None if weight is None else _vector(weight, "weight", cols, device)
    b = None if bias is None else _vector(bias, "bias", cols, device)
    if out is not None:
        if out.dtype != x.dtype or out.shape != x.shape or out.device != device:
            raise ValueError(f"out must be {x.dtype} of shape {tuple(x.shape)} on {device}")
        out_step = _rows(out, "out")[2]
    lib = load_linear()

    def body(handle):
        y = torch.empty(x.shape, dtype=x.dtype, device=device) if out is None else out
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
        rc = lib.layer_norm_forward(x.data_ptr(), step, w, b, y.data_ptr(), cols if out is None else out_step,
                                    mean.data_ptr(), rstd.data_ptr(), rows, cols, eps, code, wcode, handle)
        if rc != 0:
            _raise(rc, "layer_norm")
        return y, mean, rstd

    return _enqueue(body, device, stream, (x, weight, bias, out))


def layer_norm_backward(dy, x, weight, mean, rstd, *, dx=None, stream=None):
    """(dx, dweight, dbias): the gradient of ``layer_norm`` at x, from its mean and rstd.

    dx has x's dtype and shape; dweight and dbias have weight's dtype, and are None where weight is
    None.  Sums over rows are fp32 in a fixed order: the same inputs give the same bits.  ``dx``:
    the memory for dx, which must not overlap the inputs.
    """
    code = _dtype(x, "x")
    rows, cols, step = _rows(x, "x")
    if cols == 0:
        raise ValueError("x: rows of no elements have no norm")
    device = x.device
    if dy.dtype != x.dtype or dy.shape != x.shape or dy.device != device:
        raise ValueError(f"dy must be {x.dtype} of shape {tuple(x.shape)} on {device}")
    dy_step = _rows(dy, "dy")[2]
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or t.numel() != rows or not t.is_contiguous() or t.device != device:
            raise ValueError(f"{name} must be contiguous float32 of {rows} rows on {device}")
    wdtype = _weight_dtype(x, ("weight", weight))
    w = None if weight is None else _vector(weight, "weight", cols, device)
    if dx is not None:
        if dx.dtype != x.dtype or dx.shape != x.shape or dx.device != device:
            raise ValueError(f"dx must be {x.dtype} of shape {tuple(x.shape)} on {device}")
        dx_step = _rows(dx, "dx")[2]
    lib = load_linear()

    def body(handle):
        gx = torch.empty(x.shape, dtype=x.dtype, device=device) if dx is None else dx
        gw = gb = space = None
        need = 0
        if weight is not None:
            gw = torch.empty(cols, dtype=wdtype, device=device)
            gb = torch.empty(cols, dtype=wdtype, device=device)
            need = lib.layer_norm_backward_workspace_size(rows, cols)
            if need < 0:
                _raise(need, "layer_norm_backward")
            space = torch.empty(need, dtype=torch.uint8, device=device)
        rc = lib.layer_norm_backward(dy.data_ptr(), dy_step, x.data_ptr(), step, w, mean.data_ptr(), rstd.data_ptr(),
                                     gx.data_ptr(), cols if dx is None else dx_step,
                                     None if gw is None else gw.data_ptr(), None if gb is None else gb.data_ptr(),
                                     rows, cols, code, _DTYPES[wdtype], None if space is None else space.data_ptr(),
                                     need, handle)
        if rc != 0:
            _raise(rc, "layer_norm_backward")
        return gx, gw, gb

    return _enqueue(body, device, stream, (dy, x, weight, mean, rstd, dx))


def _format(name, exponent):
    code = _FORMATS.get(name)
    if code is None:
        raise ValueError(f'format must be "mx" or "nv", not {name!r}')
    if not -100 <= exponent <= 100 or (exponent and code == 0):
        raise ValueError('exponent must be in [-100, 100], and 0 for format "mx"')
    return code


def _fp4_shapes(rows, cols, code):
    units = -(-cols // 32)
    return (rows, units * 16), (-(-rows // 128), -(-units // (2 if code else 4)), 32, 4, 4)


def _check_fp4(q, name):
    """The format code of an Fp4Tensor whose parts fit together."""
    code = _format(q.format, q.exponent)
    data, scales = q.data, q.scales
    if data.dim() != 2 or q.cols < 0:
        raise ValueError(f"{name}: data must be [rows, bytes] and cols not negative")
    want = _fp4_shapes(data.shape[0], q.cols, code)
    if data.shape != want[0] or scales.shape != want[1]:
        raise ValueError(f"{name}: data and scales of {data.shape[0]} x {q.cols} are {want[0]} and {want[1]}, "
                         f"got {tuple(data.shape)} and {tuple(scales.shape)}")
    if data.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TypeError(f"{name}: data and scales must be uint8")
    if not (data.is_cuda and scales.device == data.device and data.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name}: data and scales must be contiguous tensors of one CUDA device")
    return code


def quantize_fp4(x, format: str = "mx", *, exponent: int = 0, out: Fp4Tensor | None = None, stream=None) -> Fp4Tensor:
    """x (a matrix of float16, bfloat16 or float32) as microscaled 4-bit floats.

    With amax a block's largest magnitude, its scale is 2**(floor(log2(amax)) - 2) for "mx", and
    amax / 6 / 2**exponent rounded to E4M3 within [2**-9, 448], times 2**exponent, for "nv"; each
    element is x / scale rounded to E2M1, ties to the even code, magnitudes past 6 to 6.  A block
    that holds an infinity or NaN becomes NaN.  ``out``: the Fp4Tensor whose memory is written.
    """
    code, fcode = _dtype(x, "x"), _format(format, exponent)
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    rows, cols, step = _rows(x, "x")
    device = x.device
    if out is not None and (_check_fp4(out, "out") != fcode or out.cols != cols or out.rows != rows
                            or out.exponent != exponent or out.data.device != device):
        raise ValueError("out must have x's shape and device, and the format and exponent asked for")
    lib = load_linear()

    def body(handle):
        q = out
        if q is None:
            data, scales = _fp4_shapes(rows, cols, fcode)
            q = Fp4Tensor(torch.empty(data, dtype=torch.uint8, device=device),
                          torch.empty(scales, dtype=torch.uint8, device=device), cols, format, exponent)
        rc = lib.fp4_quantize(x.data_ptr(), step, rows, cols, code, fcode, exponent, q.data.data_ptr(),
                              q.scales.data_ptr(), handle)
        if rc != 0:
            _raise(rc, "quantize_fp4")
        return q

    return _enqueue(body, device, stream, (x,) if out is None else (x, out.data, out.scales))


def dequantize_fp4(q: Fp4Tensor, dtype=torch.float32, *, out=None, stream=None):
    """The values of q as a rows x cols matrix of `dtype` (float32 and, short of its range, bfloat16
    hold every one exactly)."""
    fcode = _check_fp4(q, "q")
    if out is not None:
        dtype = out.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be float16, bfloat16 or float32, not {dtype}")
    rows, cols, device = q.rows, q.cols, q.data.device
    if out is not None and (out.shape != (rows, cols) or out.device != device):
        raise ValueError(f"out must be {rows} x {cols} on {device}")
    step = cols if out is None else _rows(out, "out")[2]
    lib = load_linear()

    def body(handle):
        y = torch.empty((rows, cols), dtype=dtype, device=device) if out is None else out
        rc = lib.fp4_dequantize(q.data.data_ptr(), q.scales.data_ptr(), rows, cols, fcode, q.exponent, y.data_ptr(), step,
                                _DTYPES[dtype], handle)
        if rc != 0:
            _raise(rc, "dequantize_fp4")
        return y

    return _enqueue(body, device, stream, (q.data, q.scales, out))


def gemm_fp4_nt(A: Fp4Tensor, B: Fp4Tensor, D=None, *, dtype=torch.float16, alpha: float = 1.0, stream=None,
                options: Fp4Options | None = None):
    """D = alpha * A·Bᵀ of the values of A (M×K) and B (N×K), both of one format; returns D (M×N).

    The sum is fp32 on the tensor cores, D (float16, bfloat16 or float32) is rounded once.
    """
    fcode = _check_fp4(A, "A")
    if _check_fp4(B, "B") != fcode:
        raise ValueError(f"A and B must have one format, got {A.format!r} and {B.format!r}")
    if A.cols != B.cols:
        raise ValueError(f"expected A (M×K) and B (N×K), got {A.rows}×{A.cols} and {B.rows}×{B.cols}")
    device = A.data.device
    if B.data.device != device:
        raise ValueError("A and B must be on one device")
    M, N = A.rows, B.rows
    if D is not None:
        dtype = D.dtype
        if tuple(D.shape) != (M, N) or not D.is_contiguous() or D.device != device:
            raise ValueError(f"D must be a contiguous {M}×{N} matrix on {device}")
    dcode = _DTYPES.get(dtype)
    if dcode is None:
        raise TypeError(f"D must be float16, bfloat16 or float32, not {dtype}")
    if A.exponent or B.exponent:
        alpha = alpha * 2.0 ** (A.exponent + B.exponent)
    lib = load_linear()

    def body(handle):
        d = torch.empty((M, N), dtype=dtype, device=device) if D is None else D
        rc = lib.gemm_fp4_nt(A.data.data_ptr(), A.scales.data_ptr(), B.data.data_ptr(), B.scales.data_ptr(), d.data_ptr(),
                             M, N, A.cols, fcode, dcode, alpha, handle, options)
        if rc != 0:
            _raise(rc, "gemm_fp4_nt")
        return d

    return _enqueue(body, device, stream, (A.data, A.scales, B.data, B.scales, D))


def describe_fp4(M: int, N: int, K: int, format: str = "mx", options: Fp4Options | None = None, sms: int = 152) -> dict:
    """The tile, K split, side and CTAs that ``gemm_fp4_nt`` would launch on a device of `sms` SMs."""
    info = Fp4LaunchInfo()
    rc = load_linear().gemm_fp4_nt_describe(M, N, K, _format(format, 0), options, sms, ctypes.byref(info))
    if rc != 0:
        _raise(rc, "gemm_fp4_nt_describe")
    return {f: getattr(info, f) for f, _ in Fp4LaunchInfo._fields_}


def fp4_device_status(stream=None) -> tuple[int, int]:
    """(status, info) of the products' device status word, after synchronising `stream`; clears it."""
    handle = torch.cuda.current_stream().cuda_stream if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
    info = ctypes.c_uint64(0)
    rc = load_linear().gemm_fp4_last_device_status(handle, ctypes.byref(info))
    return rc, info.value
