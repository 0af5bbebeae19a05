"""Layer norm that keeps 8 bits an element for its backward pass.

Over the C ABI of ``include/checkpoint_ops.h`` (library ``_build/liblinear_ops.so``), by the binding and
in the manner of ``linear.py``.  In place of its input, and of its result for the product behind it, the
norm keeps its normalised rows h = (x - mean) * rstd as microscaled 8-bit floats, from which its result
and its gradient follow:

    y, kept, rstd = g.layer_norm_checkpoint(x, weight, bias)
    y = g.layer_norm_restore(kept, weight, bias, dtype)             # before the weights' gradient
    dx, dweight, dbias = g.layer_norm_backward_checkpoint(dy, kept, weight, rstd)

1.03 bytes an element stay between the passes, of 16-bit x and y 4.
"""
from __future__ import annotations

from typing import TYPE_CHECKING, NamedTuple

from . import linear as _linear

if TYPE_CHECKING:
    import torch

__all__ = ["Fp8Rows", "layer_norm_checkpoint", "layer_norm_restore", "layer_norm_backward_checkpoint"]


class Fp8Rows(NamedTuple):
    """Rows of microscaled 8-bit floats: E4M3 codes with a power-of-two scale for 32 of a row.

    ``codes``: float8_e4m3fn of the rows' shape.  ``scales``: uint8, one for each 32 (or fewer) of the
    last axis, E8M0: 2**(code - 127), 255 NaN.  The value of an element is its code's times its scale.
    """
    codes: torch.Tensor
    scales: torch.Tensor


def _parts(kept) -> tuple:
    return tuple(kept) if isinstance(kept, tuple) else (kept,)


def layer_norm_checkpoint(x, weight=None, bias=None, eps: float = 1e-5, *, out=None, stream=None):
    """(y, kept, rstd): ``layer_norm`` of x, and what its backward pass needs.

    With h = (x - mean) * rstd, y = h * weight + bias, and ``kept`` (an Fp8Rows) holds h: with amax
    the largest magnitude of 32 elements of a row, their scale is 2**(floor(log2(amax)) - 8), and each is
    h / scale rounded to E4M3, ties to the even code, magnitudes past 448 to 448.  A block that holds an
    infinity or NaN becomes NaN.  x, weight, bias, eps and ``out`` are as ``layer_norm`` takes them.
    """
    if stream is None:
        y, codes, scales, rstd = _linear._native.layer_norm_checkpoint(x, weight, bias, eps, out)
    else:
        y, codes, scales, rstd = _linear._on(stream, _linear._native.layer_norm_checkpoint, (x, weight, bias, eps, out),
                                             (x, weight, bias, out))
    return y, Fp8Rows(codes, scales), rstd


def layer_norm_restore(kept: Fp8Rows, weight=None, bias=None, dtype=None, *, out=None, stream=None):
    """y = h * weight + bias from the kept rows, rounded once to `dtype` (None: weight's, or float32).

    weight and bias have `dtype` or float32; without either y holds the kept values.
    """
    if stream is None:
        return _linear._native.layer_norm_restore(kept, weight, bias, dtype, out)
    return _linear._on(stream, _linear._native.layer_norm_restore, (kept, weight, bias, dtype, out),
                       (*_parts(kept), weight, bias, out))


def layer_norm_backward_checkpoint(dy, kept: Fp8Rows, weight, rstd, *, dx=None, grad_dtype=None, stream=None):
    """(dx, dweight, dbias): ``layer_norm_backward`` with the kept rows for (x - mean) * rstd.

    dx has dy's dtype and shape; weight, ``dx`` and ``grad_dtype`` are as ``layer_norm_backward`` takes
    them.  The same inputs give the same bits.
    """
    if stream is None:
        return _linear._native.layer_norm_backward_checkpoint(dy, kept, weight, rstd, dx, grad_dtype)
    return _linear._on(stream, _linear._native.layer_norm_backward_checkpoint, (dy, kept, weight, rstd, dx, grad_dtype),
                       (dy, *_parts(kept), weight, rstd, dx))
