"""A pre-norm linear layer, y = layer_norm(x)·Wᵀ, in training and in serving, on the package's operators.

    python -m blackwell_tensor_core_02_gb300.prenorm --tokens 1 64 2048 --width 4096 --out 4096
    python -m blackwell_tensor_core_02_gb300.prenorm --tokens 8192 --width 4096 --out 28672 --format nv

Training runs in fp16: layer norm, the product, and their gradients (three products and the norm's
gradient).  Serving quantises the weights once and each call's normalised tokens, and multiplies the
4-bit matrices.  The command prints one JSON line per number of tokens: the time of a serving call,
of the fp16 forward and of a training step (CUDA events over a run of calls), and how far the served
result is from the fp16 one (2-norm, relative).
"""
from __future__ import annotations

import argparse
import json
import math
import os
import sys

_ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if _ROOT not in sys.path:
    sys.path.insert(0, _ROOT)

import torch

import blackwell_tensor_core_02_gb300 as g


class PreNormLinear:
    """y = layer_norm(x; scale, shift)·Wᵀ for x (tokens × width), W (out × width), all fp16.

    ``forward``/``backward`` are a training step's two passes; ``quantize`` makes the 4-bit copy of
    W that ``serve`` uses.  Widths, outputs and, in ``backward``, tokens are multiples of 8
    (``gemm_f16_nt``'s shapes); ``serve`` takes any.
    """

    def __init__(self, weight, scale, shift, eps: float = 1e-5):
        self.weight, self.scale, self.shift, self.eps = weight, scale, shift, eps
        self.weight4 = None

    def forward(self, x):
        """(y, what ``backward`` needs)."""
        h, mean, rstd = g.layer_norm(x, self.scale, self.shift, self.eps)
        return g.gemm_f16_nt(h, self.weight), (x, h, mean, rstd)

    def backward(self, dy, kept):
        """(dx, dweight, dscale, dshift) for the gradient dy of y."""
        x, h, mean, rstd = kept
        dh = g.gemm_f16_nt(dy, self.weight.t().contiguous())                # dy·W
        dweight = g.gemm_f16_nt(dy.t().contiguous(), h.t().contiguous())    # dyᵀ·h
        dx, dscale, dshift = g.layer_norm_backward(dh, x, self.scale, mean, rstd)
        return dx, dweight, dscale, dshift

    def quantize(self, format: str = "mx") -> None:
        # "nv" scales reach from 2^-9 to 448: one exponent brings a layer's weights, some
        # 1 / sqrt(width) in size, into their middle (0 for weights that have none: zeros, or
        # with an infinity or NaN)
        size = 0.0 if format == "mx" else float(torch.log2(self.weight.float().abs().amax() / 6))
        exponent = round(size) - 3 if format != "mx" and math.isfinite(size) else 0
        self.weight4 = g.quantize_fp4(self.weight, format, exponent=max(-100, min(100, exponent)))

    def serve(self, x):
        h = g.layer_norm(x, self.scale, self.shift, self.eps)[0]
        return g.gemm_fp4_nt(g.quantize_fp4(h, self.weight4.format), self.weight4)


def make_layer(width: int, out: int, seed: int = 0) -> PreNormLinear:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    weight = (torch.randn(out, width, generator=gen, device="cuda") * width ** -0.5).half()
    scale = (1 + 0.1 * torch.randn(width, generator=gen, device="cuda")).half()
    shift = (0.1 * torch.randn(width, generator=gen, device="cuda")).half()
    return PreNormLinear(weight, scale, shift)


def _time(call, steps: int) -> float:
    """Microseconds a call, after a warm-up, from CUDA events around `steps` calls."""
    for _ in range(3):
        call()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    for _ in range(steps):
        call()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) / steps * 1e3


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, nargs="+", default=[1, 64, 2048])
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--out", type=int, default=4096)
    ap.add_argument("--format", choices=["mx", "nv"], default="mx")
    ap.add_argument("--steps", type=int, default=50)
    args = ap.parse_args(argv)
    layer = make_layer(args.width, args.out)
    layer.quantize(args.format)
    for tokens in args.tokens:
        x = torch.randn(tokens, args.width, device="cuda").half()
        y, kept = layer.forward(x)
        served = layer.serve(x)
        line = {"tokens": tokens, "width": args.width, "out": args.out, "format": args.format,
                "serve_us": round(_time(lambda: layer.serve(x), args.steps), 2),
                "forward_us": round(_time(lambda: layer.forward(x), args.steps), 2),
                "served_off": round(float((served.float() - y.float()).norm() / y.float().norm()), 4)}
        if tokens % 8 == 0:
            dy = torch.randn_like(y)
            line["step_us"] = round(_time(lambda: layer.backward(dy, layer.forward(x)[1]), args.steps), 2)
        status = g.fp4_device_status()[0] or g.last_device_status()[0]
        print(json.dumps({**line, "status": status}), flush=True)


if __name__ == "__main__":
    main()
