"""A pre-norm linear layer, y = layer_norm(x)·Wᵀ, in training and in serving, on the package's operators.

    python -m blackwell_tensor_core_02_gb300.prenorm --tokens 1 64 2048 --width 4096 --out 4096
    python -m blackwell_tensor_core_02_gb300.prenorm --tokens 8192 --width 4096 --out 28672 --format nv
    python -m blackwell_tensor_core_02_gb300.prenorm --tokens 64 --adapters 8 --rank 16
    python -m blackwell_tensor_core_02_gb300.prenorm --tokens 4096 --checkpoint --experts 16 --top 2

Training runs in fp16: layer norm, the product, and their gradients (three products and the norm's
gradient).  Serving quantises the weights once and each call's normalised tokens, and multiplies the
4-bit matrices.  The command prints one JSON line per number of tokens: the time of a serving call,
of the fp16 forward and of a training step (CUDA events over a run of calls), and how far the served
result is from the fp16 one (2-norm, relative).

``--checkpoint`` keeps the normalised rows in 8 bits between a training step's passes, in place of the
layer's input and of the norm's result.  ``--adapters`` serves the tokens in as many requests, each with
a low-rank adapter of its own beside the shared fp16 weights.  ``--experts`` runs the layer with a weight
matrix for each expert, each token through ``--top`` of them.
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
    """y = layer_norm(x; scale, shift)·Wᵀ for x (tokens × width), W (out × width), in fp16; scale and
    shift have that type or float32, or are None.

    ``forward``/``backward`` are a training step's two passes; ``quantize`` makes the 4-bit copy of
    W that ``serve`` uses.  Widths, outputs and, in ``backward``, tokens are multiples of 8
    (``gemm_f16_nt``'s shapes); ``serve`` takes any.  With ``checkpoint`` the normalised rows stay between
    the passes, in 8 bits (``layer_norm_checkpoint``), not x and the norm's result.
    """

    def __init__(self, weight, scale, shift, eps: float = 1e-5, checkpoint: bool = False):
        self.weight, self.scale, self.shift, self.eps, self.checkpoint = weight, scale, shift, eps, checkpoint
        self.weight4 = None

    def forward(self, x):
        """(y, what ``backward`` needs)."""
        if self.checkpoint:
            h, rows, rstd = g.layer_norm_checkpoint(x, self.scale, self.shift, self.eps)
            return g.gemm_f16_nt(h, self.weight), (rows, rstd)
        h, mean, rstd = g.layer_norm(x, self.scale, self.shift, self.eps)
        return g.gemm_f16_nt(h, self.weight), (x, h, mean, rstd)

    def backward(self, dy, kept):
        """(dx, dweight, dscale, dshift) for the gradient dy of y."""
        dh = g.gemm_f16_nt(dy, self.weight.t().contiguous())                # dy·W
        if self.checkpoint:
            rows, rstd = kept
            h = g.layer_norm_restore(rows, self.scale, self.shift, dh.dtype)
            dx, dscale, dshift = g.layer_norm_backward_checkpoint(dh, rows, self.scale, rstd)
        else:
            x, h, mean, rstd = kept
            dx, dscale, dshift = g.layer_norm_backward(dh, x, self.scale, mean, rstd)
        dweight = g.gemm_f16_nt(dy.t().contiguous(), h.t().contiguous())    # dyᵀ·h
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

    def serve_adapted(self, x, down, up, offsets, adapters, scales=None):
        """The fp16 layer for tokens of many requests, each with its own adapter (``gemm_lora_nt``)."""
        h = g.layer_norm(x, self.scale, self.shift, self.eps)[0]
        return g.gemm_lora_nt(h, self.weight, down, up, offsets, adapters, scales=scales)


class PreNormExperts:
    """y[t] = Σ_j gates[t, j]·layer_norm(x[t]; scale, shift)·W[chosen[t, j]]ᵀ, W (experts × out × width).

    x (tokens × width) and W share float16 or bfloat16, scale and shift have that type or float32, or are
    None; ``chosen`` (tokens × top, integers) names each token's experts, ``gates`` weighs them.  Widths and
    outputs are multiples of 8.  Between the passes the normalised rows stay in 8 bits; each token's rows
    are gathered from them again.
    """

    def __init__(self, weights, scale, shift, eps: float = 1e-5):
        self.weights, self.scale, self.shift, self.eps = weights, scale, shift, eps

    def route(self, chosen):
        """(token of each grouped row, place of each token's row among them, the groups' offsets); an
        expert out of range counts as none: its rows stand before or behind the groups."""
        experts = chosen.reshape(-1).long()  # small types do not hold the number of experts
        order = experts.argsort(stable=True)
        place = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=order.device))
        bounds = torch.arange(self.weights.shape[0] + 1, device=chosen.device)
        offsets = torch.searchsorted(experts[order], bounds)
        return order // max(chosen.shape[1], 1), place, offsets

    def forward(self, x, chosen, gates):
        """(y, what ``backward`` needs)."""
        h, rows, rstd = g.layer_norm_checkpoint(x, self.scale, self.shift, self.eps)
        token, place, offsets = self.route(chosen)
        out = g.grouped_gemm_nt(h[token], self.weights, offsets)
        y = (out[place].view(*chosen.shape, out.shape[1]).float() * gates.float()[..., None]).sum(1).to(x.dtype)
        return y, (rows, rstd, token, place, offsets, gates)

    def backward(self, dy, kept):
        """(dx, dweights, dscale, dshift, dgates) for the gradient dy of y."""
        rows, rstd, token, place, offsets, gates = kept
        h = g.layer_norm_restore(rows, self.scale, self.shift, dy.dtype)[token]
        dout = dy[token]
        dh = g.grouped_gemm_nn(dout, self.weights, offsets)                 # before the gates
        dgates = (dh.float() * h.float()).sum(1)[place].view(gates.shape)
        row_gates = gates.new_empty(gates.numel()).scatter_(0, place, gates.reshape(-1))
        dweights = g.grouped_gemm_tn((dout.float() * row_gates.float()[:, None]).to(dy.dtype), h, offsets)
        dh = (dh[place].view(*gates.shape, dh.shape[1]).float() * gates.float()[..., None]).sum(1).to(dy.dtype)
        dx, dscale, dshift = g.layer_norm_backward_checkpoint(dh, rows, self.scale, rstd)
        return dx, dweights, dscale, dshift, dgates.to(gates.dtype)


def make_layer(width: int, out: int, seed: int = 0, checkpoint: bool = False) -> PreNormLinear:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    weight = (torch.randn(out, width, generator=gen, device="cuda") * width ** -0.5).half()
    scale = (1 + 0.1 * torch.randn(width, generator=gen, device="cuda")).half()
    shift = (0.1 * torch.randn(width, generator=gen, device="cuda")).half()
    return PreNormLinear(weight, scale, shift, checkpoint=checkpoint)


def make_adapters(layer: PreNormLinear, adapters: int, rank: int, seed: int = 0):
    """(down, up, scales) of as many random adapters for the layer, fp16 and fp32."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out, width = layer.weight.shape
    down = (torch.randn(adapters, rank, width, generator=gen, device="cuda") * width ** -0.5).half()
    up = (torch.randn(adapters, out, rank, generator=gen, device="cuda") * rank ** -0.5).half()
    return down, up, torch.rand(adapters, generator=gen, device="cuda") + 0.5


def make_experts(width: int, out: int, experts: int, seed: int = 0, dtype=torch.bfloat16) -> PreNormExperts:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    weights = (torch.randn(experts, out, width, generator=gen, device="cuda") * width ** -0.5).to(dtype)
    scale = (1 + 0.1 * torch.randn(width, generator=gen, device="cuda")).to(dtype)
    shift = (0.1 * torch.randn(width, generator=gen, device="cuda")).to(dtype)
    return PreNormExperts(weights, scale, shift)


def even_offsets(tokens: int, requests: int):
    """Offsets of as many requests of nearly as many tokens each, on the device."""
    return torch.tensor([tokens * i // requests for i in range(requests + 1)], device="cuda")


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
    ap.add_argument("--checkpoint", action="store_true", help="keep 8 bits an element between a training step's passes")
    ap.add_argument("--adapters", type=int, default=0, help="serve as many requests, each with its own adapter")
    ap.add_argument("--rank", type=int, default=16, help="the adapters' rank")
    ap.add_argument("--experts", type=int, default=0, help="run the layer with as many experts")
    ap.add_argument("--top", type=int, default=2, help="experts of each token")
    args = ap.parse_args(argv)
    layer = make_layer(args.width, args.out, checkpoint=args.checkpoint)
    layer.quantize(args.format)
    adapters = make_adapters(layer, args.adapters, args.rank) if args.adapters else None
    experts = make_experts(args.width, args.out, args.experts) if args.experts else None
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
        if adapters:
            down, up, scales = adapters
            offsets = even_offsets(tokens, args.adapters)
            chosen = torch.arange(args.adapters, device="cuda", dtype=torch.int32)
            line["adapted_us"] = round(_time(lambda: layer.serve_adapted(x, down, up, offsets, chosen, scales), args.steps), 2)
        if experts:
            xe = x.to(experts.weights.dtype)
            chosen = torch.rand(tokens, args.experts, device="cuda").topk(args.top).indices
            gates = torch.rand(tokens, args.top, device="cuda").softmax(1)
            dy = torch.randn(tokens, args.out, device="cuda").to(xe.dtype)
            line["experts_forward_us"] = round(_time(lambda: experts.forward(xe, chosen, gates), args.steps), 2)
            line["experts_step_us"] = round(_time(lambda: experts.backward(dy, experts.forward(xe, chosen, gates)[1]), args.steps), 2)
        status = g.fp4_device_status()[0] or g.last_device_status()[0] or g.grouped_device_status()[0]
        print(json.dumps({**line, "status": status}), flush=True)


if __name__ == "__main__":
    main()
