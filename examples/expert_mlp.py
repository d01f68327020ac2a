"""An expert MLP layer from end to end on one GPU: routing, the grouped products
forward and backward, and the same layer served in 4 bits.

    python examples/expert_mlp.py [--tokens T] [--experts E] [--top K]
                                  [--width D] [--hidden H] [--format mx|nv]

Each token goes to its ``top`` most likely experts; expert e computes
SiLU(x W1_e) * (x W2_e) W_down_e, and a token's results are summed with the
router's weights.  Rows are sorted by expert, and ``offsets`` -- made on the
GPU, never read by the host -- says where each expert's rows begin.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import swiglu_mlp_gb300 as swg  # noqa: E402

FORMATS = {"mx": swg.MXFP4, "nv": swg.NVFP4}


def route(logits, top):
    """(rows' tokens, their weights, offsets): rows sorted by expert."""
    weight, expert = logits.float().softmax(-1).topk(top, -1)
    weight = weight / weight.sum(-1, keepdim=True)
    order = expert.flatten().argsort(stable=True)
    counts = torch.bincount(expert.flatten(), minlength=logits.shape[1])
    offsets = torch.zeros(logits.shape[1] + 1, dtype=torch.int32, device=logits.device)
    offsets[1:] = counts.cumsum(0)
    return order // top, weight.flatten()[order], offsets


class ExpertMLP:
    """Weights of E gated MLPs of width D and hidden size H, bfloat16."""

    def __init__(self, experts, width, hidden, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.E, self.D, self.H = experts, width, hidden
        self.w_fused = normal(experts, width, 2 * hidden, std=width ** -0.5)   # Gate, Up by columns
        self.w_down = normal(experts, hidden, width, std=hidden ** -0.5)

    def forward(self, x, offsets):
        """(rows' results, the gated activation)."""
        y = torch.empty((x.shape[0], self.H), dtype=x.dtype, device=x.device)
        swg.swiglu_grouped_into(y, x, self.w_fused, offsets)
        out = torch.empty_like(x)
        return swg.gemm_grouped_into(out, y, self.w_down, offsets), y

    def backward(self, x, d_out, offsets):
        """Gradients of x, w_fused and w_down; Gate, Up and the activation are
        computed again from x."""
        like = dict(dtype=x.dtype, device=x.device)
        dy = torch.empty((x.shape[0], self.H), **like)
        swg.gemm_grouped_into(dy, d_out, self.w_down, offsets, transB=1)
        y, dh = torch.empty_like(dy), torch.empty((x.shape[0], 2 * self.H), **like)
        swg.swiglu_grouped_grad_into(dh, x, self.w_fused, dy, offsets, Y=y)
        dx = swg.gemm_grouped_into(torch.empty_like(x), dh, self.w_fused, offsets, transB=1)
        dw = swg.gemm_grouped_wgrad_into(torch.empty_like(self.w_fused), x, dh, offsets)
        dd = swg.gemm_grouped_wgrad_into(torch.empty_like(self.w_down), y, d_out, offsets)
        return dx, dw, dd


class ExpertMLP4:
    """The same layer with weights and activations in 4 bits."""

    def __init__(self, mlp, fmt):
        self.fmt, self.E, self.D, self.H = FORMATS[fmt], mlp.E, mlp.D, mlp.H
        self.up = self._weight(mlp.w_fused.transpose(1, 2))       # 2H rows of D, Gate and Up by rows
        self.down = self._weight(mlp.w_down.transpose(1, 2))      # D rows of H

    def _weight(self, w):
        """Codes and scale tiles of [E, rows, K]; each expert's rows are a group."""
        E, rows, K = w.shape
        begin = torch.arange(E + 1, dtype=torch.int32, device=w.device) * rows
        q, s = swg.mx4_alloc(E * rows, K, self.fmt, groups=E)
        swg.mx4_quantize_into(q, s, w.reshape(E * rows, K).contiguous(), self.fmt, offsets=begin)
        return q.view(E, rows, -1), s

    def _rows(self, x, offsets):
        q, s = swg.mx4_alloc(x.shape[0], x.shape[1], self.fmt, groups=self.E)
        return swg.mx4_quantize_into(q, s, x, self.fmt, offsets=offsets)

    def forward(self, x, offsets):
        y = torch.empty((x.shape[0], self.H), dtype=x.dtype, device=x.device)
        swg.swiglu_mx4_into(y, *self._rows(x, offsets), *self.up, self.D, self.fmt, offsets=offsets)
        out = torch.empty_like(x)
        return swg.gemm_mx4_into(out, *self._rows(y, offsets), *self.down, self.H, self.fmt,
                                 offsets=offsets)


def combine(rows, tokens, weights, count):
    out = torch.zeros((count, rows.shape[1]), dtype=torch.float32, device=rows.device)
    return out.index_add_(0, tokens, rows.float() * weights[:, None])


def microseconds(f, repeats=20):
    for _ in range(3):
        f()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(repeats):
        f()
    end.record()
    end.synchronize()
    return begin.elapsed_time(end) * 1e3 / repeats


def main(argv=None):
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--tokens", type=int, default=4096)
    a.add_argument("--experts", type=int, default=16)
    a.add_argument("--top", type=int, default=2)
    a.add_argument("--width", type=int, default=4096)
    a.add_argument("--hidden", type=int, default=1792)
    a.add_argument("--format", choices=sorted(FORMATS), default="mx")
    a = a.parse_args(argv)

    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((a.tokens, a.width), generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn((a.tokens, a.experts), generator=g, device="cuda")
    tokens, weights, offsets = route(logits, a.top)
    rows = x[tokens]

    mlp = ExpertMLP(a.experts, a.width, a.hidden)
    out, _ = mlp.forward(rows, offsets)
    d_out = torch.randn_like(out)
    dx, dw, dd = mlp.backward(rows, d_out, offsets)
    mlp4 = ExpertMLP4(mlp, a.format)
    out4 = mlp4.forward(rows, offsets)
    if swg.get_device_error() != 0:
        raise RuntimeError("device error word set")
    result = combine(out, tokens, weights, a.tokens)
    result4 = combine(out4, tokens, weights, a.tokens)
    off = float((result4 - result).norm() / result.norm())
    n = rows.shape[0]
    flops = 6 * n * a.width * a.hidden
    for name, f, work in (("forward", lambda: mlp.forward(rows, offsets), flops),
                          ("backward", lambda: mlp.backward(rows, d_out, offsets), 2 * flops + flops * 2 // 3),
                          ("4-bit forward", lambda: mlp4.forward(rows, offsets), flops)):
        us = microseconds(f)
        print(f"{name:14s} {us:9.1f} us  {work / us / 1e6:8.0f} TFLOP/s  ({n} rows, {a.experts} experts)")
    print(f"4-bit result is {off:.3f} of its norm off the 16-bit one ({a.format})")
    return {"result": result, "result4": result4, "off": off, "grads": (dx, dw, dd),
            "mlp": mlp, "rows": rows, "d_out": d_out, "offsets": offsets, "tokens": tokens,
            "weights": weights, "x": x}


if __name__ == "__main__":
    main()
