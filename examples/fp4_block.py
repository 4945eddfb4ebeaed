"""A feed-forward block of a language model's decode step on 4-bit weights.

    python examples/fp4_block.py [--tokens 4] [--width 2048] [--experts 32] [--hidden 768] [--top 4] [--format nvfp4]

The block is a linear layer, a mixture of experts and a residual connection:

    a = x W_in^T                      fp4_linear (x quantised within the call)
    y = x + moe(a)                    fp4_moe (activations kept to the precision of their type)

Weights are quantised once (``fp4_quantize``; ``fp4_experts`` lays the experts' out).  The same block is then
computed in 32 bits, with the library's FP32 product on the values that the codes stand for
(``fp4_dequantize``), to show how far the two are apart: for the mixture it is the rounding of the types,
for the linear layer also the rounding of x to 4 bits.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_fp32_gemm_03_gb300 as sg


def factor(x, fmt):
    """nvfp4's factor of a matrix: its largest magnitude becomes the largest value that the format holds."""
    return (x.abs().amax().float() / 2688).reshape(1) if fmt == "nvfp4" else None


class Block:
    def __init__(self, width, hidden, experts, top, fmt, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weights(rows, cols):
            w = torch.randn(rows, cols, generator=gen, device="cuda") / cols ** 0.5
            return sg.fp4_quantize(w, fmt, scale=factor(w, fmt))
        self.format, self.top, self.experts, self.hidden, self.width = fmt, top, experts, hidden, width
        self.w_in = weights(width, width)
        self.gate_up = weights(experts * 2 * hidden, width)   # kept for the 32-bit computation only
        self.down = weights(experts * width, hidden)
        self.router = torch.randn(experts, width, generator=gen, device="cuda") / width ** 0.5
        self.layer = sg.fp4_experts(self.gate_up, self.down, experts)

    def __call__(self, x, x_scale):
        a = sg.fp4_linear(x, self.w_in, x_scale=x_scale)
        return x + sg.fp4_moe(a, self.router, self.layer, self.top)

    def in_32_bits(self, x, x_scale):
        """The same block from the values of the codes, with FP32 products."""
        xq = sg.fp4_quantize(x, self.format, scale=x_scale).dequantize()
        a = sg.sgemm(xq, self.w_in.dequantize().t().contiguous()).to(x.dtype).float()
        logits = sg.sgemm(a, self.router.t().contiguous())
        p, ids = logits.softmax(-1).topk(self.top, -1)
        p = p / p.sum(-1, keepdim=True)
        up = self.gate_up.dequantize().view(self.experts, 2 * self.hidden, self.width)
        down = self.down.dequantize().view(self.experts, self.width, self.hidden)
        y = x.float().clone()
        for t in range(x.shape[0]):
            for weight, e in zip(p[t], ids[t].tolist()):
                gu = sg.sgemm(a[t:t + 1], up[e].t().contiguous())
                h = torch.nn.functional.silu(gu[:, :self.hidden]) * gu[:, self.hidden:]
                y[t] += weight * sg.sgemm(h.contiguous(), down[e].t().contiguous())[0]
        return y


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=4)
    p.add_argument("--width", type=int, default=2048)
    p.add_argument("--hidden", type=int, default=768)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--top", type=int, default=4)
    p.add_argument("--format", choices=("mxfp4", "nvfp4"), default="nvfp4")
    a = p.parse_args(argv)
    block = Block(a.width, a.hidden, a.experts, a.top, a.format)
    x = torch.randn(a.tokens, a.width, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    scale = factor(x, a.format)
    y, exact = block(x, scale), block.in_32_bits(x, scale)
    error = float((y.float() - exact).norm() / exact.norm())
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(200):
        block(x, scale)
    torch.cuda.synchronize()
    us = (time.perf_counter() - start) / 200 * 1e6
    print(f"{a.tokens} tokens, width {a.width}, {a.experts} experts of {a.hidden}, top {a.top}, {a.format}: "
          f"{us:.1f} us a block, {error:.1e} from 32 bits on the same weights")
    return error


if __name__ == "__main__":
    main()
