"""A feed-forward block trained with activations kept in 8 bits, then served with weights in 8 bits.

    python examples/int8_block.py [--tokens 4096] [--width 1024] [--hidden 2048] [--steps 20]

The block is y = down(swiglu(gate_up(x))), its weights and activations in 32 bits.

Training.  A step's forward pass keeps x, gate, up and h as integers of 8 bits with a power of two for each 32
channels of a token (``int8_checkpoint``, ``int8_swiglu``), 1.06 bytes a value instead of 4, and its backward pass
takes the weights' gradients and the gated activation's from them:

    gate_up = x W1^T                  sgemm (FP32)
    h       = swiglu(gate, up)        int8_swiglu, keeps gate and up
    y       = h W2^T                  sgemm
    dW2     = dy^T h                  int8_weight_grad, from the kept h
    dh      = dy W2                   sgemm
    dgate, dup                        int8_swiglu_backward, from the kept gate and up
    dW1     = dgate_up^T x            int8_weight_grad, from the kept x

The gradients are compared with those of the formulas in 64 bits, once from the values that were kept (rounding of
32 bits apart) and once from x, gate, up and h themselves (what 8 bits cost).

Serving.  The weights become integers with a scale for each channel (``int8_quantize``); a token's activations are
quantised within the linear layers (``int8_linear``).
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_fp32_gemm_03_gb300 as sg


def product(a, b, trans_a=False, trans_b=False):
    """op(a) @ op(b) in FP32."""
    shape = a.shape[1] if trans_a else a.shape[0], b.shape[0] if trans_b else b.shape[1]
    return sg.sgemm_ex2(a, b, torch.empty(shape, device=a.device), trans_a=trans_a, trans_b=trans_b)


class Block:
    def __init__(self, width, hidden, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden = hidden
        self.w1 = torch.randn(2 * hidden, width, generator=gen, device="cuda") / width ** 0.5
        self.w2 = torch.randn(width, hidden, generator=gen, device="cuda") / hidden ** 0.5

    def forward(self, x):
        """(y, what the backward pass needs)"""
        gate_up = product(x, self.w1, trans_b=True)
        h, kept = sg.int8_swiglu(gate_up[:, :self.hidden], gate_up[:, self.hidden:])
        return product(h, self.w2, trans_b=True), (sg.int8_checkpoint(x), kept, sg.int8_checkpoint(h))

    def backward(self, dy, saved):
        """(dx, dW1, dW2)"""
        x, kept, h = saved
        dw2 = sg.int8_weight_grad(dy, h)
        d = torch.empty(dy.shape[0], 2 * self.hidden, device="cuda")
        sg.int8_swiglu_backward(product(dy, self.w2), kept, out=(d[:, :self.hidden], d[:, self.hidden:]))
        return product(d, self.w1), sg.int8_weight_grad(d, x), dw2

    def in_64_bits(self, x, dy, gate=None, up=None, h=None):
        """(y, dx, dW1, dW2) by the formulas; gate, up and h of the backward pass may be given."""
        x, dy, w1, w2 = x.double(), dy.double(), self.w1.double(), self.w2.double()
        g, u = (x @ w1.t()).split(self.hidden, 1)
        a = g * torch.sigmoid(g) * u
        y = a @ w2.t()
        g, u, a = (v if given is None else given.double() for v, given in ((g, gate), (u, up), (a, h)))
        s, dh = torch.sigmoid(g), dy @ w2
        d = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1)
        return y, d @ w1, d.t() @ x, dy.t() @ a

    def serve(self):
        """The block as a function of a few tokens, on weights of 8 bits."""
        w1, w2 = sg.int8_quantize(self.w1), sg.int8_quantize(self.w2)

        def call(x):
            g, u = sg.int8_linear(x, w1).split(self.hidden, 1)
            return sg.int8_linear(torch.nn.functional.silu(g) * u, w2)
        return call


def far(a, b):
    return float((a.double() - b).norm() / b.norm())


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--width", type=int, default=1024)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args(argv)
    block = Block(a.width, a.hidden)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.width, generator=gen, device="cuda")
    target = torch.randn(a.tokens, a.width, generator=gen, device="cuda")

    # Gradients of |y - target|^2 / 2 per value.
    y, saved = block.forward(x)
    dy = (y - target) / y.numel()
    grads = block.backward(dy, saved)
    kept_x, (gate, up), kept_h = saved
    exact = block.in_64_bits(x, dy)
    of_kept = block.in_64_bits(kept_x.restore(), dy, gate.restore(), up.restore(), kept_h.restore())
    result = {"y": far(y, exact[0])}
    for i, name in enumerate(("dx", "dw1", "dw2")):
        result[name], result[name + " kept"] = far(grads[i], exact[1 + i]), far(grads[i], of_kept[1 + i])
    nbytes = sum(c.nbytes for c in (kept_x, gate, up, kept_h))
    result["bytes a value"] = nbytes / (x.numel() + 3 * a.tokens * a.hidden)

    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        y, saved = block.forward(x)
        _, dw1, dw2 = block.backward((y - target) / y.numel(), saved)
        block.w1.add_(dw1, alpha=-1.0)
        block.w2.add_(dw2, alpha=-1.0)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - start) / max(1, a.steps) * 1e3

    serve = block.serve()
    tokens = x[:4].bfloat16()
    result["served"] = far(serve(tokens), block.in_64_bits(tokens, dy[:4])[0])
    print(f"{a.tokens} tokens, width {a.width}, hidden {a.hidden}: {ms:.2f} ms a step, {result['bytes a value']:.3f} bytes a kept value; "
          + ", ".join(f"{k} {v:.1e}" for k, v in result.items() if k != "bytes a value"))
    return result


if __name__ == "__main__":
    main()
