"""The example block runs the 8-bit operators together; its gradients are those of the formulas.

From the kept values they differ by the arithmetic of 32 bits: sums of K products in FP32, at most K 2^-24 of the sum of
their magnitudes (and as a rule far less), through at most three products one after another; 1e-5 of the 2-norm covers
K up to 1000.  From the activations themselves they differ by what 8 bits keep: a value is off by at most 2^-7 of its
block's largest, less than 2^-8 of it in the mean, and x, gate, up and h each add their own, so that 2^-5 covers all four.
Served with 8-bit weights and activations, two linear layers round two operands each by up to 2^-8 of a row's largest
value, which is about four times its root mean square: 4 * 2^-8 / sqrt(3) a time, four times, and the roundings of bfloat16.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("int8_block", os.path.join(ROOT, "examples", "int8_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("args", [["--tokens", "700", "--width", "256", "--hidden", "300", "--steps", "2"],
                                  ["--tokens", "65", "--width", "130", "--hidden", "72", "--steps", "1"]])
def test_gradients_are_the_formulas(example, args):
    r = example.main(args)
    assert r["y"] < 1e-5
    # dx and dW1 go through the exact forward values of x (in W1's product) and the kept gate and up.
    assert r["dw2 kept"] < 1e-5 and r["dw1 kept"] < 1e-5 and r["dx kept"] < 1e-5
    for name in ("dx", "dw1", "dw2"):
        assert r[name] < 2.0 ** -5
    assert r["served"] < 4 * 4 * 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -7
    # Lines of codes are padded to 16 bytes, of units (two bytes a block of 32 channels) to 16 too.
    tokens, width, hidden = (int(args[i]) for i in (1, 3, 5))
    up = lambda n, m: -(-n // m) * m  # noqa: E731
    channels = lambda c: c * up(tokens, 16) + -(-c // 32) * up(tokens, 8) * 2  # noqa: E731
    rows = tokens * (up(hidden, 16) + 2 * up(-(-hidden // 32), 8))
    assert r["bytes a value"] * tokens * (width + 3 * hidden) == pytest.approx(channels(width) + channels(hidden) + 2 * rows)
