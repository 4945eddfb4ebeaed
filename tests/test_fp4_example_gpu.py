"""The example block runs the 4-bit operators together; it must agree with FP32 products on the same weights.

Linear layer and mixture round to bfloat16 (half a unit, 2^-8, at most; about half of that in the
2-norm) and x itself passes unchanged, so the block is within 2^-7 of the 32-bit computation.
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
    spec = importlib.util.spec_from_file_location("fp4_block", os.path.join(ROOT, "examples", "fp4_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("args", [["--width", "512", "--hidden", "96", "--experts", "8", "--top", "2"],
                                  ["--width", "300", "--hidden", "70", "--experts", "5", "--tokens", "1", "--format", "mxfp4"],
                                  ["--width", "256", "--hidden", "64", "--experts", "40", "--tokens", "18", "--top", "6"]])
def test_block_agrees_with_32_bits(example, args):
    assert example.main(args) <= 2.0 ** -7
