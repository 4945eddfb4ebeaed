"""Rows of very small values (GPU)."""
import numpy as np
import pytest
import torch

import dense_fp32_gemm_03_gb300 as sg

import int8_ref as ref
from test_int8_gpu import F32, integers, matrix, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("low,high", [(1.0, 2.0), (2.0, 8.0)])
def test_quotients_next_to_a_tie_of_the_smallest_scales(low, high):
    """Scales from 2^-126 on, whose halves are not all 32-bit floats, and values at (n + 1/2) scales and one place to either side."""
    gen = np.random.default_rng(3)
    top = (gen.uniform(low, high, (64, 1)) * 127 * 2.0 ** -126).astype(np.float32)
    top[0] = np.float32(float.fromhex("0x1.9fc9cap-119"))
    s = np.maximum(top * (np.float32(1) / np.float32(127)), np.float32(2.0 ** -126))
    n = gen.integers(-126, 126, (64, 300)) + 0.5
    x = (n * s.astype(np.float64)).astype(np.float32)
    x[0, 0] = np.float32(float.fromhex("0x1.a30fecp-127"))
    x = np.concatenate([x, np.nextafter(x, np.float32(1)), np.nextafter(x, np.float32(-1)), top], 1)
    codes, scales = ref.quantize(x)
    rows = torch.from_numpy(x).cuda()
    q = sg.int8_quantize(rows)
    same(q.codes, torch.from_numpy(codes))
    same(q.scales, torch.from_numpy(scales))
    (b, _), sb = integers(40, x.shape[1], 1), np.full(40, 2.0 ** 100, np.float32)
    for part in (slice(0, 1), slice(0, 5), slice(0, 64)):        # quantised by each of the kernels that do
        same(sg.int8_linear(rows[part], matrix(b, sb)), ref.product(codes[part], scales[part], b, sb, F32))
