"""Host-side checks of the 4-bit operators' C ABI and of their plain implementation (no GPU needed)."""
import ctypes
import os
import re

import numpy as np
import pytest

from dense_fp32_gemm_03_gb300 import _build, binding, fp4

import fp4_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P_X, P_Q, P_S, P_Y = 0x10000000, 0x20000000, 0x30000000, 0x40000000   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fp4.load()


def test_exports_are_the_headers(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(fp4_\w+)\s*\(", text))
    assert names == set(fp4.EXPORTS)
    for name in names:
        assert hasattr(lib, name)


@pytest.mark.parametrize("fmt,rows,cols,want", [
    (0, 1, 1, (16, 16, 1024)), (1, 1, 1, (16, 16, 2048)), (0, 129, 257, (144, 129 * 144, 2 * 2 * 1024)),
    (1, 128, 256, (128, 128 * 128, 2048)), (0, 0, 64, (32, 0, 0))])
def test_layout(lib, fmt, rows, cols, want):
    out = [ctypes.c_int64() for _ in range(3)]
    assert lib.fp4_layout(fmt, rows, cols, *map(ctypes.byref, out)) == binding.OK
    assert tuple(v.value for v in out) == want


def matrix(rows=8, cols=64, fmt=0, codes=P_Q, ld=32, scales=P_S, factor=0):
    return fp4._Matrix(fmt, rows, cols, codes, ld, scales, factor)


BAD = binding.ERR_INVALID_VALUE


@pytest.mark.parametrize("q,dtype,x,ldx,want", [
    (matrix(), 3, P_X, 64, BAD), (matrix(), -1, P_X, 64, BAD), (matrix(), 0, 0, 64, BAD), (matrix(), 0, P_X, 63, BAD),
    (matrix(), 0, P_X + 2, 64, BAD), (matrix(fmt=2), 0, P_X, 64, BAD), (matrix(rows=-1), 0, P_X, 64, BAD),
    (matrix(codes=0), 0, P_X, 64, BAD), (matrix(codes=P_Q + 8), 0, P_X, 64, BAD), (matrix(ld=16), 0, P_X, 64, BAD),
    (matrix(ld=40), 0, P_X, 64, BAD), (matrix(scales=P_S + 4), 0, P_X, 64, BAD), (matrix(factor=P_X + 1), 0, P_X, 64, BAD),
    (matrix(rows=1 << 31), 0, P_X, 64, binding.ERR_UNSUPPORTED), (matrix(), 0, P_Q - 16, 64, BAD),
    (matrix(), 0, P_S + 16, 64, BAD)])
def test_bad_matrices_are_rejected(lib, q, dtype, x, ldx, want):
    assert lib.fp4_quantize(dtype, x, ldx, ctypes.addressof(q), 0) == want
    assert lib.fp4_dequantize(ctypes.addressof(q), dtype, x, ldx, 0) == want


def test_missing_structures_are_rejected(lib):
    q = matrix()
    assert lib.fp4_quantize(0, P_X, 64, 0, 0) == BAD
    assert lib.fp4_gemm(ctypes.addressof(q), 0, 0, P_Y, 8, 0) == BAD
    assert lib.fp4_linear(0, P_X, 64, 4, 0, 0, P_Y, 8, 0) == BAD
    assert lib.fp4_moe(0, P_X, 64, 4, P_Q, 64, 0, 2, 1, P_Y, 64, 0, 0, 0) == BAD


def test_products_are_checked(lib):
    a, b = matrix(), matrix(rows=16, codes=P_Q + 4096, scales=P_S + 65536)
    ra, rb = ctypes.addressof(a), ctypes.addressof(b)
    assert lib.fp4_gemm(ra, rb, 0, P_Y, 15, 0) == BAD                      # ldc < N
    assert lib.fp4_gemm(ra, rb, 0, P_Q + 4096, 16, 0) == BAD               # C overlaps B
    assert lib.fp4_gemm(ra, rb, 4, P_Y, 16, 0) == BAD                      # unknown type
    for other in (matrix(cols=32), matrix(fmt=1)):
        assert lib.fp4_gemm(ra, ctypes.addressof(other), 0, P_Y, 16, 0) == BAD
    assert lib.fp4_linear(0, P_X, 63, 4, 0, rb, P_Y, 16, 0) == BAD          # ldx < K
    assert lib.fp4_linear(0, P_X, 64, 4, P_X + 2, rb, P_Y, 16, 0) == BAD    # misaligned factor
    assert lib.fp4_linear(0, P_X, 64, 4, 0, rb, P_X + 64, 16, 0) == BAD     # y overlaps x


@pytest.mark.parametrize("change", [dict(top=0), dict(top=9), dict(top=33), dict(ldx=63), dict(ldr=10), dict(ldy=3),
                                    dict(y=P_X + 4), dict(w=dict(gate_up=0)), dict(w=dict(down=P_Q + 8)),
                                    dict(w=dict(format=7)), dict(w=dict(f=0)), dict(ids=3), dict(p=2)])
def test_layer_arguments_are_checked(lib, change):
    w = dict(format=0, experts=8, d=64, f=32, gate_up=P_Q, down=P_S, gate_up_factor=0, down_factor=0)
    w.update(change.pop("w", {}))
    c = dict(x=P_X, ldx=64, top=2, ldr=64, y=P_Y, ldy=64, ids=0, p=0)
    c.update(change)
    s = fp4._Experts(*w.values())
    assert lib.fp4_moe(0, c["x"], c["ldx"], 4, P_X + (1 << 20), c["ldr"], ctypes.addressof(s), c["top"], 1, c["y"],
                       c["ldy"], c["ids"], c["p"], 0) == BAD


def test_more_experts_than_the_layer_takes(lib):
    assert lib.fp4_experts_layout(0, 1025, 64, 64, None, None) == binding.ERR_UNSUPPORTED
    up, down = ctypes.c_int64(), ctypes.c_int64()
    assert lib.fp4_experts_layout(1, 3, 130, 20, ctypes.byref(up), ctypes.byref(down)) == binding.OK
    assert (up.value, down.value) == (3 * 1 * 1 * 18432 + 16, 3 * 2 * 1 * 18432)


def test_host_tensors_are_refused():
    import torch
    with pytest.raises(ValueError, match="CUDA tensor"):
        fp4.fp4_quantize(torch.zeros(4, 32), "mxfp4")


# --------------------------------------------- the plain implementation itself
def test_levels_round_to_nearest_even():
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.26, 4.99, 6.0])
    assert ref.LEVELS[ref.nearest_even(v, ref.LEVELS)].tolist() == [0, 1, 1, 2, 2, 4, 4, 0.5, 4, 6]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_representable_values_survive(fmt):
    """Quantising what the format holds exactly changes nothing (each block has a 6, so the scale is known)."""
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 16, (5, 64))
    codes[:, :: ref.BLOCK[fmt]] = 7
    low = 120 if fmt == "mxfp4" else 40
    scales = rng.integers(low, low + 10, (5, 64 // ref.BLOCK[fmt]))
    v = ref.values(codes, scales, fmt)
    c, s = ref.quantize(v.astype(np.float32), fmt)
    assert np.array_equal(s, scales) and np.array_equal(ref.values(c, s, fmt), v)


def test_scale_bytes_match_torch():
    import torch
    b = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(b, ref.E4M3[:127])
