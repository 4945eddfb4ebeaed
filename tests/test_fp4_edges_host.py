"""Host-side checks of the 4-bit operators' C ABI: outputs that overlap what a call reads or writes beside them."""
import ctypes

import pytest

from dense_fp32_gemm_03_gb300 import _build, binding, fp4

P_X, P_Q, P_S, P_Y, P_R, P_I, P_P = (i << 28 for i in range(1, 8))   # never dereferenced
BAD = binding.ERR_INVALID_VALUE


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fp4.load()


def matrix(rows=8, cols=64, fmt=1, codes=P_Q, ld=32, scales=P_S, factor=0):
    return fp4._Matrix(fmt, rows, cols, codes, ld, scales, factor)


@pytest.mark.parametrize("factor", [P_Y, P_Y + 8 * 64 * 4 - 4])
def test_outputs_over_a_factor_are_rejected(lib, factor):
    q = matrix(factor=factor)
    rq = ctypes.addressof(q)
    assert lib.fp4_dequantize(rq, 0, P_Y, 64, 0) == BAD
    wide = matrix(rows=64, codes=P_Q + 8192, scales=P_S + 131072)
    rw = ctypes.addressof(wide)
    assert lib.fp4_gemm(rq, rw, 0, P_Y, 64, 0) == BAD
    assert lib.fp4_gemm(rw, rq, 0, P_Y, 64, 0) == BAD
    assert lib.fp4_linear(0, P_X, 64, 8, factor, rw, P_Y, 64, 0) == BAD
    tall = matrix(rows=64, codes=P_Q + 8192, scales=P_S + 131072, factor=factor)
    assert lib.fp4_linear(0, P_X, 64, 8, 0, ctypes.addressof(tall), P_Y, 64, 0) == BAD


@pytest.mark.parametrize("factor", [P_Q + 16, P_S + 2044])
def test_a_factor_inside_its_own_matrix_is_rejected(lib, factor):
    q = matrix(factor=factor)
    assert lib.fp4_quantize(0, P_X, 64, ctypes.addressof(q), 0) == BAD


@pytest.mark.parametrize("ids,p", [(P_Y + 64, 0), (0, P_Y + 4 * 64 * 4 - 4), (P_X, 0), (0, P_X + 1020), (P_R, 0), (0, P_R + 64),
                                   (P_Q, 0), (0, P_S), (P_I, P_I + 28)])
def test_routing_outputs_that_overlap_are_rejected(lib, ids, p):
    """4 tokens of 64 values, two experts each: 32 bytes of ids and of weights."""
    w = fp4._Experts(0, 8, 64, 32, P_Q, P_S, 0, 0)
    assert lib.fp4_moe(0, P_X, 64, 4, P_R, 64, ctypes.addressof(w), 2, 1, P_Y, 64, ids, p, 0) == BAD


@pytest.mark.parametrize("factor", [P_Y, P_Y + 1020])
def test_a_layer_over_its_factors_is_rejected(lib, factor):
    for factors in ((factor, 0), (0, factor)):
        w = fp4._Experts(1, 8, 64, 32, P_Q, P_S, *factors)
        assert lib.fp4_moe(0, P_X, 64, 4, P_R, 64, ctypes.addressof(w), 2, 1, P_Y, 64, 0, 0, 0) == BAD


def test_package_is_imported_without_torch():
    """As before the 4-bit operators: addresses and the build need no torch, and no time for it."""
    import os
    import subprocess
    import sys
    code = ("import sys; sys.modules['torch'] = None\n"
            "import dense_fp32_gemm_03_gb300 as p\n"
            "assert callable(p.sgemm_raw) and 'fp4_moe' in dir(p) and 'fp4_moe' in p.__all__\n"
            "del sys.modules['torch']\n"
            "assert callable(p.fp4_moe) and p.Fp4Matrix.__module__ == p.__name__ + '.fp4'\n"
            "try:\n    p.fp5\nexcept AttributeError:\n    print('fine')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.stdout.strip() == "fine", r.stderr
