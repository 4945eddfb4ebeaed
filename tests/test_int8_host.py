"""Host-side checks of the 8-bit integer operators' C ABI and of their plain implementation (no GPU needed)."""
import ctypes
import os
import re

import numpy as np
import pytest

from dense_fp32_gemm_03_gb300 import _build, binding, int8

import int8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P_X, P_Q, P_S, P_Y, P_Z = (i << 28 for i in range(1, 6))   # never dereferenced
BAD, UNSUPPORTED = binding.ERR_INVALID_VALUE, binding.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return int8.load()


def test_exports_are_the_headers(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "int8.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(int8_\w+)\s*\(", text))
    assert names == set(int8.EXPORTS)
    for name in names:
        assert hasattr(lib, name)


def test_the_package_offers_them_lazily():
    import dense_fp32_gemm_03_gb300 as sg
    assert {"int8_linear", "Int8Checkpoint"} <= set(dir(sg)) and sg.int8_linear is int8.int8_linear
    assert {n for n in int8.EXPORTS if n != "int8_checkpoint_layout"} <= set(sg.__all__)


def matrix(rows=8, cols=64, codes=P_Q, ld=64, scales=P_S):
    return int8._Matrix(rows, cols, codes, ld, scales)


def kept(dtype=0, order=0, rows=40, cols=64, codes=P_Q, ld=None, units=P_S, ldu=None):
    entries = rows if order == 0 else cols
    unit_entries = rows if order == 0 else (cols + 31) // 32
    return int8._Checkpoint(dtype, order, rows, cols, codes, (entries + 15) // 16 * 16 if ld is None else ld, units,
                            (unit_entries + 7) // 8 * 8 if ldu is None else ldu)


def at(s):
    return ctypes.addressof(s)


def test_structures_as_bytes():
    m = matrix(3, 70, P_Q, 80, P_S)
    assert int8._pack_matrix(3, 70, P_Q, 80, P_S) == bytes(m)
    c = kept(2, 1, 9, 100)
    assert int8._pack_checkpoint(2, 1, 9, 100, P_Q, c.ld, P_S, c.ld_units) == bytes(c)


@pytest.mark.parametrize("q,dtype,x,ldx,want", [
    (matrix(), 3, P_X, 64, BAD), (matrix(), -1, P_X, 64, BAD), (matrix(), 0, 0, 64, BAD), (matrix(), 0, P_X, 63, BAD),
    (matrix(), 0, P_X + 2, 64, BAD), (matrix(rows=-1), 0, P_X, 64, BAD), (matrix(codes=0), 0, P_X, 64, BAD),
    (matrix(codes=P_Q + 8), 0, P_X, 64, BAD), (matrix(ld=48), 0, P_X, 64, BAD), (matrix(ld=72), 0, P_X, 64, BAD),
    (matrix(scales=0), 0, P_X, 64, BAD), (matrix(scales=P_S + 2), 0, P_X, 64, BAD), (matrix(cols=60, ld=60), 0, P_X, 64, BAD),
    (matrix(rows=1 << 31), 0, P_X, 64, UNSUPPORTED), (matrix(), 0, P_Q - 16, 64, BAD), (matrix(), 0, P_S + 16, 64, BAD)])
def test_bad_matrices_are_rejected(lib, q, dtype, x, ldx, want):
    assert lib.int8_quantize(dtype, x, ldx, at(q), 0) == want
    assert lib.int8_dequantize(at(q), dtype, x, ldx, 0) == want


def test_quantise_refuses_codes_over_scales(lib):
    assert lib.int8_quantize(0, P_X, 64, at(matrix(scales=P_Q + 64)), 0) == BAD


def test_missing_structures_are_rejected(lib):
    q, c, k = matrix(), kept(), kept(order=1)
    assert lib.int8_quantize(0, P_X, 64, 0, 0) == BAD
    assert lib.int8_gemm(at(q), 0, 0, P_Y, 8, 0) == BAD
    assert lib.int8_linear(0, P_X, 64, 4, 0, P_Y, 8, 0) == BAD
    assert lib.int8_checkpoint(P_X, 64, 0, 0) == BAD
    assert lib.int8_restore(0, 0, P_Y, 64, 0) == BAD
    assert lib.int8_weight_grad(P_X, 64, 64, 0, 0, 0, P_Y, 64, 0) == BAD
    assert lib.int8_swiglu(0, 40, 64, P_X, 64, P_Y, 64, P_Z, 64, at(k), 0, 0) == BAD
    assert lib.int8_swiglu_backward(P_X, 64, 0, at(k), P_Y, 64, P_Z, 64, 0) == BAD
    assert lib.int8_restore(at(c), 5, P_Y, 64, 0) == BAD


def test_products_are_checked(lib):
    a, b = matrix(), matrix(rows=16, codes=P_Q + 4096, scales=P_S + 65536)
    assert lib.int8_gemm(at(a), at(b), 0, P_Y, 15, 0) == BAD                      # ldc < N
    assert lib.int8_gemm(at(a), at(b), 0, P_Q + 4096, 16, 0) == BAD               # C overlaps B
    assert lib.int8_gemm(at(a), at(b), 0, P_S + 65536, 16, 0) == BAD              # C overlaps B's scales
    assert lib.int8_gemm(at(a), at(b), 4, P_Y, 16, 0) == BAD                      # unknown type
    assert lib.int8_gemm(at(a), at(matrix(cols=32)), 0, P_Y, 16, 0) == BAD
    wide = matrix(cols=131072, ld=131072)
    assert lib.int8_gemm(at(wide), at(wide), 0, P_Y, 16, 0) == UNSUPPORTED
    assert lib.int8_linear(0, P_X, 131072, 4, at(wide), P_Y, 16, 0) == UNSUPPORTED
    assert lib.int8_linear(0, P_X, 63, 4, at(b), P_Y, 16, 0) == BAD               # ldx < K
    assert lib.int8_linear(1, P_X + 1, 64, 4, at(b), P_Y, 16, 0) == BAD           # misaligned
    assert lib.int8_linear(0, P_X, 64, 4, at(b), P_X + 64, 16, 0) == BAD          # y overlaps x
    assert lib.int8_linear(0, P_X, 64, -1, at(b), P_Y, 16, 0) == BAD


@pytest.mark.parametrize("order,rows,cols,want", [
    (0, 1, 1, (16, 8, 16, 16)), (1, 1, 1, (16, 8, 16, 16)), (0, 130, 65, (144, 136, 65 * 144, 3 * 136 * 2)),
    (1, 130, 300, (304, 16, 130 * 304, 130 * 16 * 2)), (0, 0, 64, (0, 0, 0, 0)), (1, 5, 0, (0, 0, 0, 0))])
def test_checkpoint_layout(lib, order, rows, cols, want):
    out = [ctypes.c_int64() for _ in range(4)]
    assert lib.int8_checkpoint_layout(order, rows, cols, *map(ctypes.byref, out)) == binding.OK
    assert tuple(v.value for v in out) == want
    assert lib.int8_checkpoint_layout(2, rows, cols, *map(ctypes.byref, out)) == BAD
    assert lib.int8_checkpoint_layout(order, -1, cols, *map(ctypes.byref, out)) == BAD


@pytest.mark.parametrize("change", [
    dict(dtype=3), dict(order=2), dict(order=1), dict(rows=-1), dict(codes=0), dict(codes=P_Q + 8), dict(ld=32), dict(ld=56),
    dict(units=0), dict(units=P_S + 2), dict(ldu=32), dict(ldu=44), dict(codes=P_X + 64), dict(units=P_X), dict(units=P_Q + 16)])
def test_bad_checkpoints_are_rejected(lib, change):
    assert lib.int8_checkpoint(P_X, 64, at(kept(**change)), 0) == BAD


def test_gradients_are_checked(lib):
    c = kept(dtype=1)

    def call(dy=P_X, lddy=48, n=48, c=c, dtype=1, dw=P_Y, ldw=64):
        return lib.int8_weight_grad(dy, lddy, n, at(c), dtype, 0, dw, ldw, 0)
    for bad in (dict(dy=0), dict(dy=P_X + 1), dict(lddy=47), dict(n=-1), dict(dtype=2), dict(dtype=7), dict(dw=0), dict(ldw=63),
                dict(dw=P_X + 2), dict(dw=P_Q + 64), dict(dw=P_S), dict(dw=P_Y + 2, dtype=0), dict(c=kept(dtype=1, order=1))):
        assert call(**bad) == BAD, bad


def test_too_many_tokens_are_refused(lib):
    c = int8._Checkpoint(1, 0, (1 << 27) + 1, 32, 1 << 28, 1 << 30, 1 << 27, 1 << 30)
    assert lib.int8_weight_grad(1 << 40, 8, 8, at(c), 1, 0, 1 << 41, 32, 0) == UNSUPPORTED
    c = int8._Checkpoint(1, 0, 32, 32, 1 << 28, 32, 1 << 27, 32)
    assert lib.int8_weight_grad(1 << 40, 1 << 30, (1 << 29) + 1, at(c), 1, 0, 1 << 45, 32, 0) == UNSUPPORTED


def test_swiglu_is_checked(lib):
    g, u = kept(order=1), kept(order=1, codes=P_Q + (1 << 20), units=P_S + (1 << 20))

    def call(dtype=0, m=40, f=64, gate=P_X, ldg=128, up=P_X + 256, ldu=128, h=P_Y, ldh=64, g=g, u=u):
        return lib.int8_swiglu(dtype, m, f, gate, ldg, up, ldu, h, ldh, at(g), at(u), 0)
    for bad in (dict(dtype=1), dict(m=39), dict(f=63), dict(gate=0), dict(ldg=63), dict(up=P_X + 2), dict(h=P_X), dict(h=P_X + 256, ldh=128),
                dict(h=P_Q), dict(h=P_S), dict(g=u), dict(g=kept()), dict(u=g), dict(gate=P_Q - 64), dict(ldh=60)):
        assert call(**bad) == BAD, bad

    def back(dh=P_X, ldd=64, g=g, u=u, dgate=P_Y, ldg=128, dup=P_Y + 256, ldu=128):
        return lib.int8_swiglu_backward(dh, ldd, at(g), at(u), dgate, ldg, dup, ldu, 0)
    for bad in (dict(dh=0), dict(ldd=63), dict(dup=P_Y), dict(dup=P_Y + 252), dict(dup=P_Y + 260), dict(dup=P_Y + 255), dict(dgate=P_X),
                dict(dgate=P_Q), dict(dup=P_S), dict(u=kept(order=1, rows=41, ldu=48)), dict(u=kept(dtype=1, order=1)), dict(g=kept()),
                dict(dup=P_Y + 256, ldu=64)):
        assert back(**bad) == BAD, bad


# -------------------------------------------------------- the plain implementation
def test_plain_rows():
    q, s = ref.quantize(np.array([[127.0, 0.5, 1.5, -2.5, 2.6], [0, 0, 0, 0, 0], [np.nan, 1, 1, 1, 1]]))
    assert q.tolist() == [[127, 0, 2, -2, 3], [0] * 5, [0] * 5]
    assert s[0] == 1 and s[1] == np.float32(2.0 ** -126) and np.isnan(s[2])


def test_plain_blocks():
    x = np.zeros((1, 40))
    x[0, :5], x[0, 35] = [1.0, 0.5 / 64, 1.5 / 64, 1.999, 1.0 / 128], 2.0 ** -130
    q, u = ref.keep(x, False)
    assert u.tolist() == [[2.0 ** -6, 2.0 ** -126]]
    assert q[0, 0, :5].tolist() == [64, 0, 2, 127, 0] and (q[0, 1] == 0).all()
    assert ref.keep(np.full((1, 1), 2.0 ** -24), True)[1].item() == 2.0 ** -24


def test_a_kept_value_is_near():
    x = np.random.default_rng(0).normal(size=(20, 320))
    top = np.abs(x.reshape(20, 10, 32)).max(-1).repeat(32, -1).reshape(20, 320)
    assert (np.abs(ref.kept(x, False) - x) <= top * 2.0 ** -7).all()


def test_swiglu_gradients_are_difference_quotients():
    g, u = np.random.default_rng(1).normal(size=(2, 1000)) * 3
    dg, du = ref.swiglu_backward(1.0, g, u)
    h = 1e-6
    assert np.allclose(dg, (ref.swiglu(g + h, u) - ref.swiglu(g - h, u)) / (2 * h), rtol=1e-6, atol=1e-8)
    assert np.allclose(du, ref.swiglu(g, u + 1) - ref.swiglu(g, u), rtol=1e-9, atol=1e-12)
