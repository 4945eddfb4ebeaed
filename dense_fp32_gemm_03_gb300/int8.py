"""8-bit integer operators on CUDA tensors (ctypes binding of ``include/int8.h``).

* For serving: rows as integers with a scale each (:func:`int8_quantize`,
  :func:`int8_matrix`), their products (:func:`int8_gemm`), and linear layers on
  such weights, which quantise their input token by token (:func:`int8_linear`).
* For training: activations kept in 8 bits from the forward pass
  (:func:`int8_checkpoint`) and a linear layer's weight gradient taken from them
  (:func:`int8_weight_grad`); the gated activation of a feed-forward block that
  keeps its two inputs so (:func:`int8_swiglu`, :func:`int8_swiglu_backward`).

As in ``binding``, this module marshals arguments only: all arithmetic runs in
the library's CUDA kernels, and there is no CPU fallback.  None of the calls
takes part in autograd: forward and backward are calls of their own.

Every call takes a ``stream`` (default: the current one).  It does not wait for
the stream on which its inputs were made; a ``stream`` that was passed is
recorded on them, so they may be dropped once the call returned.  Scratch
belongs to the stream: the first call that needs more of it is made outside
graph capture, and two graphs captured on one stream do not run at one time.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import binding
from .fp4 import _DTYPES, _call, _dense, _empty, _output, _read_on

ORDERS = ("channels", "tokens")

# Every entry point include/int8.h declares.
EXPORTS = ("int8_quantize", "int8_dequantize", "int8_gemm", "int8_linear", "int8_checkpoint_layout", "int8_checkpoint",
           "int8_restore", "int8_weight_grad", "int8_swiglu", "int8_swiglu_backward")


class _Matrix(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("ld", ctypes.c_int64), ("scales", ctypes.c_void_p)]


class _Checkpoint(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("order", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("codes", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("units", ctypes.c_void_p), ("ld_units", ctypes.c_int64)]


# The same structures as bytes, which the calls take where a structure is made at each of them.
_pack_matrix = struct.Struct("@qqQqQ").pack
_pack_checkpoint = struct.Struct("@iiqqQqQq").pack
_lib = None


def load():
    """The library with int8.h's argument types set (raises if it is absent)."""
    global _lib
    if _lib is None:
        lib = binding.load()
        i, i32, i64, vp = ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
        out = ctypes.POINTER(i64)
        lib.int8_quantize.argtypes = [i, vp, i64, vp, vp]
        lib.int8_dequantize.argtypes = [vp, i, vp, i64, vp]
        lib.int8_gemm.argtypes = [vp, vp, i, vp, i64, vp]
        lib.int8_linear.argtypes = [i, vp, i64, i64, vp, vp, i64, vp]
        lib.int8_checkpoint_layout.argtypes = [i, i64, i64, out, out, out, out]
        lib.int8_checkpoint.argtypes = [vp, i64, vp, vp]
        lib.int8_restore.argtypes = [vp, i, vp, i64, vp]
        lib.int8_weight_grad.argtypes = [vp, i64, i64, vp, i, i32, vp, i64, vp]
        lib.int8_swiglu.argtypes = [i, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp]
        lib.int8_swiglu_backward.argtypes = [vp, i64, vp, vp, vp, i64, vp, i64, vp]
        for name in EXPORTS:
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


# -------------------------------------------------------------------- arguments
def _same_device(index, *others):
    for t in others:
        other = t.index if type(t) is Int8Matrix or type(t) is Int8Checkpoint else t.get_device()
        if other != index:
            raise ValueError(f"operands are on different devices (cuda:{index} and cuda:{other})")


def _cuda_device(device):
    if type(device) is not torch.device:
        device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"an 8-bit matrix lives on a CUDA device, not on {device}")
    return device if device.index is not None else torch.device("cuda", torch.cuda.current_device())


def _type(dtype, name="dtype"):
    if dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return _DTYPES[dtype]


# ------------------------------------------------------------------------- rows
def _pitch(cols):
    """Bytes of a row that is allocated here: a multiple of 16, long ones of 128 (whole lines of memory)."""
    return (cols + 127) // 128 * 128 if cols > 2048 else (cols + 15) // 16 * 16


class Int8Matrix:
    """Rows of integers with a scale each, on the GPU: ``shape``, ``device``, ``codes`` (int8, rows x cols), ``scales`` (float32).

    Made by :func:`int8_quantize` or, from a checkpoint's arrays, by :func:`int8_matrix`.
    """

    __slots__ = ("shape", "device", "index", "_memory", "_arrays", "_ref", "__weakref__")

    def __init__(self, rows, cols, device="cuda", stream=None):
        device = _cuda_device(device)
        # One allocation: the codes, then the scales.
        pitch = _pitch(cols)
        memory = _empty((rows * (pitch + 4),), torch.uint8, device, stream)
        self.shape, self.device, self.index, self._memory, self._arrays = (rows, cols), device, device.index, (memory,), None
        base = memory.data_ptr()
        self._ref = _pack_matrix(rows, cols, base, pitch, base + rows * pitch)

    @classmethod
    def _of(cls, codes, scales):
        """The matrix that these arrays (as the library takes them) are."""
        self = cls.__new__(cls)
        rows, cols = codes.shape
        # The library has the addresses of these two: they stay.
        self.shape, self.device, self.index, self._memory, self._arrays = (
            (rows, cols), codes.device, codes.get_device(), (codes, scales), (codes, scales))
        ld = codes.stride(0) if rows > 1 else (cols + 15) // 16 * 16
        self._ref = _pack_matrix(rows, cols, codes.data_ptr(), ld, scales.data_ptr())
        return self

    def _views(self):
        if self._arrays is None:
            (rows, cols), memory = self.shape, self._memory[0]
            pitch = _pitch(cols)
            self._arrays = (memory[:rows * pitch].view(torch.int8).view(rows, pitch)[:, :cols],
                            memory[rows * pitch:].view(torch.float32))
        return self._arrays

    codes = property(lambda self: self._views()[0])
    scales = property(lambda self: self._views()[1])

    def dequantize(self, dtype=torch.float32):
        """The values (:func:`int8_dequantize`)."""
        return int8_dequantize(self, dtype)

    def __repr__(self):
        return f"Int8Matrix({self.shape[0]}x{self.shape[1]}, {self.device})"


def _rows(q, name):
    if not isinstance(q, Int8Matrix):
        raise TypeError(f"{name} must be an Int8Matrix")
    return q


def int8_quantize(x, out=None, stream=None):
    """x (2-D float32, bfloat16 or float16 CUDA tensor, any row stride) in 8 bits with a scale a row: an :class:`Int8Matrix`.

    ``out`` (an ``Int8Matrix`` of x's shape that an earlier call returned) is filled if given.
    """
    ld, rows, cols = _dense(x, "x")
    if out is None:
        out = Int8Matrix(rows, cols, x.device, stream)
    else:
        if _rows(out, "out").shape != (rows, cols):
            raise ValueError(f"out is {out}, expected {(rows, cols)}")
        if len(out._memory) > 1:
            raise ValueError("out is a matrix of a checkpoint's arrays, which may lie between others")
        _same_device(x.get_device(), out)
    if stream is not None:
        _read_on(stream, x, *out._memory)
    _call("int8_quantize", out.index, stream, load().int8_quantize, _DTYPES[x.dtype], x.data_ptr(), ld, out._ref)
    return out


def int8_matrix(codes, scales, stream=None):
    """An :class:`Int8Matrix` from a checkpoint's arrays: ``codes`` int8, rows x cols, ``scales`` float32, one a row.

    Arrays whose rows start at multiples of 16 bytes are used where they are
    (they must not change while the matrix is in use); others are copied.
    """
    for t, name, dtype, dims in ((codes, "codes", torch.int8, 2), (scales, "scales", torch.float32, 1)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda or t.dtype != dtype or t.dim() != dims:
            raise ValueError(f"{name} must be a {dims}-D {dtype} CUDA tensor, got {t.dtype} {tuple(t.shape)} on {t.device}")
    rows, cols = codes.shape
    if scales.shape[0] != rows:
        raise ValueError(f"{rows} rows take as many scales, got {scales.shape[0]}")
    _same_device(codes.get_device(), scales)
    pitch = (cols + 15) // 16 * 16
    device = codes.device
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(device):
        if stream is not None:
            _read_on(stream, codes, scales)
        # In place only if what the library may read of the last row, up to 16 bytes, is there too.
        size = codes.untyped_storage().nbytes() - codes.storage_offset()
        if codes.data_ptr() % 16 or (cols > 1 and codes.stride(1) != 1) or (
                rows > 1 and (codes.stride(0) % 16 or codes.stride(0) < pitch)) or (
                rows and size < (rows - 1) * codes.stride(0) + pitch):
            memory = torch.zeros((rows, _pitch(cols)), dtype=torch.int8, device=device)
            memory[:, :cols].copy_(codes)
            codes = memory[:, :cols]
        return Int8Matrix._of(codes, scales.contiguous())


def int8_dequantize(q, dtype=torch.float32, out=None, stream=None):
    """The values of ``q``, computed in 32 bits and rounded once to ``dtype``."""
    _rows(q, "q")
    if out is not None:
        dtype = out.dtype
    number = _type(dtype)
    out, ld = _output(out, q.shape, dtype, q.device, q.index, stream)
    if stream is not None:
        _read_on(stream, *q._memory, out)
    _call("int8_dequantize", q.index, stream, load().int8_dequantize, q._ref, number, out.data_ptr(), ld)
    return out


# --------------------------------------------------------------------- products
def int8_gemm(A, B, out=None, out_dtype=torch.float32, stream=None):
    """C = A @ B.T of two :class:`Int8Matrix` (M x K and N x K): M x N of ``out_dtype``.

    The integer sums are exact; scales are applied in 32 bits, and the result
    is rounded once.  ``out`` receives the result if given (its type counts
    then).
    """
    _rows(A, "A")
    _rows(B, "B")
    if A.shape[1] != B.shape[1]:
        raise ValueError(f"inner dimensions differ: {A.shape} @ {B.shape}.T")
    _same_device(A.index, B)
    if out is not None:
        out_dtype = out.dtype
    number = _type(out_dtype, "out_dtype")
    out, ld = _output(out, (A.shape[0], B.shape[0]), out_dtype, A.device, A.index, stream)
    if stream is not None:
        _read_on(stream, *A._memory, *B._memory, out)
    _call("int8_gemm", A.index, stream, load().int8_gemm, A._ref, B._ref, number, out.data_ptr(), ld)
    return out


def int8_linear(x, W, out=None, stream=None):
    """y = Q(x) @ W.T: x (M x K) quantised row by row within the call, W an :class:`Int8Matrix` (N x K).

    y has x's type.  The result is bit for bit that of :func:`int8_quantize`
    followed by :func:`int8_gemm`.
    """
    _rows(W, "W")
    n, k = W.shape
    ldx, m, _ = _dense(x, "x", k)
    index, dtype = W.index, x.dtype
    _same_device(index, x)
    out, ldy = _output(out, (m, n), dtype, W.device, index, stream)
    if stream is not None:
        _read_on(stream, x, *W._memory, out)
    _call("int8_linear", index, stream, load().int8_linear, _DTYPES[dtype], x.data_ptr(), ldx, m, W._ref, out.data_ptr(),
          ldy)
    return out


# ------------------------------------------------------------------ checkpoints
def _lines(order, rows, cols):
    """int8_checkpoint_layout()'s lines and pitches: of the codes, then of the units, which follow them in one allocation."""
    blocks = (cols + 31) // 32
    if order == "channels":
        return cols, (rows + 15) // 16 * 16, blocks, (rows + 7) // 8 * 8
    return rows, (cols + 15) // 16 * 16, rows, (blocks + 7) // 8 * 8


def _bytes(lines):
    return lines[0] * lines[1] + 2 * lines[2] * lines[3]


class Int8Checkpoint:
    """Activations kept in 8 bits: ``shape`` (tokens, channels), ``dtype`` (of what was kept), ``order``, ``device``.

    ``order`` is ``"channels"`` for :func:`int8_checkpoint`, whose integers are
    read by :func:`int8_weight_grad`, and ``"tokens"`` for
    :func:`int8_swiglu`'s.  ``codes`` and ``units`` are the arrays that
    ``include/int8.h`` describes, ``nbytes`` their size.
    """

    __slots__ = ("shape", "dtype", "order", "device", "index", "_memory", "_start", "_ref", "__weakref__")

    def __init__(self, rows, cols, dtype, order, device="cuda", stream=None):
        if order not in ORDERS:
            raise ValueError(f"order must be one of {ORDERS}, got {order!r}")
        number, device, lines = _type(dtype), _cuda_device(device), _lines(order, rows, cols)
        self._set(rows, cols, dtype, number, order, device, lines, _empty((_bytes(lines),), torch.uint8, device, stream), 0)

    def _set(self, rows, cols, dtype, number, order, device, lines, memory, start):
        self.shape, self.dtype, self.order, self.device, self.index = (rows, cols), dtype, order, device, device.index
        self._memory, self._start = memory, start
        base = memory.data_ptr() + start
        self._ref = _pack_checkpoint(number, 0 if order == "channels" else 1, rows, cols, base, lines[1],
                                     base + lines[0] * lines[1], lines[3])
        return self

    @property
    def codes(self):
        """The integers, int8 (lines x pitch)."""
        lines, ld, _, _ = _lines(self.order, *self.shape)
        return self._memory[self._start:self._start + lines * ld].view(torch.int8).view(lines, ld)

    @property
    def units(self):
        """The blocks' units (lines x pitch), bfloat16 or float16."""
        lines, ld, unit_lines, ldu = _lines(self.order, *self.shape)
        kind, start = torch.float16 if self.dtype == torch.float16 else torch.bfloat16, self._start + lines * ld
        return self._memory[start:start + 2 * unit_lines * ldu].view(kind).view(unit_lines, ldu)

    nbytes = property(lambda self: _bytes(_lines(self.order, *self.shape)))

    def restore(self, dtype=None):
        """The values (:func:`int8_restore`)."""
        return int8_restore(self, dtype)

    def __repr__(self):
        return f"Int8Checkpoint({self.shape[0]}x{self.shape[1]}, {self.dtype}, {self.order}, {self.device})"


def _kept(c, name, order=None):
    if not isinstance(c, Int8Checkpoint):
        raise TypeError(f"{name} must be an Int8Checkpoint")
    if order is not None and c.order != order:
        raise ValueError(f"{name} is in the order of {c.order}, expected {order}")
    return c


def int8_checkpoint(x, out=None, stream=None):
    """Keeps x (tokens x channels, any row stride) in 8 bits for :func:`int8_weight_grad`: an :class:`Int8Checkpoint`.

    Blocks of 32 channels of a token share a power of two; the error is at most
    2^-7 of a block's largest value (in float32 and bfloat16 of one above
    2^-120; what is below 2^-127 becomes 0).  ``out`` (of x's shape and type, order
    ``"channels"``) is filled if given.
    """
    ld, rows, cols = _dense(x, "x")
    if out is None:
        lines, device = _lines("channels", rows, cols), x.device
        out = Int8Checkpoint.__new__(Int8Checkpoint)._set(rows, cols, x.dtype, _DTYPES[x.dtype], "channels", device, lines,
                                                          _empty((_bytes(lines),), torch.uint8, device, stream), 0)
    else:
        if _kept(out, "out", "channels").shape != (rows, cols) or out.dtype != x.dtype:
            raise ValueError(f"out is {out}, expected {(rows, cols)} {x.dtype}")
        _same_device(x.get_device(), out)
    if stream is not None:
        _read_on(stream, x, out._memory)
    _call("int8_checkpoint", out.index, stream, load().int8_checkpoint, x.data_ptr(), ld, out._ref)
    return out


def int8_restore(c, dtype=None, out=None, stream=None):
    """The values of a checkpoint, tokens x channels, of ``dtype`` (default: the type of what was kept, which holds them exactly)."""
    _kept(c, "c")
    dtype = out.dtype if out is not None else c.dtype if dtype is None else dtype
    number = _type(dtype)
    out, ld = _output(out, c.shape, dtype, c.device, c.index, stream)
    if stream is not None:
        _read_on(stream, c._memory, out)
    _call("int8_restore", c.index, stream, load().int8_restore, c._ref, number, out.data_ptr(), ld)
    return out


def int8_weight_grad(dy, c, out=None, accumulate=False, out_dtype=None, stream=None):
    """dW = dy.T @ X of a linear layer whose input X was kept in ``c`` (order ``"channels"``): N x channels.

    dy is tokens x N of the type that was kept.  ``out_dtype`` is that type
    (the default) or float32.  ``out`` receives the result if given (its type
    counts then); with ``accumulate`` the gradient is added to what it holds.
    """
    _kept(c, "c", "channels")
    lddy, rows, n = _dense(dy, "dy")
    if rows != c.shape[0] or dy.dtype != c.dtype:
        raise ValueError(f"dy must have {c.shape[0]} rows of {c.dtype}, got {rows} of {dy.dtype}")
    _same_device(c.index, dy)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    dtype = out.dtype if out is not None else c.dtype if out_dtype is None else out_dtype
    if dtype not in (c.dtype, torch.float32):
        raise ValueError(f"the gradient's type must be {c.dtype} or float32, got {dtype}")
    out, ldw = _output(out, (n, c.shape[1]), dtype, c.device, c.index, stream)
    if stream is not None:
        _read_on(stream, dy, c._memory, out)
    _call("int8_weight_grad", c.index, stream, load().int8_weight_grad, dy.data_ptr(), lddy, n, c._ref, _DTYPES[dtype],
          1 if accumulate else 0, out.data_ptr(), ldw)
    return out


# ------------------------------------------------------------- gated activation
def int8_swiglu(gate, up, out=None, stream=None):
    """(h, kept): h = gate * sigmoid(gate) * up, and gate and up in 8 bits for :func:`int8_swiglu_backward`.

    gate and up have one shape and type, each any row stride (halves of one
    projection's output, for instance).  ``kept`` is a pair of
    :class:`Int8Checkpoint`.
    """
    ldg, rows, cols = _dense(gate, "gate")
    ldu, other, _ = _dense(up, "up", cols)
    if other != rows or up.dtype != gate.dtype:
        raise ValueError(f"gate and up differ: {tuple(gate.shape)} {gate.dtype} and {tuple(up.shape)} {up.dtype}")
    index, dtype, device = gate.get_device(), gate.dtype, gate.device
    _same_device(index, up)
    number, lines = _DTYPES[dtype], _lines("tokens", rows, cols)
    size = _bytes(lines)                       # (a multiple of 16)
    memory = _empty((2 * size,), torch.uint8, device, stream)
    kept = tuple([Int8Checkpoint.__new__(Int8Checkpoint)._set(rows, cols, dtype, number, "tokens", device, lines, memory, start)
                  for start in (0, size)])
    out, ldh = _output(out, (rows, cols), dtype, device, index, stream)
    if stream is not None:
        _read_on(stream, gate, up, out)
    _call("int8_swiglu", index, stream, load().int8_swiglu, number, rows, cols, gate.data_ptr(), ldg,
          up.data_ptr(), ldu, out.data_ptr(), ldh, kept[0]._ref, kept[1]._ref)
    return out, kept


def int8_swiglu_backward(dh, kept, out=None, stream=None):
    """(dgate, dup) from h's gradient and the pair that :func:`int8_swiglu` kept.

    ``out``, a pair of matrices (the halves of one projection's gradient, for
    instance), receives them if given.
    """
    if not isinstance(kept, (tuple, list)) or len(kept) != 2:
        raise TypeError("kept must be the pair that int8_swiglu returned")
    g, u = _kept(kept[0], "kept", "tokens"), _kept(kept[1], "kept", "tokens")
    if u.shape != g.shape or u.dtype != g.dtype:
        raise ValueError(f"kept values differ: {g} and {u}")
    lddh, rows, _ = _dense(dh, "dh", g.shape[1])
    if rows != g.shape[0] or dh.dtype != g.dtype:
        raise ValueError(f"dh must be {g.shape} {g.dtype}, got {tuple(dh.shape)} {dh.dtype}")
    _same_device(g.index, u, dh)
    if out is None:
        dgate, dup = _empty(g.shape, g.dtype, g.device, stream), _empty(g.shape, g.dtype, g.device, stream)
        ldg = ldu = g.shape[1] or 1
    elif not isinstance(out, (tuple, list)) or len(out) != 2:
        raise TypeError("out must be a pair of tensors")
    else:
        (dgate, ldg), (dup, ldu) = (_output(t, g.shape, g.dtype, g.device, g.index, stream) for t in out)
    if stream is not None:
        _read_on(stream, dh, g._memory, u._memory, dgate, dup)
    _call("int8_swiglu_backward", g.index, stream, load().int8_swiglu_backward, dh.data_ptr(), lddh, g._ref, u._ref,
          dgate.data_ptr(), ldg, dup.data_ptr(), ldu)
    return dgate, dup
