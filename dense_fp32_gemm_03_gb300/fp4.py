"""Microscaled 4-bit operators on CUDA tensors (ctypes binding of ``include/fp4.h``).

Quantisation to two formats, products of quantised matrices, a linear layer on
unquantised activations and a mixture-of-experts layer for a few tokens.  As in
``binding``, this module marshals arguments only: all arithmetic runs in the
library's CUDA kernels, and there is no CPU fallback.

Formats (``include/fp4.h`` has the full definition):

* ``"mxfp4"``: blocks of 32 values with a power-of-two scale byte;
* ``"nvfp4"``: blocks of 16 values with an 8-bit float scale byte, times one
  32-bit factor of the whole matrix (a one-element tensor, usually
  ``x.abs().amax() / 2688``; ``None`` means 1).

Every call takes a ``stream`` (default: the current one).  It does not wait for
the stream on which its inputs were made; a ``stream`` that was passed is
recorded on them, so they may be dropped once the call returned.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import OK, SgemmError

FORMATS = {"mxfp4": 0, "nvfp4": 1}
BLOCK = {"mxfp4": 32, "nvfp4": 16}
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

# Every entry point include/fp4.h declares.
EXPORTS = ("fp4_layout", "fp4_quantize", "fp4_pack", "fp4_dequantize", "fp4_gemm", "fp4_linear",
           "fp4_experts_layout", "fp4_experts_pack", "fp4_moe")


class _Matrix(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("ld", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("factor", ctypes.c_void_p)]


class _Experts(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("experts", ctypes.c_int64), ("d", ctypes.c_int64),
                ("f", ctypes.c_int64), ("gate_up", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("gate_up_factor", ctypes.c_void_p), ("down_factor", ctypes.c_void_p)]


_lib = None


def load():
    """The library with fp4.h's argument types set (raises if it is absent)."""
    global _lib
    if _lib is None:
        lib = binding.load()
        i, i64, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
        out = ctypes.POINTER(i64)
        lib.fp4_layout.argtypes = [i, i64, i64, out, out, out]
        lib.fp4_quantize.argtypes = [i, vp, i64, vp, vp]
        lib.fp4_pack.argtypes = [vp, i64, vp, i64, vp, vp]
        lib.fp4_dequantize.argtypes = [vp, i, vp, i64, vp]
        lib.fp4_gemm.argtypes = [vp, vp, i, vp, i64, vp]
        lib.fp4_linear.argtypes = [i, vp, i64, i64, vp, vp, vp, i64, vp]
        lib.fp4_experts_layout.argtypes = [i, i64, i64, i64, out, out]
        lib.fp4_experts_pack.argtypes = [vp, vp, vp, vp]
        lib.fp4_moe.argtypes = [i, vp, i64, i64, vp, i64, vp, ctypes.c_int32, ctypes.c_int32, vp, i64, vp, vp, vp]
        for name in EXPORTS:
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


# -------------------------------------------------------------------- arguments
# The calls are short (a few microseconds on the GPU for a token), so the checks
# ask each tensor for each property once.
def _dense(t, name, cols=None):
    """(row stride, rows, columns) of a 2-D CUDA tensor of an unquantised type."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype not in _DTYPES or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D float32, bfloat16 or float16 CUDA tensor, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    rows, n = t.shape
    stride, unit = t.stride()
    if n > 1 and unit != 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    if cols is not None and n != cols:
        raise ValueError(f"{name} has {n} columns, expected {cols}")
    if rows <= 1:
        return n or 1, rows, n
    if stride < n:
        raise ValueError(f"{name} has overlapping rows (row stride {stride}, {n} columns)")
    return stride or 1, rows, n


def _format(fmt):
    if fmt not in FORMATS:
        raise ValueError(f"format must be one of {tuple(FORMATS)}, got {fmt!r}")
    return FORMATS[fmt]


def _scale(scale, fmt, index, name="scale"):
    """Address of nvfp4's factor, or 0."""
    if scale is None:
        return 0
    if fmt != "nvfp4":
        raise ValueError(f"{name} belongs to nvfp4 only")
    if not isinstance(scale, torch.Tensor) or scale.dtype != torch.float32 or scale.numel() != 1 \
            or scale.get_device() != index:
        raise ValueError(f"{name} must be a one-element float32 tensor on cuda:{index}")
    return scale.data_ptr()


def _same_device(index, *tensors):
    for t in tensors:
        other = t.index if isinstance(t, (Fp4Matrix, Fp4Experts)) else t.get_device()
        if other != index:
            raise ValueError(f"operands are on different devices (cuda:{index} and cuda:{other})")


def _call(what, index, stream, fn, *args):
    handle = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st != OK:
        raise SgemmError(st, what)


def _empty(shape, dtype, device, stream):
    """A new tensor whose memory belongs to the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _read_on(stream, *tensors):
    """A stream that was passed in uses these tensors: their memory is not given out again before it is done with them."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _output(out, shape, dtype, device, index, stream):
    """(out or a new tensor, its row stride)"""
    if out is None:
        return _empty(shape, dtype, device, stream), shape[1] or 1
    ld, rows, cols = _dense(out, "out")
    if (rows, cols) != shape or out.dtype != dtype:
        raise ValueError(f"out must be {shape} {dtype}, got {(rows, cols)} {out.dtype}")
    _same_device(index, out)
    return out, ld


# --------------------------------------------------------------------- matrices
class Fp4Matrix:
    """A quantised matrix on the GPU: ``shape``, ``format``, ``device``, ``codes``, ``scales``, ``scale`` (nvfp4's factor).

    ``codes`` holds two codes a byte, row by row; ``scales`` the scale bytes in
    the tensor core's order (``include/fp4.h``).  Made by :func:`fp4_quantize`
    or, from a checkpoint's arrays, by :func:`fp4_matrix`.
    """

    __slots__ = ("format", "shape", "device", "index", "_scale", "_memory", "_start", "_ld", "_c", "_ref", "__weakref__")

    def __init__(self, rows, cols, fmt, scale=None, device="cuda", stream=None):
        number = _format(fmt)
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"a quantised matrix lives on a CUDA device, not on {device}")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        index = device.index
        # fp4_layout()'s sizes, in one allocation: the codes, then the scales at the next 256 bytes.
        ld = (cols + 31) // 32 * 16
        start = (rows * ld + 255) // 256 * 256
        memory = _empty((start + (rows + 127) // 128 * ((cols + 255) // 256) * (1024 << number),), torch.uint8, device,
                        stream)
        self.format, self.shape, self.device, self.index, self._scale = fmt, (rows, cols), device, index, scale
        self._memory, self._start, self._ld = memory, start, ld
        base = memory.data_ptr()
        self._c = c = _Matrix(number, rows, cols, base, ld, base + start, _scale(scale, fmt, index))
        self._ref = ctypes.addressof(c)

    @property
    def scale(self):
        """nvfp4's factor.  The library has its address: another factor takes another matrix, or a write into this tensor."""
        return self._scale

    @property
    def codes(self):
        """rows x pitch bytes, two codes a byte."""
        return self._memory[:self.shape[0] * self._ld].view(self.shape[0], self._ld)

    @property
    def scales(self):
        """The scale bytes, in the tensor core's order."""
        return self._memory[self._start:]

    def dequantize(self, dtype=torch.float32):
        """The values the codes stand for (:func:`fp4_dequantize`)."""
        return fp4_dequantize(self, dtype)

    def __repr__(self):
        return f"Fp4Matrix({self.shape[0]}x{self.shape[1]}, {self.format}, {self.device})"


def _quantized(q, name):
    if not isinstance(q, Fp4Matrix):
        raise TypeError(f"{name} must be an Fp4Matrix")
    return q


def fp4_quantize(x, format="mxfp4", scale=None, out=None, stream=None):
    """x (2-D float32, bfloat16 or float16 CUDA tensor, any row stride) in 4 bits: an :class:`Fp4Matrix`.

    ``scale`` is nvfp4's factor of the whole matrix.  ``out`` (an
    ``Fp4Matrix`` of x's shape and this format) is filled if given, with its
    own ``scale``.
    """
    ld, rows, cols = _dense(x, "x")
    if out is None:
        out = Fp4Matrix(rows, cols, format, scale, x.device, stream)
    else:
        _quantized(out, "out")
        if out.shape != (rows, cols) or out.format != format:
            raise ValueError(f"out is {out}, expected {(rows, cols)} {format}")
        if scale is not None and scale is not out.scale:
            raise ValueError("out has its own scale: make it with this one")
        _same_device(x.get_device(), out)
    if stream is not None:
        _read_on(stream, x, out._memory, out.scale)
    _call("fp4_quantize", out.index, stream, load().fp4_quantize, _DTYPES[x.dtype], x.data_ptr(), ld, out._ref)
    return out


def fp4_matrix(codes, scales, format="mxfp4", cols=None, scale=None, stream=None):
    """An :class:`Fp4Matrix` from a checkpoint's row-major arrays.

    ``codes``: uint8, rows x ceil(cols / 2), two codes a byte, the even column
    in the low four bits; ``scales``: one byte a block (uint8, or an 8-bit
    float type), rows x ceil(cols / block).  ``cols`` defaults to twice the
    width of ``codes``.
    """
    _format(format)
    for t, name in ((codes, "codes"), (scales, "scales")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda or t.dim() != 2 or t.element_size() != 1:
            raise ValueError(f"{name} must be a 2-D CUDA tensor of bytes")
        if t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must be row-major (unit column stride)")
        if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
            raise ValueError(f"{name} has overlapping rows")
    rows = codes.shape[0]
    cols = 2 * codes.shape[1] if cols is None else int(cols)
    blocks = -(-cols // BLOCK[format])
    if tuple(codes.shape) != (rows, (cols + 1) // 2) or tuple(scales.shape) != (rows, blocks):
        raise ValueError(f"{rows} x {cols} values in {format} take codes {(rows, (cols + 1) // 2)} and scales "
                         f"{(rows, blocks)}, got {tuple(codes.shape)} and {tuple(scales.shape)}")
    _same_device(codes.get_device(), scales)
    q = Fp4Matrix(rows, cols, format, scale, codes.device, stream)
    if stream is not None:
        _read_on(stream, codes, scales)
    _call("fp4_pack", q.index, stream, load().fp4_pack, codes.data_ptr(), max(codes.stride(0), codes.shape[1], 1),
          scales.data_ptr(), max(scales.stride(0), scales.shape[1], 1), q._ref)
    return q


def fp4_dequantize(q, dtype=torch.float32, out=None, stream=None):
    """The values of ``q``, computed in 32 bits and rounded once to ``dtype``."""
    _quantized(q, "q")
    if out is not None:
        dtype = out.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    out, ld = _output(out, q.shape, dtype, q.device, q.index, stream)
    if stream is not None:
        _read_on(stream, q._memory, q.scale, out)
    _call("fp4_dequantize", q.index, stream, load().fp4_dequantize, q._ref, _DTYPES[dtype], out.data_ptr(), ld)
    return out


# --------------------------------------------------------------------- products
def fp4_gemm(A, B, out=None, out_dtype=torch.float32, stream=None):
    """C = A @ B.T of two :class:`Fp4Matrix` (M x K and N x K, one format): M x N of ``out_dtype``.

    Sums are kept in 32 bits and rounded once.  ``out`` receives the result if
    given (its type counts then).
    """
    _quantized(A, "A")
    _quantized(B, "B")
    if A.shape[1] != B.shape[1]:
        raise ValueError(f"inner dimensions differ: {A.shape} @ {B.shape}.T")
    if A.format != B.format:
        raise ValueError(f"formats differ: {A.format} and {B.format}")
    _same_device(A.index, B)
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in _DTYPES:
        raise ValueError(f"out_dtype must be float32, bfloat16 or float16, got {out_dtype}")
    out, ld = _output(out, (A.shape[0], B.shape[0]), out_dtype, A.device, A.index, stream)
    if stream is not None:
        _read_on(stream, A._memory, A.scale, B._memory, B.scale, out)
    _call("fp4_gemm", A.index, stream, load().fp4_gemm, A._ref, B._ref, _DTYPES[out_dtype], out.data_ptr(), ld)
    return out


def fp4_linear(x, W, x_scale=None, out=None, stream=None):
    """y = Q(x) @ W.T: x (M x K) quantised in W's format within the call, W an :class:`Fp4Matrix` (N x K).

    ``x_scale`` is nvfp4's factor for x.  y has x's type.  The result is that
    of :func:`fp4_quantize` followed by :func:`fp4_gemm` (up to M = 16 with the
    32-bit sums in another order).
    """
    _quantized(W, "W")
    n, k = W.shape
    ldx, m, _ = _dense(x, "x", k)
    index, dtype = W.index, x.dtype
    _same_device(index, x)
    factor = _scale(x_scale, W.format, index, "x_scale")
    out, ldy = _output(out, (m, n), dtype, W.device, index, stream)
    if stream is not None:
        _read_on(stream, x, x_scale, W._memory, W.scale, out)
    _call("fp4_linear", index, stream, load().fp4_linear, _DTYPES[dtype], x.data_ptr(), ldx, m, factor, W._ref,
          out.data_ptr(), ldy)
    return out


# ---------------------------------------------------------- mixture of experts
class Fp4Experts:
    """The weights of a mixture-of-experts layer, laid out once for :func:`fp4_moe` (made by :func:`fp4_experts`)."""

    def __init__(self, experts, d, f, fmt, gate_up_scale, down_scale, device, stream=None):
        number = _format(fmt)
        up, down = ctypes.c_int64(), ctypes.c_int64()
        st = load().fp4_experts_layout(number, experts, d, f, ctypes.byref(up), ctypes.byref(down))
        if st != OK:
            raise SgemmError(st, "fp4_experts_layout")
        self.experts, self.d, self.f, self.format, self.device, self.index = experts, d, f, fmt, device, device.index
        # The library has the addresses of these four: they stay.
        self._gate_up = _empty((up.value,), torch.uint8, device, stream)
        self._down = _empty((down.value,), torch.uint8, device, stream)
        self._gate_up_scale, self._down_scale = gate_up_scale, down_scale
        self._c = _Experts(number, experts, d, f, self.gate_up.data_ptr(), self.down.data_ptr(),
                           *(0 if s is None else s.data_ptr() for s in (gate_up_scale, down_scale)))
        self._ref = ctypes.addressof(self._c)

    gate_up = property(lambda self: self._gate_up)
    down = property(lambda self: self._down)
    gate_up_scale = property(lambda self: self._gate_up_scale)
    down_scale = property(lambda self: self._down_scale)

    def __repr__(self):
        return f"Fp4Experts({self.experts} experts, d {self.d}, f {self.f}, {self.format}, {self.device})"


def fp4_experts(gate_up, down, experts, stream=None):
    """Lays out a layer's quantised weights for :func:`fp4_moe`.

    ``gate_up``: :class:`Fp4Matrix` of (experts * 2 f) x d, each expert's f
    gate rows and then its f up rows; ``down``: (experts * d) x f.  The
    matrices may be dropped afterwards.
    """
    _quantized(gate_up, "gate_up")
    _quantized(down, "down")
    experts = int(experts)
    d, f = gate_up.shape[1], down.shape[1]
    if experts < 1 or gate_up.shape[0] != experts * 2 * f or down.shape[0] != experts * d:
        raise ValueError(f"{experts} experts need gate_up (experts * 2 f) x d and down (experts * d) x f, got "
                         f"{gate_up.shape} and {down.shape}")
    if gate_up.format != down.format:
        raise ValueError(f"formats differ: {gate_up.format} and {down.format}")
    _same_device(gate_up.index, down)
    w = Fp4Experts(experts, d, f, gate_up.format, gate_up.scale, down.scale, gate_up.device, stream)
    if stream is not None:
        _read_on(stream, gate_up._memory, gate_up.scale, down._memory, down.scale)
    _call("fp4_experts_pack", w.index, stream, load().fp4_experts_pack, gate_up._ref, down._ref, w._ref)
    return w


def fp4_moe(x, router, experts, top_k, renormalize=True, out=None, return_routing=False, stream=None):
    """A mixture-of-experts layer for a few tokens (``fp4_moe`` in ``include/fp4.h``).

    x: M x d (float32, bfloat16 or float16); router: experts x d float32;
    ``experts``: an :class:`Fp4Experts`.  Each token goes to the ``top_k``
    experts of its largest logits, weighted by their softmax (divided by its
    sum over them if ``renormalize``).  Returns y (M x d, x's type), and with
    ``return_routing`` also the experts' indices (int32) and weights (float32),
    M x top_k.
    """
    if not isinstance(experts, Fp4Experts):
        raise TypeError("experts must be an Fp4Experts")
    ldx, tokens, d = _dense(x, "x", experts.d)
    ldr, rows, _ = _dense(router, "router", d)
    if router.dtype != torch.float32 or rows != experts.experts:
        raise ValueError(f"router must be {experts.experts} x {d} float32, got {tuple(router.shape)} {router.dtype}")
    device, index, top_k, dtype = experts.device, experts.index, int(top_k), x.dtype
    _same_device(index, x, router)
    if not 1 <= top_k <= min(32, experts.experts):
        raise ValueError(f"top_k must be between 1 and {min(32, experts.experts)}, got {top_k}")
    out, ldy = _output(out, (tokens, d), dtype, device, index, stream)
    ids = p = None
    if return_routing:
        ids = _empty((tokens, top_k), torch.int32, device, stream)
        p = _empty((tokens, top_k), torch.float32, device, stream)
    if stream is not None:
        _read_on(stream, x, router, experts.gate_up, experts.down, experts.gate_up_scale, experts.down_scale, out)
    _call("fp4_moe", index, stream, load().fp4_moe, _DTYPES[dtype], x.data_ptr(), ldx, tokens, router.data_ptr(), ldr,
          experts._ref, top_k, 1 if renormalize else 0, out.data_ptr(), ldy, ids.data_ptr() if return_routing else 0,
          p.data_ptr() if return_routing else 0)
    return (out, ids, p) if return_routing else out
