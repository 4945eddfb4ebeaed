"""Plain implementation of the 8-bit integer operators for the tests, in numpy.

Written from the definitions in ``include/int8.h``: scales and the last steps
with their 32-bit roundings (each one IEEE operation), everything else in 64
bits, which hold the sums of integers exactly.  Nothing here uses the library.
"""
import numpy as np
import torch

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def array(t):
    """A tensor's values in 64 bits."""
    return t.detach().cpu().double().numpy()


def quantize(x):
    """(integers, 32-bit scales) of the rows of x (values that 32 bits hold)."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(-1)
    y = np.where(bad[:, None], 0.0, x)
    top = np.abs(y).max(-1, initial=0.0).astype(np.float32)
    s = np.maximum(top * (np.float32(1) / np.float32(127)), np.float32(2.0 ** -126))
    # Quotients of two 24-bit numbers: 64 bits tell each from a tie that it is not.
    q = np.rint(y / s.astype(np.float64)[:, None])
    return q.astype(np.int8), np.where(bad, np.float32(np.nan), s)


def round_to(v, dtype):
    """32-bit values rounded to `dtype` (a torch type), as a tensor of it."""
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(dtype)


def product(qa, sa, qb, sb, dtype):
    """The product, bit for bit: exact sums, three roundings to 32 bits, one to the type."""
    total = (qa.astype(np.float64) @ qb.astype(np.float64).T).astype(np.float32)
    a, b = np.broadcast_arrays(sa[:, None], sb[None, :])
    first = np.abs(b) <= np.abs(a)
    low, high = np.where(first, b, a), np.where(first, a, b)
    with np.errstate(all="ignore"):
        return round_to(total * low * high, dtype)


def keep(x, half):
    """(integers, units in 64 bits) of the blocks of the rows of x: rows x blocks x 32 and rows x blocks."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    b = np.zeros((rows, -(-cols // 32) * 32))
    b[:, :cols] = x
    b = b.reshape(rows, -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1, initial=0.0)
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 6, -1000)
    u = 2.0 ** np.maximum(e, -24 if half else -126).astype(np.float64)
    return np.clip(np.rint(b / u[..., None]), -127, 127), np.where(bad, np.nan, u)


def kept(x, half):
    """The values that the checkpoint of x stands for."""
    q, u = keep(x, half)
    return (q * u[..., None]).reshape(x.shape[0], -1)[:, :x.shape[1]]


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_backward(d, g, u):
    s = sigmoid(g)
    return d * u * s * (1 + g * (1 - s)), d * g * s


def half_step(dtype):
    """What a rounding to `dtype` adds, relative to the value."""
    return torch.finfo(dtype).eps / 2
