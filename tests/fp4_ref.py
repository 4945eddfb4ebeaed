"""Plain implementation of the microscaled 4-bit operators for the tests, in numpy.

Written from the definitions in ``include/fp4.h``: quantisation with its
32-bit roundings (each one IEEE operation), everything else in 64 bits.
Nothing here uses the library.
"""
import numpy as np
import torch

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def e4m3_values():
    """Value of every scale byte of nvfp4 (127: NaN)."""
    b = np.arange(128)
    e, m = b >> 3, b & 7
    v = np.where(e > 0, 2.0 ** (e - 7.0) * (1 + m / 8.0), m * 2.0 ** -9)
    v[127] = np.nan
    return v


E4M3 = e4m3_values()


def nearest_even(v, table):
    """Index of the nearest entry of an increasing table, ties to the even index."""
    i = np.clip(np.searchsorted(table, v, side="right") - 1, 0, len(table) - 2)
    lo, hi = v - table[i], table[i + 1] - v
    return np.where((hi < lo) | ((hi == lo) & (i % 2 == 1)), i + 1, i)


def quantize(x, fmt, g=1.0):
    """(codes rows x cols, scale bytes rows x blocks) of a 2-D array that 32 bits hold exactly."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    n = BLOCK[fmt]
    blocks = -(-cols // n)
    b = np.zeros((rows, blocks * n), dtype=np.float32)
    b[:, :cols] = x
    b = b.reshape(rows, blocks, n)
    bad = ~np.isfinite(b).all(-1)
    a = np.where(bad, 0, np.abs(np.where(np.isfinite(b), b, 0)).max(-1)).astype(np.float32)
    if fmt == "mxfp4":
        e = np.clip(np.frexp(a.astype(np.float64))[1] - 1 - 2, -127, 127)
        byte = np.where(a > 0, e + 127, 0)
        unit = 2.0 ** (byte - 127.0)
        byte = np.where(bad, 255, byte)
    else:
        g = np.float32(g)
        t = (a / (np.float32(6) * g)).astype(np.float32) if g else np.where(a > 0, np.inf, 0)
        byte = nearest_even(np.minimum(t, 448).astype(np.float64), E4M3[:127])
        unit = (E4M3[byte].astype(np.float32) * g).astype(np.float32).astype(np.float64)
        byte = np.where(bad, 127, byte)
    with np.errstate(all="ignore"):
        q = np.where(unit[..., None] > 0, (b.astype(np.float64) / unit[..., None]).astype(np.float32), 0)
    q = np.where(bad[..., None], 0, q).astype(np.float64)
    code = nearest_even(np.minimum(np.abs(q), 6), LEVELS) | (np.signbit(q).astype(int) << 3)
    return code.reshape(rows, -1)[:, :cols], byte


def values(codes, scales, fmt, g=1.0):
    """64-bit values of codes (one an element) and scale bytes."""
    n = BLOCK[fmt]
    v = LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    if fmt == "mxfp4":
        unit = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    else:
        unit = E4M3[scales & 127] * float(np.float32(g))
    return v * np.repeat(unit, n, axis=1)[:, : codes.shape[1]]


def packed(codes):
    """Two codes a byte, the even column in the low bits."""
    c = np.pad(codes, ((0, 0), (0, codes.shape[1] % 2))).astype(np.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4)


def read_codes(q):
    """(codes rows x cols, scale bytes rows x blocks) of a library matrix, and whether its padding is zero."""
    rows, cols = q.shape
    raw = q.codes.cpu().numpy()
    codes = np.stack((raw & 15, raw >> 4), -1).reshape(rows, -1)
    n = BLOCK[q.format]
    blocks, atoms = -(-cols // n), -(-cols // 256) * 64 // n
    r, k = np.meshgrid(np.arange(rows), np.arange(atoms * 4), indexing="ij")
    at = (((r // 128) * atoms + k // 4) * 32 + r % 32) * 16 + (r % 128) // 32 * 4 + k % 4
    scales = q.scales.cpu().numpy()[at]
    clean = not codes[:, cols:].any() and not scales[:, blocks:].any()
    return codes[:, :cols].astype(int), scales[:, :blocks].astype(int), clean


def moe(x, router, gate_up, down, top, renormalize):
    """(y, ids, p) in 64 bits; gate_up experts x 2f x d and down experts x d x f are 64-bit values."""
    x, router = np.asarray(x, dtype=np.float64), np.asarray(router, dtype=np.float64)
    f = gate_up.shape[1] // 2
    logits = x @ router.T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top]
    e = np.exp(logits - logits.max(1, keepdims=True))
    p = np.take_along_axis(e / e.sum(1, keepdims=True), ids, 1)
    if renormalize:
        p = p / p.sum(1, keepdims=True)
    y = np.zeros_like(x)
    for t in range(len(x)):
        for j in range(top):
            gu = gate_up[ids[t, j]] @ x[t]
            gate = gu[:f]
            with np.errstate(over="ignore"):
                h = gate / (1 + np.exp(-gate)) * gu[f:]
            y[t] += p[t, j] * (down[ids[t, j]] @ h)
    return y, ids, p


def as_numpy(t):
    return t.detach().to(torch.float64).cpu().numpy()
