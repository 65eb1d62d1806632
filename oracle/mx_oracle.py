"""Plain CPU oracle of the rotated 4-bit linear (MXFP4), numpy float64.

Shares no code with the HIP path.  The rotated rows come from the linears'
oracle or the caller; codes are found by comparing with the borders between
neighbouring values, exponents by comparing with powers of two.  Bfloat16
arrays are passed as float32 arrays of their values.
"""

import numpy as np

from .convrot_oracle import hadamard256

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])   # codes 0 .. 7; 8 .. 15 are their negatives


def rotate_f32(x: np.ndarray) -> np.ndarray:
    """fp32(x H) in groups of 256; a sum of 0 is +0.  The sums are in extended
    precision (64 bits of mantissa), so that those of equal sizes and unlike
    signs, partial sums k c of c in float64, cancel exactly."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        u = x.reshape(-1, 256).astype(np.longdouble) @ hadamard256().astype(np.longdouble)
        return (u + 0.0).astype(np.float32).reshape(x.shape)


def exponent(top: np.ndarray) -> np.ndarray:
    """max(floor(log2 top) - 2, -127), -127 for 0, by comparison with powers of two."""
    powers = 2.0 ** np.arange(-149, 128)
    e = np.searchsorted(powers, np.asarray(top, dtype=np.float64), side="right") - 1 - 149
    return np.maximum(np.where(top > 0, e - 2, -127), -127)


def encode(v: np.ndarray) -> np.ndarray:
    """The 4-bit codes of values v, nearest, ties to the even code, beyond 6 to 6."""
    a = np.abs(v)
    c = np.zeros(v.shape, dtype=np.int64)
    for i in range(7):
        border = (GRID[i] + GRID[i + 1]) / 2
        c += (a >= border) if i % 2 else (a > border)      # a tie goes up where the upper code is even
    return np.where(np.signbit(v), c + 8, c)


def decode(c: np.ndarray) -> np.ndarray:
    return np.concatenate([GRID, -GRID])[c]


def quantize(u: np.ndarray):
    """u float32 [rows, K] -> (codes int64 [rows, K], scale bytes int64 [rows, K / 32])."""
    rows, k = u.shape
    b = u.astype(np.float64).reshape(rows, k // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    e = exponent(np.abs(b).max(-1))
    c = encode(b / 2.0 ** e[..., None])
    c = np.where(bad[..., None], 0, c)
    return c.reshape(rows, k), np.where(bad, 255, e + 127)


def pack(codes: np.ndarray, scales: np.ndarray):
    """Codes and scale bytes as the library holds them."""
    rows, k = codes.shape
    q = (codes[:, 0::2] + 16 * codes[:, 1::2]).astype(np.uint8)
    return q, np.ascontiguousarray(scales.astype(np.uint8).reshape(rows, k // 256, 8).transpose(1, 0, 2))


def unpack(q: np.ndarray, s: np.ndarray):
    rows, k = q.shape[0], 2 * q.shape[1]
    c = np.empty((rows, k), dtype=np.int64)
    c[:, 0::2], c[:, 1::2] = q % 16, q // 16
    return c, s.transpose(1, 0, 2).reshape(rows, k // 32).astype(np.int64)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What codes and scale bytes stand for, in the rotated basis, float64."""
    rows, k = codes.shape
    s = np.where(scales == 255, np.nan, 2.0 ** (scales - 127.0))
    return (decode(codes).reshape(rows, k // 32, 32) * s[..., None]).reshape(rows, k)


def dequantize(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The rows themselves, un-rotated, float64 (before the roundings to fp32 and to the type)."""
    v = values(codes, scales)
    return (v.reshape(-1, 256) @ hadamard256()).reshape(v.shape)


def product(x: np.ndarray, w: np.ndarray, bias=None, residual=None):
    """(y, terms): x w^T + bias + residual of rows as values, float64, and the sum of its terms' sizes."""
    y, t = x @ w.T, np.abs(x) @ np.abs(w).T
    for extra in (bias, residual):
        if extra is not None:
            y, t = y + np.asarray(extra, dtype=np.float64), t + np.abs(extra)
    return y, t
