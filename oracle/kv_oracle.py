"""Plain CPU oracle of the rotated, quantised key/value cache, numpy float64.

Shares no code with the HIP path.  Rotation by the explicitly built +-1
matrix (popcount form); quantisation in the fp32 steps that the contract
states; attention by the definition on the de-quantised, un-rotated rows.
Bfloat16 arrays are passed as float32 arrays of their values.
"""

import numpy as np


def signs(d: int) -> np.ndarray:
    """W[i, j] = (-1)^popcount(i & j), the Sylvester-Hadamard matrix."""
    a = np.arange(d)
    m = a[:, None] & a[None, :]
    odd = np.zeros_like(m)
    while m.any():
        odd ^= m & 1
        m = m >> 1
    return 1.0 - 2.0 * odd


def qmax(bits: int) -> int:
    return 7 if bits == 4 else 127


def quantize(x: np.ndarray, bits: int):
    """x [..., D] -> (codes int8 [..., D], scale float32 [...])."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        u = (x @ signs(d)).astype(np.float32)
        top = np.abs(u).max(-1)
        s = (top / np.float32(qmax(bits))).astype(np.float32)
        c = np.rint(u / s[..., None])
        bad = ~np.isfinite(u).all(-1)
        c = np.where((s[..., None] > 0) & ~bad[..., None], c, 0.0)
        scale = s * np.float32(1.0 / np.sqrt(d))
    scale = np.where(bad, np.float32(np.nan), scale).astype(np.float32)
    return c.astype(np.int8), scale


def pack(codes: np.ndarray, bits: int) -> np.ndarray:
    """Codes as the cache holds them: int8, or two 4-bit codes a byte, the even element low."""
    if bits == 8:
        return codes
    c = codes.astype(np.int64) & 15
    return (c[..., 0::2] + 16 * c[..., 1::2]).astype(np.uint8)


def unpack(raw: np.ndarray, bits: int) -> np.ndarray:
    if bits == 8:
        return raw.astype(np.int64)
    r = raw.astype(np.int64)
    c = np.empty(r.shape[:-1] + (2 * r.shape[-1],), dtype=np.int64)
    c[..., 0::2] = r % 16
    c[..., 1::2] = r // 16
    return np.where(c > 7, c - 16, c)


def rows(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """The rows that codes [..., D] and scales stand for, float64."""
    d = codes.shape[-1]
    return (codes.astype(np.float64) @ signs(d)) * (scale.astype(np.float64) / np.sqrt(d))[..., None]


def read_f32(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """The value kv_read rounds to its output type: fp32(c W) * fp32(scale * fp32(D^-1/2)), fp32."""
    d = codes.shape[-1]
    n = (codes.astype(np.float64) @ signs(d)).astype(np.float32)
    return n * (scale * np.float32(1.0 / np.sqrt(d)))[..., None]


def attention(q, k, v, scale, causal):
    """q [n, heads_q, D], k and v [m, heads, D] of one sequence, float64 ->
    (o [n, heads_q, D], spread [n, heads_q, 2]): o by the definition (zeros
    where no key is visible), and what rounding errors of the softmax weights
    are relative to: spread[..., 0] = sum_j p_j |v_j| for errors that add up,
    spread[..., 1] = sqrt(sum_j p_j^2 |v_j|^2) for independent ones."""
    n, hq, d = q.shape
    m, h = k.shape[0], k.shape[1]
    o, spread = np.zeros((n, hq, d)), np.zeros((n, hq, 2))
    for a in range(hq if m else 0):
        s = scale * (q[:, a] @ k[:, a // (hq // h)].T)
        if causal:
            s = np.where(np.arange(m)[None] <= (m - n + np.arange(n))[:, None], s, -np.inf)
        top = s.max(-1, keepdims=True)
        e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
        total = e.sum(-1, keepdims=True)
        p = np.divide(e, total, out=np.zeros_like(e), where=total > 0)
        vh = v[:, a // (hq // h)]
        o[:, a] = p @ vh
        size = (vh * vh).sum(-1)
        spread[:, a, 0] = p @ np.sqrt(size)
        spread[:, a, 1] = np.sqrt((p * p) @ size)
    return o, spread
