"""Plain CPU oracle of the norms around the linears, numpy float64.

Shares no code with the HIP path: the formulas as they stand, one row after
another where that is plainest.  Bfloat16 arrays are passed as float32 arrays
of their values.
"""

import math

import numpy as np

from . import convrot_oracle as base
from . import mx_oracle as mx


def norm(v, kind, eps, weight=None, bias=None):
    """((v - mu) r) weight + bias of rows [M, D], before any modulation."""
    v = np.asarray(v, dtype=np.float64)
    out = np.empty_like(v)
    for i, row in enumerate(v):
        mu = math.fsum(row) / len(row) if kind == "layer" and np.isfinite(row).all() else \
            (row.mean() if kind == "layer" else 0.0)
        d = row - mu
        with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
            out[i] = d * (1.0 / np.sqrt((d * d).mean() + eps))
    if weight is not None:
        out = out * np.asarray(weight, dtype=np.float64)
    if bias is not None:
        out = out + np.asarray(bias, dtype=np.float64)
    return out


def modulate(n, scale=None, shift=None):
    """n (1 + scale) + shift with a modulation's row for each of n's."""
    if scale is not None:
        n = n * (1.0 + np.asarray(scale, dtype=np.float64))
    if shift is not None:
        n = n + np.asarray(shift, dtype=np.float64)
    return n


def residual(x, y, residual_scale=1.0, gate=None, post=None):
    """h = residual_scale x + gate post(y); post: (kind, eps, weight, bias) or None."""
    y = np.asarray(y, dtype=np.float64) if post is None else norm(y, *post)
    if gate is not None:
        y = y * np.asarray(gate, dtype=np.float64)
    return residual_scale * np.asarray(x, dtype=np.float64) + y


def quantize_int8(n):
    """Rotated and quantised by row: (codes int8, scales fp32); a row that is not finite: 0 and NaN."""
    u = mx.rotate_f32(n)
    bad = ~np.isfinite(u).all(1)
    q, s = base.quantize_rows(np.where(bad[:, None], np.float32(0), u))
    return np.where(bad[:, None], 0, q).astype(np.int8), np.where(bad, np.float32(np.nan), s).astype(np.float32)
