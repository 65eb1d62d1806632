"""The norms around the linears: Python binding of include/convrot_norm.h.

  n = norm(x, scale=scale, shift=shift)                       # in front of a linear
  q, s = norm_quant(x, bits=4, scale=scale, shift=shift)      # ... as mx_gemm (4) or gemm_i8_f16 (8) reads it
  h, n = residual_norm(x, y, gate=gate, scale=..., shift=...) # behind a block, with the next block's norm
  h, q, s = residual_norm_quant(x, y, bits=4, gate=gate, ...)

with n = (norm(x) weight + bias)(1 + scale) + shift and
h = residual_scale x + gate post(y).  scale, shift and gate are rows of a
modulation, [rows, D] (or [D]) of x's dtype or fp32, with any stride between
rows (slices of a conditioning's projection are read in place): each serves
M / rows consecutive rows of x, or those whose ``index`` (int32 [M]) names it.
A row with an index out of range is padding: nothing is written for it, so it
keeps what ``out`` held, or whatever the memory of a new output held.

As in the rest of the package only arguments are marshalled here; every step
runs in the library's HIP kernels on the current stream.
"""

from __future__ import annotations

import ctypes
import struct
from typing import Optional, Tuple

import torch

from . import GROUP, _DTYPES, _f32, _i64, _vp
from . import lib as _base_lib
from .kv import _call
from .mx import _empty4

_int = ctypes.c_int
_KINDS = {"rms": 1, "layer": 2}
_OUT_16, _OUT_INT8, _OUT_MXFP4 = 0, 1, 2
_MOD_F32 = 2


# The call's structures as their bytes (native alignment): packing them takes a
# third of a ctypes.Structure's time, which is most of a small call's.
_DESC = struct.Struct("@ifPP0P")          # kind, eps, weight, bias
_MOD = struct.Struct("@PPPqqqiqP")        # scale, shift, gate, their strides, dtype, rows, index
_OUT = struct.Struct("@iPP0P")            # kind, values, scales

_NORM_SIGNATURES = {
    "convrot_norm": (_int, [_vp, _i64, _int, _i64, _i64, _vp, _vp, _vp, _vp]),
    "convrot_residual_norm": (_int, [_vp, _i64, _vp, _i64, _int, _i64, _i64, _f32, _vp, _vp, _vp, _vp, _vp, _vp]),
}

_norm_lib: Optional[ctypes.CDLL] = None


def _lib() -> ctypes.CDLL:
    global _norm_lib
    if _norm_lib is None:
        handle = _base_lib()
        for name, (res, args) in _NORM_SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _norm_lib = handle
    return _norm_lib


def _rows(t: torch.Tensor, name: str) -> Tuple[torch.Tensor, int, int, int]:
    """t [..., D] as rows [M, D] with contiguous elements, their stride, M and D."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a float16 or bfloat16 tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (no CPU path exists)")
    shape = t.shape
    if not shape or shape[-1] == 0:
        raise ValueError(f"{name} must be [..., D] with D at least 1")
    d = shape[-1]
    if len(shape) != 2:
        t = t.reshape(t.numel() // d, d)
    row, one = t.stride()
    if one != 1 and d > 1 or not 0 <= row <= 0x7FFFFFFF:
        t = t.contiguous()
        row = d
    return t, row, t.shape[0], d


def _desc(kind: str, eps: float, weight, bias, d: int, index: int) -> Tuple[bytes, tuple]:
    if kind not in _KINDS:
        raise ValueError(f"the norm's kind must be 'rms' or 'layer', got {kind!r}")
    kept = (weight, bias)
    if weight is None and bias is None:
        return _DESC.pack(_KINDS[kind], eps, 0, 0), kept
    for t in kept:
        if t is not None:
            if t.dtype is not torch.float32:
                raise TypeError(f"a norm's weight and bias must be float32, got {t.dtype}")
            if t.shape != (d,) or t.get_device() != index:
                raise ValueError(f"a norm's weight and bias must be [{d}] on x's device")
    kept = tuple(None if t is None else t.contiguous() for t in kept)
    return _DESC.pack(_KINDS[kind], eps, *(0 if t is None else t.data_ptr() for t in kept)), kept


def _modulation(x: torch.Tensor, m: int, d: int, scale, shift, gate, index) -> Tuple[Optional[bytes], list]:
    kept, at, step, rows, dtype, device = [], [], [], None, None, x.get_device()
    for t in (scale, shift, gate):
        if t is None:
            at.append(0)
            step.append(0)
            continue
        if dtype is None:
            dtype = t.dtype
            if dtype is not x.dtype and dtype is not torch.float32:
                raise TypeError("scale, shift and gate must have x's dtype or float32")
        elif t.dtype is not dtype:
            raise TypeError("scale, shift and gate must have one dtype")
        shape = t.shape
        if len(shape) == 1:
            t, shape = t[None], (1, shape[0])
        if len(shape) != 2 or shape[1] != d or rows not in (None, shape[0]) or t.get_device() != device:
            raise ValueError(f"scale, shift and gate must be [rows, {d}], of as many rows each, on x's device")
        rows = shape[0]
        row, one = t.stride()
        if one != 1 and d > 1 or not 0 <= row <= 0x7FFFFFFF:
            t = t.contiguous()
            row = d
        kept.append(t)
        at.append(t.data_ptr())
        step.append(row)
    if rows is None:
        if index is not None:
            raise ValueError("index names rows of scale, shift or gate, which are not given")
        return None, kept
    if rows == 0 and m == 0:             # an empty batch
        return None, kept
    if index is not None:
        if index.dtype is not torch.int32:
            raise TypeError(f"index must be int32, got {index.dtype}")
        if index.shape != (m,) or index.get_device() != device:
            raise ValueError(f"index must be [{m}] on x's device")
        index = index.contiguous()
        kept.append(index)
    elif rows == 0 or m % rows:
        raise ValueError(f"{m} rows do not split into {rows} equal parts (give index)")
    return _MOD.pack(*at, *step, _MOD_F32 if dtype is torch.float32 else _DTYPES[dtype], rows,
                     0 if index is None else index.data_ptr()), kept


def _dense(t: Optional[torch.Tensor], like: torch.Tensor, name: str) -> torch.Tensor:
    """The output [M, D] for x, given or new."""
    if t is None:
        return like.new_empty(like.shape)
    if t.dtype is not like.dtype or t.shape != like.shape or not t.is_contiguous() or t.device != like.device:
        raise ValueError(f"{name} must be a contiguous tensor of x's shape, dtype and device")
    return t


def _given(t: torch.Tensor, shape: tuple, dtype: torch.dtype, like: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != like.device or t.data_ptr() % 16:
        raise ValueError(f"out's {name} must be a contiguous {dtype} tensor {list(shape)} on x's device, aligned to 16 bytes")
    return t


def _quantised(m: int, d: int, bits: int, like: torch.Tensor, out=None) -> Tuple[int, torch.Tensor, torch.Tensor]:
    """The output's kind, and codes and scales, new or (either of the two) given."""
    if out is not None:
        values, scales = out
        if values is None or scales is None:
            _, v, s = _quantised(m, d, bits, like)
            values, scales = v if values is None else values, s if scales is None else scales
        if bits == 4:
            return (_OUT_MXFP4, _given(values, (m, d // 2), torch.uint8, like, "codes"),
                    _given(scales, (d // GROUP, m, 8), torch.uint8, like, "scales"))
    elif bits == 4:
        return (_OUT_MXFP4, *_empty4(m, d, like))
    if bits != 8:
        raise ValueError("bits must be 4 or 8")
    if d % GROUP:
        raise ValueError(f"the row length must be a multiple of {GROUP}, got {d}")
    if out is not None:
        return (_OUT_INT8, _given(values, (m, d), torch.int8, like, "codes"),
                _given(scales, (m,), torch.float32, like, "scales"))
    return _OUT_INT8, like.new_empty((m, d), dtype=torch.int8), like.new_empty((m,), dtype=torch.float32)


def _norm(rows, stride, m, d, kind, eps, weight, bias, scale, shift, index, out, values, scales):
    desc, kept = _desc(kind, eps, weight, bias, d, rows.get_device())
    mod, kept_mod = _modulation(rows, m, d, scale, shift, None, index)
    o = _OUT.pack(out, values.data_ptr(), 0 if scales is None else scales.data_ptr())
    _call(_lib().convrot_norm, "convrot_norm", rows.device, rows.data_ptr(), stride, _DTYPES[rows.dtype], m, d, desc,
          mod, o)
    del kept, kept_mod


def norm(x: torch.Tensor, kind: str = "layer", eps: float = 1e-6, weight: Optional[torch.Tensor] = None,
         bias: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
         shift: Optional[torch.Tensor] = None, index: Optional[torch.Tensor] = None,
         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The norm ("layer" or "rms") of x fp16 or bf16 [..., D] with its weight
    and bias (fp32 [D]) and modulation; returns x's shape and dtype (into
    ``out``, contiguous, where given)."""
    rows = _rows(x, "x")
    out = _dense(out, x, "out")
    _norm(*rows, kind, eps, weight, bias, scale, shift, index, _OUT_16, out, None)
    return out


def norm_quant(x: torch.Tensor, bits: int, kind: str = "layer", eps: float = 1e-6,
               weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
               index: Optional[torch.Tensor] = None,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The norm of x [..., D] (M rows), rotated and quantised: with bits 8 the
    codes int8 [M, D] and scales fp32 [M] that gemm_i8_f16 takes, with bits 4
    the codes and scales that mx_gemm takes (into ``out``, where given)."""
    rows = _rows(x, "x")
    how, values, scales = _quantised(*rows[2:], bits, x, out)
    _norm(*rows, kind, eps, weight, bias, scale, shift, index, how, values, scales)
    return values, scales


def _residual(rows, stride, m, d, y, kind, eps, weight, bias, scale, shift, gate, index, residual_scale, post, post_eps,
              post_weight, post_bias, h, out, values, scales):
    block, block_stride, _, _ = _rows(y, "y")
    device = rows.get_device()
    kept = []
    after = before = o = None
    if post is not None:
        after, k = _desc(post, post_eps, post_weight, post_bias, d, device)
        kept.append(k)
    elif post_weight is not None or post_bias is not None:
        raise ValueError("post_weight and post_bias belong to a norm of y: give post")
    if kind is not None:
        before, k = _desc(kind, eps, weight, bias, d, device)
        kept.append(k)
        o = _OUT.pack(out, values.data_ptr(), 0 if scales is None else scales.data_ptr())
    elif weight is not None or bias is not None or scale is not None or shift is not None:
        raise ValueError("weight, bias, scale and shift belong to a norm of h: give kind")
    mod, kept_mod = _modulation(rows, m, d, scale, shift, gate, index)
    _call(_lib().convrot_residual_norm, "convrot_residual_norm", rows.device, rows.data_ptr(), stride,
          block.data_ptr(), block_stride, _DTYPES[rows.dtype], m, d, residual_scale, after, before, mod, h.data_ptr(), o)
    del kept, kept_mod


def _alike(x: torch.Tensor, y: torch.Tensor) -> None:
    if not isinstance(y, torch.Tensor):
        raise TypeError("y must be a float16 or bfloat16 tensor")
    if y.dtype is not x.dtype or y.shape != x.shape or y.get_device() != x.get_device():
        raise ValueError("y must have x's shape, dtype and device")


def residual_norm(x: torch.Tensor, y: torch.Tensor, kind: Optional[str] = "layer", eps: float = 1e-6,
                  weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, index: Optional[torch.Tensor] = None,
                  residual_scale: float = 1.0, post: Optional[str] = None, post_eps: float = 1e-6,
                  post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None,
                  out: Optional[Tuple[torch.Tensor, Optional[torch.Tensor]]] = None):
    """h = residual_scale x + gate post(y) of x and y [..., D], and the norm of
    h before its rounding; returns (h, n) of x's shape and dtype (into ``out``,
    where given; its h may be x or y itself).  ``post`` is None, "rms" or
    "layer"; with kind None there is no norm and n is None."""
    rows = _rows(x, "x")
    _alike(x, y)
    h, n = out if out is not None else (None, None)
    h = _dense(h, x, "out's h")
    n = _dense(n, x, "out's n") if kind is not None else None
    _residual(*rows, y, kind, eps, weight, bias, scale, shift, gate, index, residual_scale, post, post_eps, post_weight,
              post_bias, h, _OUT_16, n, None)
    return h, n


def residual_norm_quant(x: torch.Tensor, y: torch.Tensor, bits: int, kind: str = "layer", eps: float = 1e-6,
                        weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                        scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, index: Optional[torch.Tensor] = None,
                        residual_scale: float = 1.0, post: Optional[str] = None, post_eps: float = 1e-6,
                        post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None,
                        out=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """residual_norm with the norm rotated and quantised as by norm_quant:
    returns (h, codes, scales).  ``out`` is where h goes (x or y itself may be
    it), or a tuple of where all three go, None for a new one."""
    rows = _rows(x, "x")
    _alike(x, y)
    if kind is None:
        raise ValueError("kind must be 'rms' or 'layer'")
    h, codes = (out[0], out[1:]) if isinstance(out, (tuple, list)) else (out, None)
    h = _dense(h, x, "out's h")
    how, values, scales = _quantised(*rows[2:], bits, x, codes)
    _residual(*rows, y, kind, eps, weight, bias, scale, shift, gate, index, residual_scale, post, post_eps, post_weight,
              post_bias, h, how, values, scales)
    return h, values, scales
