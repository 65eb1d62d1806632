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
A row with an index out of range is padding: nothing is written for it.

As in the rest of the package only arguments are marshalled here; every step
runs in the library's HIP kernels on the current stream.
"""

from __future__ import annotations

import ctypes
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


class _Desc(ctypes.Structure):
    _fields_ = [("kind", _int), ("eps", _f32), ("weight", _vp), ("bias", _vp)]


class _Modulation(ctypes.Structure):
    _fields_ = [("scale", _vp), ("shift", _vp), ("gate", _vp), ("scale_stride", _i64), ("shift_stride", _i64),
                ("gate_stride", _i64), ("dtype", _int), ("rows", _i64), ("index", _vp)]


class _Out(ctypes.Structure):
    _fields_ = [("kind", _int), ("values", _vp), ("scales", _vp)]


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


def _rows(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, int]:
    """t [..., D] as rows [M, D] with contiguous elements, and their stride."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a float16 or bfloat16 tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (no CPU path exists)")
    if like is not None and (t.dtype != like.dtype or t.shape != like.shape or t.device != like.device):
        raise ValueError(f"{name} must have x's shape, dtype and device")
    if t.dim() == 0 or t.shape[-1] == 0:
        raise ValueError(f"{name} must be [..., D] with D at least 1")
    if t.dim() != 2:
        m = t.numel() // t.shape[-1]
        t = t.reshape(m, t.shape[-1])
    if t.stride(1) != 1 and t.shape[1] > 1 or not 0 <= t.stride(0) <= 0x7FFFFFFF:
        t = t.contiguous()
    return t, t.stride(0)


def _desc(kind: str, eps: float, weight, bias, d: int, device) -> Tuple[_Desc, tuple]:
    if kind not in _KINDS:
        raise ValueError(f"the norm's kind must be 'rms' or 'layer', got {kind!r}")
    kept = []
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            if t.dtype != torch.float32:
                raise TypeError(f"a norm's {name} must be float32, got {t.dtype}")
            if t.shape != (d,) or t.device != device:
                raise ValueError(f"a norm's {name} must be [{d}] on {device}")
            t = t.contiguous()
        kept.append(t)
    return _Desc(_KINDS[kind], eps, *(None if t is None else t.data_ptr() for t in kept)), kept


def _modulation(x: torch.Tensor, scale, shift, gate, index) -> Tuple[Optional[_Modulation], list]:
    m, d = x.shape
    kept, rows, dtype = [], None, None
    for name, t in (("scale", scale), ("shift", shift), ("gate", gate)):
        if t is None:
            kept.append(None)
            continue
        if t.dtype != x.dtype and t.dtype != torch.float32 or dtype not in (None, t.dtype):
            raise TypeError("scale, shift and gate must have one dtype, x's or float32")
        if t.dim() == 1:
            t = t[None]
        if t.dim() != 2 or t.shape[1] != d or rows not in (None, t.shape[0]) or t.device != x.device:
            raise ValueError(f"{name} must be [rows, {d}] on {x.device}, with as many rows as the others")
        if t.stride(1) != 1 and d > 1 or not 0 <= t.stride(0) <= 0x7FFFFFFF:
            t = t.contiguous()
        rows, dtype = t.shape[0], t.dtype
        kept.append(t)
    if rows is None:
        if index is not None:
            raise ValueError("index names rows of scale, shift or gate, which are not given")
        return None, kept
    if index is not None:
        if index.dtype != torch.int32:
            raise TypeError(f"index must be int32, got {index.dtype}")
        if index.shape != (m,) or index.device != x.device:
            raise ValueError(f"index must be [{m}] on {x.device}")
        index = index.contiguous()
    elif rows == 0 or m % rows:
        raise ValueError(f"{m} rows do not split into {rows} equal parts (give index)")
    kept.append(index)
    at = [None if t is None else t.data_ptr() for t in kept[:3]]
    step = [0 if t is None else t.stride(0) for t in kept[:3]]
    return _Modulation(*at, *step, _MOD_F32 if dtype == torch.float32 and x.dtype != dtype else _DTYPES[x.dtype],
                       rows, None if index is None else index.data_ptr()), kept


def _ref(s):
    return None if s is None else ctypes.addressof(s)


def _dense(t: Optional[torch.Tensor], like: torch.Tensor, name: str) -> torch.Tensor:
    """The output [M, D] for x, given or new."""
    if t is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    if t.dtype != like.dtype or t.shape != like.shape or not t.is_contiguous() or t.device != like.device:
        raise ValueError(f"{name} must be a contiguous tensor of x's shape, dtype and device")
    return t


def _quantised(m: int, d: int, bits: int, device) -> Tuple[int, torch.Tensor, torch.Tensor]:
    if bits == 4:
        return (_OUT_MXFP4, *_empty4(m, d, device))
    if bits != 8:
        raise ValueError("bits must be 4 or 8")
    if d % GROUP:
        raise ValueError(f"the row length must be a multiple of {GROUP}, got {d}")
    return (_OUT_INT8, torch.empty((m, d), dtype=torch.int8, device=device),
            torch.empty((m,), dtype=torch.float32, device=device))


def _norm(x, kind, eps, weight, bias, scale, shift, index, out):
    """One call; out is (kind, values, scales) for x's rows."""
    rows, stride = _rows(x, "x")
    m, d = rows.shape
    desc, kept = _desc(kind, eps, weight, bias, d, rows.device)
    mod, kept_mod = _modulation(rows, scale, shift, None, index)
    o = _Out(out[0], out[1].data_ptr(), None if out[2] is None else out[2].data_ptr())
    _call(_lib().convrot_norm, "convrot_norm", rows.device, rows.data_ptr(), stride, _DTYPES[rows.dtype], m, d,
          _ref(desc), _ref(mod), _ref(o))
    del kept, kept_mod


def norm(x: torch.Tensor, kind: str = "layer", eps: float = 1e-6, weight: Optional[torch.Tensor] = None,
         bias: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
         shift: Optional[torch.Tensor] = None, index: Optional[torch.Tensor] = None,
         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The norm ("layer" or "rms") of x fp16 or bf16 [..., D] with its weight
    and bias (fp32 [D]) and modulation; returns x's shape and dtype (into
    ``out``, contiguous, where given)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a float16 or bfloat16 tensor")
    out = _dense(out, x, "out")
    _norm(x, kind, eps, weight, bias, scale, shift, index, (_OUT_16, out, None))
    return out


def norm_quant(x: torch.Tensor, bits: int, kind: str = "layer", eps: float = 1e-6,
               weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
               index: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The norm of x [..., D] (M rows), rotated and quantised: with bits 8 the
    codes int8 [M, D] and scales fp32 [M] that gemm_i8_f16 takes, with bits 4
    the codes and scales that mx_gemm takes."""
    rows, _ = _rows(x, "x")
    how, values, scales = _quantised(*rows.shape, bits, rows.device)
    _norm(x, kind, eps, weight, bias, scale, shift, index, (how, values, scales))
    return values, scales


def _residual(x, y, kind, eps, weight, bias, scale, shift, gate, index, residual_scale, post, post_eps, post_weight,
              post_bias, h, out):
    rows, stride = _rows(x, "x")
    block, block_stride = _rows(y, "y", like=x)
    m, d = rows.shape
    kept = []
    after = before = None
    if post is not None:
        after, k = _desc(post, post_eps, post_weight, post_bias, d, rows.device)
        kept.append(k)
    elif post_weight is not None or post_bias is not None:
        raise ValueError("post_weight and post_bias belong to a norm of y: give post")
    if kind is not None:
        before, k = _desc(kind, eps, weight, bias, d, rows.device)
        kept.append(k)
    elif any(t is not None for t in (weight, bias, scale, shift)):
        raise ValueError("weight, bias, scale and shift belong to a norm of h: give kind")
    mod, kept_mod = _modulation(rows, scale, shift, gate, index)
    o = None if out is None else _Out(out[0], out[1].data_ptr(), None if out[2] is None else out[2].data_ptr())
    _call(_lib().convrot_residual_norm, "convrot_residual_norm", rows.device, rows.data_ptr(), stride,
          block.data_ptr(), block_stride, _DTYPES[rows.dtype], m, d, residual_scale, _ref(after), _ref(before),
          _ref(mod), h.data_ptr(), _ref(o))
    del kept, kept_mod


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
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a float16 or bfloat16 tensor")
    h, n = out if out is not None else (None, None)
    h = _dense(h, x, "out's h")
    n = _dense(n, x, "out's n") if kind is not None else None
    _residual(x, y, kind, eps, weight, bias, scale, shift, gate, index, residual_scale, post, post_eps, post_weight,
              post_bias, h, None if n is None else (_OUT_16, n, None))
    return h, n


def residual_norm_quant(x: torch.Tensor, y: torch.Tensor, bits: int, kind: str = "layer", eps: float = 1e-6,
                        weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                        scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, index: Optional[torch.Tensor] = None,
                        residual_scale: float = 1.0, post: Optional[str] = None, post_eps: float = 1e-6,
                        post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """residual_norm with the norm rotated and quantised as by norm_quant:
    returns (h, codes, scales); h into ``out`` where given (x or y itself)."""
    rows, _ = _rows(x, "x")
    if kind is None:
        raise ValueError("kind must be 'rms' or 'layer'")
    h = _dense(out, x, "out")
    how, values, scales = _quantised(*rows.shape, bits, rows.device)
    _residual(x, y, kind, eps, weight, bias, scale, shift, gate, index, residual_scale, post, post_eps, post_weight,
              post_bias, h, (how, values, scales))
    return h, values, scales
