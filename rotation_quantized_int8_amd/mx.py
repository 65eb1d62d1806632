"""The rotated 4-bit linear (MXFP4): Python binding of include/convrot_mx.h.

  q_w, s_w = mx_quantize_weights(w)                  # offline, w fp32 [N, K]
  y = mx_linear(x, q_w, s_w, bias, residual)         # x fp16 or bf16 [..., K]

and its stages: mx_act_quant, mx_gemm, mx_dequantize.  A tensor in 4 bits is
two: codes uint8 [rows, K / 2] (e2m1, two a byte, the even element low) and
scales uint8 [K / 256, rows, 8] (exponent + 127 of each block of 32).

As in the rest of the package only arguments are marshalled here; every step
runs in the library's HIP kernels on the current stream.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import GROUP, _DTYPES, _flatten, _i64, _prep, _sz, _vp
from . import lib as _base_lib
from .kv import _call

_int = ctypes.c_int

_MX_SIGNATURES = {
    "convrot_mx_quantize_weights": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "convrot_mx_act_quant": (_int, [_vp, _int, _i64, _i64, _vp, _vp, _vp]),
    "convrot_mx_dequantize": (_int, [_vp, _vp, _i64, _i64, _vp, _int, _vp]),
    "convrot_mx_gemm": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _int, _vp]),
    "convrot_mx_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "convrot_mx_linear": (_int, [_vp, _int, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _int, _vp, _sz, _vp]),
}

_BAD_SIZE = ctypes.c_size_t(-1).value
_mx_lib: Optional[ctypes.CDLL] = None


def _lib() -> ctypes.CDLL:
    global _mx_lib
    if _mx_lib is None:
        handle = _base_lib()
        for name, (res, args) in _MX_SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _mx_lib = handle
    return _mx_lib


def _empty4(rows: int, k: int, like: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Uninitialised codes and scales on like's device."""
    if k % GROUP:
        raise ValueError(f"the row length must be a multiple of {GROUP}, got {k}")
    return (like.new_empty((rows, k // 2), dtype=torch.uint8),
            like.new_empty((k // GROUP, rows, 8), dtype=torch.uint8))


def _ready(t: torch.Tensor, dtype: torch.dtype, name: str) -> torch.Tensor:
    """t as the library takes it; the usual case first, since these checks are most of a small call's time."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.is_cuda and t.is_contiguous() and not t.data_ptr() % 16:
        return t
    return _prep(t, dtype, name)


def _pair(codes: torch.Tensor, scales: torch.Tensor, name: str) -> Tuple[torch.Tensor, torch.Tensor, int, int]:
    """Checked codes and scales, their rows and row length."""
    codes, scales = _ready(codes, torch.uint8, f"{name} codes"), _ready(scales, torch.uint8, f"{name} scales")
    shape = codes.shape
    if len(shape) != 2 or shape[1] % (GROUP // 2):
        raise ValueError(f"{name} codes must be [rows, K / 2] with K a multiple of {GROUP}, got {list(shape)}")
    rows, k = shape[0], shape[1] * 2
    if scales.shape != (k // GROUP, rows, 8):
        raise ValueError(f"{name} scales must be {[k // GROUP, rows, 8]}, got {list(scales.shape)}")
    return codes, scales, rows, k


def _same_device(like: torch.Tensor, *tensors) -> None:
    index = like.get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors of a call must be on one GPU, got {like.device} and {t.device}")


def _rows16(x: torch.Tensor) -> torch.Tensor:
    """x [..., K] as [M, K]."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise TypeError("x must be a float16 or bfloat16 tensor")
    x = _ready(x, x.dtype, "x")
    return x if x.dim() == 2 else _flatten(x)[0]


def mx_quantize_weights(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Offline: w fp32 [N, K] -> (codes uint8 [N, K / 2], scales uint8 [K / 256, N, 8])."""
    w = _ready(w, torch.float32, "W")
    if w.dim() != 2:
        raise ValueError("W must be [N, K]")
    n, k = w.shape
    codes, scales = _empty4(n, k, w)
    _call(_lib().convrot_mx_quantize_weights, "convrot_mx_quantize_weights", w.device, w.data_ptr(), n, k,
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def mx_act_quant(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """x fp16 or bf16 [..., K], M rows -> (codes uint8 [M, K / 2], scales uint8 [K / 256, M, 8])."""
    x = _rows16(x)
    m, k = x.shape
    codes, scales = _empty4(m, k, x)
    _call(_lib().convrot_mx_act_quant, "convrot_mx_act_quant", x.device, x.data_ptr(), _DTYPES[x.dtype], m, k,
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def mx_dequantize(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.float16) -> torch.Tensor:
    """The rows that codes and scales stand for, un-rotated, as dtype [rows, K]."""
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float16 or bfloat16")
    codes, scales, rows, k = _pair(codes, scales, "the")
    _same_device(codes, scales)
    out = codes.new_empty((rows, k), dtype=dtype)
    _call(_lib().convrot_mx_dequantize, "convrot_mx_dequantize", codes.device, codes.data_ptr(), scales.data_ptr(),
          rows, k, out.data_ptr(), _DTYPES[dtype])
    return out


def _product_args(m: int, n: int, like: torch.Tensor, bias, residual, dtype, out):
    """Checked bias, residual [m, n] and output [m, n] of a product."""
    if dtype not in _DTYPES:
        raise TypeError("out_dtype must be float16 or bfloat16")
    if bias is not None:
        bias = _ready(bias, torch.float32, "bias")
        if bias.shape != (n,):
            raise ValueError(f"bias must be [{n}], got {list(bias.shape)}")
    if out is None:
        y = like.new_empty((m, n), dtype=dtype)
    else:
        if out.dtype != dtype or not out.is_contiguous() or out.numel() != m * n or out.data_ptr() % 16:
            raise ValueError(f"out must be a contiguous {dtype} tensor of {m} x {n} elements, aligned to 16 bytes")
        y = out.view(m, n)
    res = None
    if residual is not None:
        if residual.dtype != dtype or residual.numel() != m * n or residual.shape[-1:] != (n,):
            raise ValueError(f"residual must be {dtype} [..., {n}] with {m} rows")
        if out is not None and residual.data_ptr() == out.data_ptr() and residual.is_contiguous():
            res = y   # in-place residual update
        else:
            res = _ready(residual, dtype, "residual")
    _same_device(like, bias, res, y)
    return bias, res, y


def _at(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def mx_gemm(q_x: torch.Tensor, s_x: torch.Tensor, q_w: torch.Tensor, s_w: torch.Tensor,
            bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
            out_dtype: torch.dtype = torch.float16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] = out_dtype(x w^T + bias + residual) of rows in 4 bits; ``out`` may be ``residual`` itself."""
    q_x, s_x, m, k = _pair(q_x, s_x, "x")
    q_w, s_w, n, kw = _pair(q_w, s_w, "w")
    if k != kw:
        raise ValueError(f"w has K={kw}, x has K={k}")
    _same_device(q_x, s_x, q_w, s_w)
    bias, res, y = _product_args(m, n, q_x, bias, residual, out_dtype, out)
    _call(_lib().convrot_mx_gemm, "convrot_mx_gemm", q_x.device, q_x.data_ptr(), s_x.data_ptr(), q_w.data_ptr(),
          s_w.data_ptr(), _at(bias), _at(res), m, n, k, y.data_ptr(), _DTYPES[out_dtype])
    return y if out is None else out


def mx_workspace_bytes(m: int, n: int, k: int) -> int:
    """Bytes of workspace that mx_linear needs for these sizes."""
    v = _lib().convrot_mx_workspace_bytes(m, n, k)
    if v == _BAD_SIZE:
        raise ValueError(f"invalid sizes for workspace: M={m} N={n} K={k}")
    return v


def mx_linear(x: torch.Tensor, q_w: torch.Tensor, s_w: torch.Tensor, bias: Optional[torch.Tensor] = None,
              residual: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The 4-bit linear: x fp16 or bf16 [..., K] -> out_dtype [..., N] (default
    x's), the activations rotated and quantised on the way; optional bias fp32
    [N] and residual [..., N] of out_dtype (``out`` may be ``residual`` itself)."""
    x2 = _rows16(x)
    q_w, s_w, n, kw = _pair(q_w, s_w, "w")
    m, k = x2.shape
    if k != kw:
        raise ValueError(f"w has K={kw}, x has K={k}")
    out_dtype = out_dtype or x2.dtype
    _same_device(x2, q_w, s_w, workspace)
    bias, res, y = _product_args(m, n, x2, bias, residual, out_dtype, out)
    if workspace is None:
        need = mx_workspace_bytes(m, n, k)
        if need:
            workspace = x2.new_empty(need, dtype=torch.uint8)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    _call(_lib().convrot_mx_linear, "convrot_mx_linear", x2.device, x2.data_ptr(), _DTYPES[x2.dtype], m, k,
          q_w.data_ptr(), s_w.data_ptr(), n, _at(bias), _at(res), y.data_ptr(), _DTYPES[out_dtype], _at(workspace),
          0 if workspace is None else workspace.numel())
    return out if out is not None else y if x.dim() == 2 else y.view(*x.shape[:-1], n)
