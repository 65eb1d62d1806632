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

from . import GROUP, _DTYPES, _flatten, _i64, _prep, _prep16, _sz, _vp
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


def _empty4(rows: int, k: int, device) -> Tuple[torch.Tensor, torch.Tensor]:
    """Uninitialised codes and scales."""
    if k % GROUP:
        raise ValueError(f"the row length must be a multiple of {GROUP}, got {k}")
    return (torch.empty((rows, k // 2), dtype=torch.uint8, device=device),
            torch.empty((k // GROUP, rows, 8), dtype=torch.uint8, device=device))


def _pair(codes: torch.Tensor, scales: torch.Tensor, name: str) -> Tuple[torch.Tensor, torch.Tensor, int, int]:
    """Checked codes and scales, their rows and row length."""
    codes, scales = _prep(codes, torch.uint8, f"{name} codes"), _prep(scales, torch.uint8, f"{name} scales")
    if codes.dim() != 2 or codes.shape[1] % (GROUP // 2):
        raise ValueError(f"{name} codes must be [rows, K / 2] with K a multiple of {GROUP}, got {list(codes.shape)}")
    rows, k = codes.shape[0], codes.shape[1] * 2
    if scales.shape != (k // GROUP, rows, 8):
        raise ValueError(f"{name} scales must be {[k // GROUP, rows, 8]}, got {list(scales.shape)}")
    return codes, scales, rows, k


def _same_device(device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")


def mx_quantize_weights(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Offline: w fp32 [N, K] -> (codes uint8 [N, K / 2], scales uint8 [K / 256, N, 8])."""
    w = _prep(w, torch.float32, "W")
    if w.dim() != 2:
        raise ValueError("W must be [N, K]")
    n, k = w.shape
    codes, scales = _empty4(n, k, w.device)
    _call(_lib().convrot_mx_quantize_weights, "convrot_mx_quantize_weights", w.device, w.data_ptr(), n, k,
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def mx_act_quant(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """x fp16 or bf16 [..., K], M rows -> (codes uint8 [M, K / 2], scales uint8 [K / 256, M, 8])."""
    x, _ = _flatten(_prep16(x, "x"))
    m, k = x.shape
    codes, scales = _empty4(m, k, x.device)
    _call(_lib().convrot_mx_act_quant, "convrot_mx_act_quant", x.device, x.data_ptr(), _DTYPES[x.dtype], m, k,
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def mx_dequantize(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.float16) -> torch.Tensor:
    """The rows that codes and scales stand for, un-rotated, as dtype [rows, K]."""
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float16 or bfloat16")
    codes, scales, rows, k = _pair(codes, scales, "the")
    _same_device(codes.device, scales=scales)
    out = torch.empty((rows, k), dtype=dtype, device=codes.device)
    _call(_lib().convrot_mx_dequantize, "convrot_mx_dequantize", codes.device, codes.data_ptr(), scales.data_ptr(),
          rows, k, out.data_ptr(), _DTYPES[dtype])
    return out


def _product_args(m: int, n: int, device, bias, residual, dtype, out):
    """Checked bias, residual [m, n] and output [m, n] of a product."""
    if dtype not in _DTYPES:
        raise TypeError("out_dtype must be float16 or bfloat16")
    if bias is not None:
        bias = _prep(bias, torch.float32, "bias")
        if bias.shape != (n,):
            raise ValueError(f"bias must be [{n}], got {list(bias.shape)}")
    if out is None:
        y = torch.empty((m, n), dtype=dtype, device=device)
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
            res = _prep(residual, dtype, "residual").view(m, n)
    _same_device(device, bias=bias, residual=res, out=y)
    return bias, res, y


def mx_gemm(q_x: torch.Tensor, s_x: torch.Tensor, q_w: torch.Tensor, s_w: torch.Tensor,
            bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
            out_dtype: torch.dtype = torch.float16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] = out_dtype(x w^T + bias + residual) of rows in 4 bits; ``out`` may be ``residual`` itself."""
    q_x, s_x, m, k = _pair(q_x, s_x, "x")
    q_w, s_w, n, kw = _pair(q_w, s_w, "w")
    if k != kw:
        raise ValueError(f"w has K={kw}, x has K={k}")
    _same_device(q_x.device, x_scales=s_x, w_codes=q_w, w_scales=s_w)
    bias, res, y = _product_args(m, n, q_x.device, bias, residual, out_dtype, out)
    _call(_lib().convrot_mx_gemm, "convrot_mx_gemm", q_x.device, q_x.data_ptr(), s_x.data_ptr(), q_w.data_ptr(),
          s_w.data_ptr(), None if bias is None else bias.data_ptr(), None if res is None else res.data_ptr(), m, n, k,
          y.data_ptr(), _DTYPES[out_dtype])
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
    x2, lead = _flatten(_prep16(x, "x"))
    q_w, s_w, n, kw = _pair(q_w, s_w, "w")
    m, k = x2.shape
    if k != kw:
        raise ValueError(f"w has K={kw}, x has K={k}")
    out_dtype = out_dtype or x2.dtype
    _same_device(x2.device, w_codes=q_w, w_scales=s_w, workspace=workspace)
    bias, res, y = _product_args(m, n, x2.device, bias, residual, out_dtype, out)
    if workspace is None:
        need = mx_workspace_bytes(m, n, k)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x2.device)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    _call(_lib().convrot_mx_linear, "convrot_mx_linear", x2.device, x2.data_ptr(), _DTYPES[x2.dtype], m, k,
          q_w.data_ptr(), s_w.data_ptr(), n, None if bias is None else bias.data_ptr(),
          None if res is None else res.data_ptr(), y.data_ptr(), _DTYPES[out_dtype], workspace.data_ptr(),
          workspace.numel())
    return out if out is not None else y.view(*lead, n)
