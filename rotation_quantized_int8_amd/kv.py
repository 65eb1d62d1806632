"""The rotated, quantised key/value cache: Python binding of include/convrot_kv.h.

  cache = KVCache.empty(pages, page_size, heads, head_dim, bits=4, device="cuda")
  kv_append(cache, k, v, slots)                      # quantise new tokens into their slots
  k, v = kv_read(cache, slots)                       # the rows of slots, un-rotated
  o = kv_attention(cache, q, table, kv_lens)         # attention over the cached rows

As in the rest of the package only arguments are marshalled here; every step
runs in the library's HIP kernels on the current stream.
"""

from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import _DTYPES, _check, _f32, _i64, _sz, _vp
from . import lib as _base_lib

_int = ctypes.c_int


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("k_scale", _vp), ("v_codes", _vp), ("v_scale", _vp),
                ("pages", _i64), ("page_size", _i64), ("heads", _i64), ("head_dim", _i64), ("bits", _int)]


_KV_SIGNATURES = {
    "convrot_kv_append": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _int, _vp, _i64, _vp]),
    "convrot_kv_read": (_int, [_vp, _vp, _i64, _vp, _vp, _int, _vp]),
    "convrot_kv_workspace_bytes": (_sz, [_vp, _i64, _i64, _i64, _i64, _i64]),
    "convrot_kv_attention": (_int, [_vp, _vp, _i64, _i64, _int, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _i64,
                                    _f32, _int, _vp, _vp, _sz, _vp]),
}

_BAD_SIZE = ctypes.c_size_t(-1).value
_kv_lib: Optional[ctypes.CDLL] = None


def _lib() -> ctypes.CDLL:
    global _kv_lib
    if _kv_lib is None:
        handle = _base_lib()
        for name, (res, args) in _KV_SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _kv_lib = handle
    return _kv_lib


class KVCache:
    """A paged cache of rotated, quantised keys and values, over four tensors:
    codes [pages, heads, page_size, head_dim / 2] uint8 (4 bits, two a byte)
    or [pages, heads, page_size, head_dim] int8 (8 bits), and scales fp32
    [pages, heads, page_size].  The tensors are the cache: they are kept, not
    copied, and may be saved, moved or shared as such."""

    __slots__ = ("k_codes", "k_scale", "v_codes", "v_scale", "pages", "page_size", "heads", "head_dim", "bits",
                 "device", "_struct", "_ref")

    def __init__(self, k_codes: torch.Tensor, k_scale: torch.Tensor, v_codes: torch.Tensor, v_scale: torch.Tensor):
        kind, shape, index = k_codes.dtype, k_codes.shape, k_codes.get_device()
        if kind not in (torch.uint8, torch.int8) or v_codes.dtype != kind:
            raise TypeError("codes must both be uint8 (4 bits, two a byte) or both int8 (8 bits)")
        if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
            raise TypeError("scales must be float32")
        if len(shape) != 4 or v_codes.shape != shape or k_scale.shape != shape[:3] or v_scale.shape != k_scale.shape:
            raise ValueError("codes must be [pages, heads, page_size, bytes] and scales [pages, heads, page_size]")
        tensors = (k_codes, k_scale, v_codes, v_scale)
        at = [t.data_ptr() for t in tensors]
        for t in tensors:
            if index < 0 or t.get_device() != index:
                raise ValueError("the cache's tensors must be on one GPU (no CPU path exists)")
            if not t.is_contiguous():
                raise ValueError("the cache's tensors must be contiguous and aligned to 16 bytes")
        if (at[0] | at[1] | at[2] | at[3]) % 16:
            raise ValueError("the cache's tensors must be contiguous and aligned to 16 bytes")
        self.device = k_codes.device
        self.k_codes, self.k_scale, self.v_codes, self.v_scale = k_codes, k_scale, v_codes, v_scale
        self.pages, self.heads, self.page_size, row = shape
        self.bits = 4 if kind == torch.uint8 else 8
        self.head_dim = row * 2 if self.bits == 4 else row
        self._struct = _Cache(*at, self.pages, self.page_size, self.heads, self.head_dim, self.bits)
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, head_dim: int, bits: int = 4,
              device="cuda") -> "KVCache":
        """A cache of zeros (every slot a row of zeros)."""
        if bits not in (4, 8):
            raise ValueError("bits must be 4 or 8")
        row, kind = (head_dim // 2, torch.uint8) if bits == 4 else (head_dim, torch.int8)
        if head_dim not in (64, 128, 256) or page_size not in (16, 32, 64, 128, 256) or pages < 1 or heads < 1:
            raise ValueError("head_dim must be 64, 128 or 256, page_size a power of two from 16 to 256, "
                             "and pages and heads at least 1")
        shape = (pages, heads, page_size)
        return cls(torch.zeros((*shape, row), dtype=kind, device=device),
                   torch.zeros(shape, dtype=torch.float32, device=device),
                   torch.zeros((*shape, row), dtype=kind, device=device),
                   torch.zeros(shape, dtype=torch.float32, device=device))


# The current stream's handle by device number; torch.cuda.current_stream(dev)
# builds a Python object around it (2.8 us of a call's 9, against 0.1).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(fn, name: str, device: torch.device, *args) -> None:
    """fn(*args, stream) with the device current, on its current stream."""
    index = device.index
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _check(status, name)


def _rows(t: torch.Tensor, cache: KVCache, heads: Optional[int], name: str) -> Tuple[torch.Tensor, int, int]:
    """t as [tokens, heads, head_dim] with the strides the library takes, and these strides."""
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    if t.device != cache.device:
        raise ValueError(f"{name} must be on the cache's GPU ({cache.device})")
    if t.dim() != 3 or t.shape[2] != cache.head_dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {cache.head_dim}], "
                         f"got {list(t.shape)}")
    token, head, last = t.stride()
    if last != 1 or (token | head) & ~0x7FFFFFF8 or t.data_ptr() % 16:   # multiples of 8 below 2^31
        t = torch.empty(t.shape, dtype=t.dtype, device=t.device).copy_(t)
        token, head, last = t.stride()
    return t, token, head


def _ints(t: torch.Tensor, dtype: torch.dtype, cache: KVCache, name: str) -> torch.Tensor:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != cache.device:
        raise ValueError(f"{name} must be on the cache's GPU ({cache.device})")
    if not t.is_contiguous():
        t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantises k and v, fp16 or bf16 [tokens, heads, head_dim] (any strides;
    slices of a fused projection are read in place), into their slots int64
    [tokens] (page * page_size + offset).  A slot out of range drops its token."""
    k, k_token, k_head = _rows(k, cache, cache.heads, "k")
    v, v_token, v_head = _rows(v, cache, cache.heads, "v")
    slots = _ints(slots, torch.int64, cache, "slots")
    if v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("k and v must have one shape and dtype")
    if slots.shape != k.shape[:1]:
        raise ValueError(f"slots must be [{k.shape[0]}], got {list(slots.shape)}")
    _call(_lib().convrot_kv_append, "convrot_kv_append", cache.device, cache._ref, k.data_ptr(), k_token, k_head,
          v.data_ptr(), v_token, v_head, _DTYPES[k.dtype], slots.data_ptr(), k.shape[0])


def kv_read(cache: KVCache, slots: torch.Tensor, dtype: torch.dtype = torch.float16,
            out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The keys and values of slots int64 [tokens], un-rotated, as dtype
    [tokens, heads, head_dim] (into ``out``, two contiguous tensors, where
    given).  A slot out of range gives zeros."""
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float16 or bfloat16")
    slots = _ints(slots, torch.int64, cache, "slots")
    if slots.dim() != 1:
        raise ValueError("slots must be one-dimensional")
    shape = (slots.shape[0], cache.heads, cache.head_dim)
    if out is None:
        k = slots.new_empty(shape, dtype=dtype)
        v = torch.empty_like(k)
    else:
        k, v = out
        for t in (k, v):
            if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != cache.device:
                raise ValueError(f"out must be two contiguous {dtype} tensors {list(shape)} on {cache.device}")
    _call(_lib().convrot_kv_read, "convrot_kv_read", cache.device, cache._ref, slots.data_ptr(), shape[0],
          k.data_ptr(), v.data_ptr(), _DTYPES[dtype])
    return k, v


def kv_workspace_bytes(cache: KVCache, tokens: int, q_heads: int, batch: int, max_q: int, max_kv: int) -> int:
    """Bytes of workspace that kv_attention needs for these sizes."""
    v = _lib().convrot_kv_workspace_bytes(cache._ref, tokens, q_heads, batch, max_q, max_kv)
    if v == _BAD_SIZE:
        raise ValueError(f"invalid sizes: tokens={tokens} q_heads={q_heads} batch={batch} max_q={max_q} "
                         f"max_kv={max_kv}")
    return v


def kv_attention(cache: KVCache, q: torch.Tensor, table: torch.Tensor, kv_lens: torch.Tensor,
                 q_start: Optional[torch.Tensor] = None, max_q: Optional[int] = None,
                 max_kv: Optional[int] = None, scale: Optional[float] = None, causal: bool = True,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of q, fp16 or bf16 [tokens, q_heads, head_dim], over the cached
    rows of each sequence; returns [tokens, q_heads, head_dim] of q's dtype.

    table int32 [batch, width] holds each sequence's pages in order, kv_lens
    int32 [batch] its cached tokens, q_start int32 [batch + 1] the first row
    of each sequence's queries (None: tokens / batch queries each); rows of no
    sequence, or past its first max_q, are not written.  max_q and max_kv bound
    the queries and the cached tokens of a sequence; tight values make the call
    faster (defaults: all tokens, and the table's width).  With
    ``causal`` the queries are each sequence's last tokens; without it every
    query sees every token (cross attention).  A query that sees no token
    gives zeros.  scale defaults to head_dim ** -0.5."""
    q, q_token, q_head = _rows(q, cache, None, "q")
    tokens, q_heads, _ = q.shape
    table = _ints(table, torch.int32, cache, "table")
    kv_lens = _ints(kv_lens, torch.int32, cache, "kv_lens")
    if table.dim() != 2 or kv_lens.shape != table.shape[:1]:
        raise ValueError("table must be [batch, width] and kv_lens [batch]")
    batch, width = table.shape
    if q_start is not None:
        q_start = _ints(q_start, torch.int32, cache, "q_start")
        if q_start.shape != (batch + 1,):
            raise ValueError(f"q_start must be [{batch + 1}], got {list(q_start.shape)}")
        if max_q is None:
            max_q = tokens
    elif max_q is None:
        max_q = -(-tokens // batch) if batch else 0
    if max_kv is None:
        max_kv = width * cache.page_size
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif out.dtype != q.dtype or out.shape != q.shape or not out.is_contiguous() or out.device != q.device:
        raise ValueError("out must be a contiguous tensor of q's shape, dtype and device")
    need = kv_workspace_bytes(cache, tokens, q_heads, batch, max_q, max_kv)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != q.device:
        raise TypeError("workspace must be a contiguous uint8 tensor on q's device")
    _call(_lib().convrot_kv_attention, "convrot_kv_attention", cache.device, cache._ref, q.data_ptr(), q_token,
          q_head, _DTYPES[q.dtype], tokens, q_heads, table.data_ptr(), width, batch, kv_lens.data_ptr(),
          None if q_start is None else q_start.data_ptr(), max_q, max_kv,
          1.0 / math.sqrt(cache.head_dim) if scale is None else scale, 1 if causal else 0, out.data_ptr(),
          None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel())
    return out
