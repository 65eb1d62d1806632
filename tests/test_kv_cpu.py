"""The key/value cache without a GPU: its oracle against facts known by hand,
the exported symbols, and every refusal of the C entry points and the binding
(each call here returns from the host-side checks; no kernel runs)."""

import ctypes
import os
import re

import numpy as np
import pytest
import scipy.linalg
import torch

import rotation_quantized_int8_amd as cr
from oracle import kv_oracle as O
from rotation_quantized_int8_amd import build as crbuild
from rotation_quantized_int8_amd import kv

OK, INVALID, SHAPE, ALIGN, DEVICE, LAUNCH, WORKSPACE, TOO_LARGE = range(8)
HEADER = os.path.join(os.path.dirname(cr.HEADER_PATH), "convrot_kv.h")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(cr.LIB_PATH):
        crbuild.build()
    return kv._lib()


# ------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("d", [64, 128, 256])
def test_signs_are_sylvester(d):
    assert np.array_equal(O.signs(d), scipy.linalg.hadamard(d))


def test_quantize_one_hot_and_zero():
    x = np.zeros((2, 128))
    x[0, 5] = 3.0
    c, s = O.quantize(x, 4)
    assert np.array_equal(c[0], 7 * O.signs(128)[5]) and not c[1].any() and s[1] == 0
    assert s[0] == np.float32(np.float32(3) / np.float32(7)) * np.float32(1 / np.sqrt(128))
    # codes of one magnitude: the row comes back to within the two fp32 roundings of its scale
    assert np.allclose(O.rows(c, s)[0], x[0], rtol=2.0 ** -22, atol=2.0 ** -22)


@pytest.mark.parametrize("bits", [4, 8])
def test_quantize_error_bound_and_packing(bits):
    x = np.random.default_rng(bits).normal(size=(50, 64)).astype(np.float16)
    c, s = O.quantize(x, bits)
    assert np.abs(c).max() == O.qmax(bits)
    assert np.array_equal(O.unpack(O.pack(c, bits), bits), c)
    # half a step in each rotated element: sqrt(D) / 2 steps in the 2-norm
    err = np.linalg.norm(O.rows(c, s) - x, axis=-1)
    assert (err <= np.sqrt(64) * s * 0.5 * (1 + 1e-6)).all()
    assert np.allclose(O.read_f32(c, s), O.rows(c, s), rtol=2.0 ** -21, atol=0)


def test_quantize_non_finite_rows():
    x = np.ones((3, 64))
    x[0, 1], x[1, 1], x[1, 2] = np.nan, np.inf, -np.inf
    c, s = O.quantize(x, 8)
    assert np.isnan(s[:2]).all() and not c[:2].any() and np.isfinite(s[2])


def test_attention_oracle_by_hand():
    k = np.zeros((3, 1, 64))
    v = np.random.default_rng(1).normal(size=(3, 1, 64))
    q = np.ones((5, 2, 64))
    o, spread = O.attention(q, k, v, 1.0, True)        # equal scores: means over the visible rows
    assert not o[:2].any() and not spread[:2].any()    # 5 queries, 3 tokens: two see none
    assert np.allclose(o[2, 0], v[0, 0]) and np.allclose(o[3, 1], v[:2, 0].mean(0))
    assert np.allclose(o[4], v[:, 0].mean(0))
    k[1, 0, 0] = np.log(3.0)                           # one score log 3 above the others
    o, _ = O.attention(q[:1], k, v, 1.0, False)
    assert np.allclose(o[0, 0], (v[0, 0] + 3 * v[1, 0] + v[2, 0]) / 5)


# ------------------------------------------------------------------- refusals

def test_exports_every_declared_symbol(L):
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = set(re.findall(r"\b(convrot_kv_[a-z0-9_]+)\s*\(", text))
    assert declared == set(kv._KV_SIGNATURES)
    for name in declared:
        assert hasattr(L, name)


# fake, 16-byte aligned "device" addresses, far apart: never dereferenced
KC, KS, VC, VS, A, B, C, D, E, F, G = (i << 36 for i in range(1, 12))


def _cache(**over):
    f = dict(k_codes=KC, k_scale=KS, v_codes=VC, v_scale=VS, pages=8, page_size=16, heads=2, head_dim=128, bits=4)
    f.update(over)
    return kv._Cache(**f)


BAD_CACHES = [dict(pages=0), dict(pages=1 << 31), dict(page_size=8), dict(page_size=24), dict(page_size=512),
              dict(heads=0), dict(heads=65536), dict(head_dim=32), dict(head_dim=96), dict(bits=3), dict(bits=16)]


def test_append_refusals(L):
    def call(c=None, k=A, kt=256, kh=128, v=B, vt=256, vh=128, dtype=0, slots=C, T=3):
        c = _cache() if c is None else c
        return L.convrot_kv_append(ctypes.addressof(c), k, kt, kh, v, vt, vh, dtype, slots, T, None)

    assert L.convrot_kv_append(None, A, 256, 128, B, 256, 128, 0, C, 3, None) == INVALID
    for bad in BAD_CACHES:
        assert call(_cache(**bad)) == SHAPE, bad
    assert call(T=-1) == SHAPE and call(T=1 << 40) == SHAPE and call(T=1 << 31) == SHAPE
    assert call(dtype=2) == INVALID and call(dtype=-1) == INVALID
    assert call(T=0) == OK and call(T=0, k=None, v=None, slots=None) == OK
    assert call(kt=-256) == SHAPE and call(kh=4) == SHAPE and call(vt=1 << 40) == SHAPE and call(vh=-8) == SHAPE
    assert call(k=None) == INVALID and call(v=None) == INVALID and call(slots=None) == INVALID
    assert call(_cache(k_codes=None)) == INVALID and call(_cache(v_scale=None)) == INVALID
    assert call(k=A + 8) == ALIGN and call(v=B + 2) == ALIGN and call(slots=C + 8) == ALIGN
    assert call(_cache(v_codes=VC + 8)) == ALIGN and call(_cache(k_scale=KS + 4)) == ALIGN
    assert call(k=KC + 16) == INVALID and call(v=VS) == INVALID and call(slots=KS) == INVALID
    # the last row of strided keys reaches into the codes
    assert call(k=KC - 2 * 2 * 1024, kt=1024, T=3) == INVALID


def test_read_refusals(L):
    def call(c=None, slots=C, T=3, k=A, v=B, dtype=0):
        c = _cache() if c is None else c
        return L.convrot_kv_read(ctypes.addressof(c), slots, T, k, v, dtype, None)

    assert L.convrot_kv_read(None, C, 3, A, B, 0, None) == INVALID
    for bad in BAD_CACHES:
        assert call(_cache(**bad)) == SHAPE, bad
    assert call(T=-1) == SHAPE and call(T=1 << 31) == SHAPE and call(dtype=7) == INVALID
    assert call(T=0, slots=None, k=None, v=None) == OK
    assert call(slots=None) == INVALID and call(k=None, v=None) == INVALID and call(_cache(v_codes=None)) == INVALID
    assert call(k=A + 2) == ALIGN and call(v=B + 8) == ALIGN and call(slots=C + 8) == ALIGN
    assert call(k=A, v=A + 1024) == INVALID       # 3 tokens x 2 heads x 128: 1536 bytes each
    assert call(k=VC) == INVALID and call(v=KS + 16) == INVALID and call(slots=A + 16) == INVALID


def test_attention_refusals(L):
    def call(c=None, q=A, qt=512, qh=128, dtype=0, T=4, hq=4, table=B, width=3, batch=2, lens=C, start=D, max_q=3,
             max_kv=48, scale=1.0, causal=1, o=E, ws=F, nbytes=1 << 34):
        c = _cache() if c is None else c
        return L.convrot_kv_attention(ctypes.addressof(c), q, qt, qh, dtype, T, hq, table, width, batch, lens, start,
                                      max_q, max_kv, scale, causal, o, ws, nbytes, None)

    assert L.convrot_kv_attention(None, A, 512, 128, 0, 4, 4, B, 3, 2, C, D, 3, 48, 1.0, 1, E, F, 1 << 34,
                                  None) == INVALID
    for bad in BAD_CACHES:
        assert call(_cache(**bad)) == SHAPE, bad
    assert call(T=-1) == SHAPE and call(T=1 << 31) == SHAPE and call(batch=-1) == SHAPE and call(batch=65536) == SHAPE
    assert call(hq=0) == SHAPE and call(hq=3) == SHAPE and call(hq=65536) == SHAPE
    assert call(max_q=-1) == SHAPE and call(max_kv=-1) == SHAPE and call(max_kv=49) == SHAPE
    assert call(max_kv=(1 << 31) - 1, width=1 << 30) == SHAPE and call(width=-1) == SHAPE
    assert call(max_q=(1 << 31) - 1) == SHAPE        # times the group of 2
    assert call(dtype=2) == INVALID
    assert call(T=0, q=None, o=None) == OK and call(batch=0, table=None, lens=None) == OK and call(max_q=0) == OK
    assert call(start=None, T=5) == SHAPE            # not a multiple of the batch
    assert call(start=None, max_q=1) == SHAPE        # two queries each
    assert call(qt=-8) == SHAPE and call(qh=100) == SHAPE
    assert call(q=None) == INVALID and call(o=None) == INVALID and call(lens=None) == INVALID
    assert call(table=None) == INVALID and call(_cache(k_codes=None)) == INVALID
    for name, at in (("q", A), ("table", B), ("lens", C), ("start", D), ("o", E), ("ws", F)):
        assert call(**{name: at + 8}) == ALIGN, name
    assert call(o=A) == INVALID and call(o=KC) == INVALID and call(o=B) == INVALID and call(o=C) == INVALID
    assert call(o=D) == INVALID
    small = _cache()
    assert L.convrot_kv_workspace_bytes(ctypes.addressof(small), 4, 4, 2, 3, 48) != kv._BAD_SIZE
    big = _cache(pages=1 << 14)                      # one query over 131072 tokens: split, so it needs a workspace
    need = L.convrot_kv_workspace_bytes(ctypes.addressof(big), 1, 2, 1, 1, 131072)
    long = dict(c=big, T=1, hq=2, qt=256, batch=1, width=1 << 13, max_q=1, max_kv=131072)
    if need:
        assert call(**long, ws=None) == WORKSPACE and call(**long, nbytes=need - 1) == WORKSPACE
        for at in (A, B, C, D, E, KC, VS):
            assert call(**long, ws=at) == INVALID


def test_workspace_refusals(L):
    f = L.convrot_kv_workspace_bytes
    c = _cache()
    p = ctypes.addressof(c)
    assert f(None, 4, 4, 2, 3, 48) == kv._BAD_SIZE
    for bad in BAD_CACHES:
        b = _cache(**bad)
        assert f(ctypes.addressof(b), 4, 4, 2, 3, 48) == kv._BAD_SIZE, bad
    for args in ((-1, 4, 2, 3, 48), (4, 3, 2, 3, 48), (4, 4, -1, 3, 48), (4, 4, 2, -1, 48), (4, 4, 2, 3, -1)):
        assert f(p, *args) == kv._BAD_SIZE, args
    assert f(p, 0, 4, 2, 3, 48) == 0 and f(p, 4, 4, 0, 3, 48) == 0 and f(p, 4, 4, 2, 0, 48) == 0


def test_binding_refuses_before_the_library():
    codes, scale = torch.zeros((2, 1, 16, 64), dtype=torch.uint8), torch.zeros((2, 1, 16))
    with pytest.raises(ValueError, match="GPU"):
        cr.KVCache(codes, scale, codes, scale)
    with pytest.raises(TypeError):
        cr.KVCache(codes.float(), scale, codes, scale)
    with pytest.raises(TypeError):
        cr.KVCache(codes, scale.double(), codes, scale)
    with pytest.raises(ValueError, match="codes must be"):
        cr.KVCache(codes, scale[:1], codes, scale)
    for bad in (dict(bits=5), dict(head_dim=100), dict(page_size=48), dict(pages=0)):
        with pytest.raises(ValueError):
            cr.KVCache.empty(**{**dict(pages=2, page_size=16, heads=1, head_dim=128, device="cpu"), **bad})


def test_attention_refuses_queries_that_no_sequence_has(L):
    """Without q_start every query belongs to a sequence: no batch, or no room for its queries, is no empty call."""
    c = _cache()

    def call(T, batch, max_q, start=None):
        return L.convrot_kv_attention(ctypes.addressof(c), A, 512, 128, 0, T, 4, B, 3, batch, C, start, max_q, 48, 1.0, 1, E,
                                      F, 1 << 34, None)

    assert call(4, 0, 3) == SHAPE and call(4, 0, 0) == SHAPE
    assert call(4, 2, 0) == SHAPE and call(4, 2, 1) == SHAPE and call(5, 2, 3) == SHAPE
    assert call(0, 0, 0) == OK and call(0, 2, 3) == OK
    assert call(4, 0, 3, D) == OK and call(4, 2, 0, D) == OK     # with q_start these are rows of no sequence


def test_rows_are_copied_where_the_library_does_not_take_their_strides():
    """Strides of 2^31 elements and more, no multiples of 8, or an odd address: the binding hands on a copy."""
    class At:
        device, head_dim = torch.device("cpu"), 64

    x = torch.arange(3 * 2 * 64, dtype=torch.float16).view(3, 2, 64)
    assert kv._rows(x, At, 2, "x") == (x, 128, 64)
    kept, token, head = kv._rows(x[:1, :1].expand(3, 2, 64), At, 2, "x")
    assert (token, head) == (0, 0)
    one = x[:1, :1]
    for strides in ((1 << 31, 64, 1), (128, 1 << 31, 1), (1 << 40, 1 << 35, 1), (12, 64, 1), (128, 4, 1)):
        odd = torch.as_strided(one, (1, 1, 64), strides)
        copy, token, head = kv._rows(odd, At, 1, "x")
        assert torch.equal(copy, one) and copy.data_ptr() != one.data_ptr()
        assert 0 <= token <= 0x7FFFFFFF and 0 <= head <= 0x7FFFFFFF and token % 8 == head % 8 == 0
    for odd in (torch.arange(385, dtype=torch.float16)[1:].view(3, 2, 64), x.transpose(0, 2).contiguous().transpose(0, 2)):
        copy, token, head = kv._rows(odd, At, 2, "x")
        assert torch.equal(copy, odd) and copy.stride(2) == 1 and copy.data_ptr() % 16 == 0
