"""The 4-bit linear without a GPU: its oracle against facts known by hand, the
exported symbols, and every refusal of the C entry points and the binding (each
call here returns from the host-side checks; no kernel runs)."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import rotation_quantized_int8_amd as cr
from oracle import convrot_oracle as base
from oracle import mx_oracle as O
from rotation_quantized_int8_amd import build as crbuild
from rotation_quantized_int8_amd import mx

OK, INVALID, SHAPE, ALIGN, DEVICE, LAUNCH, WORKSPACE, TOO_LARGE = range(8)
HEADER = os.path.join(os.path.dirname(cr.HEADER_PATH), "convrot_mx.h")
A, B, C, D, E, F, G, H = (i << 40 for i in range(1, 9))   # fake aligned addresses, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(cr.LIB_PATH):
        crbuild.build()
    return mx._lib()


# ------------------------------------------------------------------ the oracle

def test_encode_by_hand():
    v = np.array([0, .25, .26, .5, .75, .74, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5, 5.01, 6, 7.9, -.25, -.3, -5, -9])
    want = [0, 0, .5, .5, 1, .5, 1, 1.5, 2, 2, 3, 4, 4, 6, 6, 6, 0, -.5, -4, -6]
    assert O.decode(O.encode(v)).tolist() == want
    assert O.encode(np.array([0.0, 6.0, -0.5, -6.0])).tolist() == [0, 7, 9, 15]


def test_encode_is_the_nearest_value():
    v = np.random.default_rng(0).uniform(-7, 7, 20000)
    grid = np.concatenate([O.GRID, -O.GRID])
    assert np.array_equal(O.decode(O.encode(v)), grid[np.abs(v[:, None] - grid).argmin(1)])


def test_exponent_by_hand():
    top = np.array([0, 1, 1.99, 2, 4, 7.99, 8, 2.0 ** -124, 2.0 ** -125, 2.0 ** -140, 3e38, np.nextafter(1, 0)])
    assert O.exponent(top).tolist() == [-127, -2, -2, -1, 0, 0, 1, -126, -127, -127, 125, -3]


def test_quantize_error_and_packing():
    u = np.random.default_rng(1).normal(size=(9, 512)).astype(np.float32)
    c, s = O.quantize(u)
    q, t = O.pack(c, s)
    assert q.shape == (9, 256) and t.shape == (2, 9, 8)
    assert all(np.array_equal(a, b) for a, b in zip(O.unpack(q, t), (c, s)))
    assert t[1, 4, 3] == s[4, 11] and q[2, 5] == c[2, 10] + 16 * c[2, 11]
    # half the coarsest step within 6, and at most 2 of the scale past it
    e = np.repeat(2.0 ** (s - 127.0), 32, 1)
    a = np.abs(u) / e
    assert (np.abs(O.values(c, s) - u) <= e * np.where(a <= 2, .25, np.where(a <= 4, .5, np.where(a <= 6, 1, 2)))).all()


def test_quantize_not_finite_and_zero():
    u = np.ones((3, 256), dtype=np.float32)
    u[0, 5], u[1, 40], u[2] = np.nan, -np.inf, 0
    c, s = O.quantize(u)
    assert s[0, 0] == 255 and s[1, 1] == 255 and (s == 255).sum() == 2 and (s[2] == 0).all()
    assert not c[0, :32].any() and not c[1, 32:64].any() and not c[2].any()


def test_rotation_and_dequantize():
    x = np.random.default_rng(2).normal(size=(3, 512)).astype(np.float16)
    assert np.array_equal(O.rotate_f32(x), base.rotate_activations_f32(x))
    assert not np.signbit(O.rotate_f32(np.full((1, 256), -0.0))).any()
    row = base.hadamard256()[3] * 16                              # +-1, whose un-rotation is one-hot
    c, s = O.quantize(row[None].astype(np.float32))
    assert np.array_equal(O.dequantize(c, s)[0], 16 * np.eye(256)[3])


def test_product_by_hand():
    x, w = np.array([[1.0, -2.0]]), np.array([[3.0, 0.5], [0.0, 4.0]])
    y, t = O.product(x, w, bias=np.array([1.0, -1.0]), residual=np.array([[0.5, 0.25]]))
    assert y.tolist() == [[3.5, -8.75]] and t.tolist() == [[5.5, 9.25]]


# ------------------------------------------------------------------- refusals

def test_exports_every_declared_symbol(L):
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = set(re.findall(r"\b(convrot_mx_[a-z0-9_]+)\s*\(", text))
    assert declared == set(mx._MX_SIGNATURES)
    for name in declared:
        assert hasattr(L, name)


BAD_ROWS = [(-1, 256), (3, 255), (3, -256), (3, 131072 + 256), ((1 << 24) + 1, 256), (1 << 24, 4096)]


@pytest.mark.parametrize("name", ["weights", "act", "dequantize"])
def test_rows_refusals(L, name):
    def call(v=A, rows=3, k=256, codes=B, scales=C, dtype=0):
        if name == "weights":
            return L.convrot_mx_quantize_weights(v, rows, k, codes, scales, None)
        if name == "act":
            return L.convrot_mx_act_quant(v, dtype, rows, k, codes, scales, None)
        return L.convrot_mx_dequantize(codes, scales, rows, k, v, dtype, None)

    for rows, k in BAD_ROWS:
        assert call(rows=rows, k=k) == SHAPE, (rows, k)
    if name != "weights":
        assert call(dtype=2) == INVALID and call(dtype=-1) == INVALID
    assert call(rows=0, v=None, codes=None, scales=None) == OK and call(k=0, v=None, codes=None, scales=None) == OK
    for arg in ("v", "codes", "scales"):
        assert call(**{arg: None}) == INVALID
        assert call(**{arg: A + 8}) == ALIGN
    assert call(codes=A) == INVALID and call(scales=A + 16) == INVALID and call(scales=B + 3 * 128 - 16) == INVALID


def test_gemm_refusals(L):
    def call(x=A, xs=B, w=C, ws=D, bias=E, res=F, m=4, n=5, k=256, y=G, dtype=0):
        return L.convrot_mx_gemm(x, xs, w, ws, bias, res, m, n, k, y, dtype, None)

    for rows, k in BAD_ROWS:
        assert call(m=rows, k=k) == SHAPE and call(n=rows, k=k) == SHAPE
    assert call(m=1 << 20, n=1 << 20) == SHAPE
    assert call(dtype=2) == INVALID
    assert call(m=0, x=None, y=None) == OK and call(n=0, w=None, y=None) == OK
    for arg in ("x", "xs", "w", "ws", "y"):
        assert call(**{arg: None}) == INVALID, arg
    assert call(k=0, x=None, xs=None, w=None, ws=None, y=None) == INVALID
    for arg, at in (("x", A), ("xs", B), ("w", C), ("ws", D), ("bias", E), ("res", F), ("y", G)):
        assert call(**{arg: at + 8}) == ALIGN, arg
    for at in (A, B, C, D, E):
        assert call(y=at) == INVALID
    assert call(res=G + 16) == INVALID            # part of the output


def test_linear_refusals(L):
    need = 40 * 128 + 512                         # codes, and 320 bytes of scales, in pieces of 256
    assert L.convrot_mx_workspace_bytes(40, 5, 256) == need
    assert L.convrot_mx_workspace_bytes(4, 5, 256) == 0          # few short rows: one launch

    def call(x=A, xd=0, m=40, k=256, w=C, ws=D, n=5, bias=E, res=F, y=G, yd=1, work=H, nbytes=need):
        return L.convrot_mx_linear(x, xd, m, k, w, ws, n, bias, res, y, yd, work, nbytes, None)

    for rows, k in BAD_ROWS:
        assert call(m=rows, k=k) == SHAPE and call(n=rows, k=k) == SHAPE
        assert L.convrot_mx_workspace_bytes(rows, 5, k) == mx._BAD_SIZE
    assert call(xd=2) == INVALID and call(yd=3) == INVALID
    assert call(m=0, x=None, work=None, nbytes=0) == OK and call(n=0, y=None, work=None, nbytes=0) == OK
    for arg in ("x", "w", "ws", "y"):
        assert call(**{arg: None}) == INVALID, arg
    for arg, at in (("x", A), ("w", C), ("ws", D), ("bias", E), ("res", F), ("y", G), ("work", H)):
        assert call(**{arg: at + 8}) == ALIGN, arg
    assert call(work=None) == WORKSPACE and call(nbytes=need - 1) == WORKSPACE
    for at in (A, C, D, E):
        assert call(y=at) == INVALID
    for at in (A, C, D, E, F, G):
        assert call(work=at) == INVALID
    assert call(res=G + 16) == INVALID
    assert L.convrot_mx_workspace_bytes(0, 5, 256) == 0 and L.convrot_mx_workspace_bytes(40, 5, 0) == 0


def test_binding_refuses_before_the_library():
    x, q, s = torch.zeros((2, 256)), torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((1, 4, 8), dtype=torch.uint8)
    with pytest.raises(TypeError):
        cr.mx_act_quant(x)                        # fp32
    with pytest.raises(TypeError):
        cr.mx_quantize_weights(x.half())
    with pytest.raises(TypeError):
        cr.mx_dequantize(q, s, torch.float32)
    with pytest.raises(TypeError):
        cr.mx_gemm(q.char(), s, q, s)
    for call in (lambda: cr.mx_act_quant(x.half()), lambda: cr.mx_quantize_weights(x), lambda: cr.mx_dequantize(q, s),
                 lambda: cr.mx_gemm(q, s, q, s), lambda: cr.mx_linear(x.half(), q, s)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="multiple"):
        mx._empty4(2, 300, x)
    with pytest.raises(ValueError, match="sizes"):
        cr.mx_workspace_bytes(4, 5, 100)
