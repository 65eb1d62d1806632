"""The norms around the linears without a GPU: their oracle against facts known
by hand, the exported symbols, and every refusal of the C entry points and the
binding (each call here returns from the host-side checks; no kernel runs)."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import rotation_quantized_int8_amd as cr
from oracle import norm_oracle as O
from rotation_quantized_int8_amd import build as crbuild
from rotation_quantized_int8_amd import norms

OK, INVALID, SHAPE, ALIGN, DEVICE, LAUNCH, WORKSPACE, TOO_LARGE = range(8)
HEADER = os.path.join(os.path.dirname(cr.HEADER_PATH), "convrot_norm.h")
A, B, C, D, E, F, G, H, I, J, K = (i << 40 for i in range(1, 12))   # fake aligned addresses, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(cr.LIB_PATH):
        crbuild.build()
    return norms._lib()


# ------------------------------------------------------------------ the oracle

def test_norm_by_hand():
    v = np.array([[1.0, 3.0], [2.0, 2.0], [-4.0, 4.0]])
    assert np.allclose(O.norm(v, "layer", 0.0)[[0, 2]], [[-1, 1], [-1, 1]])
    assert np.array_equal(O.norm(v, "layer", 1e-6)[1], [0, 0])
    assert np.allclose(O.norm(v, "rms", 0.0), [[1 / 5 ** .5, 3 / 5 ** .5], [1, 1], [-1, 1]])
    assert np.allclose(O.norm(v, "rms", 9.0, np.array([2.0, 1.0]), np.array([0.5, 0.0]))[2], [-8 / 5 + .5, 4 / 5])
    assert np.array_equal(O.modulate(np.array([[1.0, 2.0]]), np.array([[1.0, -1.0]]), np.array([[0.0, 3.0]])), [[2, 3]])


def test_norm_is_torchs():
    g = torch.Generator().manual_seed(0)
    x, w, b = torch.randn((5, 77), generator=g, dtype=torch.float64), *torch.randn((2, 77), generator=g).double()
    assert np.allclose(O.norm(x.numpy(), "layer", 1e-5, w.numpy(), b.numpy()),
                       torch.nn.functional.layer_norm(x, (77,), w, b, 1e-5).numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(O.norm(x.numpy(), "rms", 1e-5, w.numpy()),
                       torch.nn.functional.rms_norm(x, (77,), w, 1e-5).numpy(), rtol=1e-12, atol=1e-12)


def test_residual_by_hand():
    x, y = np.array([[1.0, 2.0]]), np.array([[3.0, -3.0]])
    assert O.residual(x, y, 0.5).tolist() == [[3.5, -2.0]]
    h = O.residual(x, y, 1.0, np.array([[2.0, 1.0]]), ("rms", 0.0, np.array([1.0, 10.0]), None))
    assert np.allclose(h, [[3.0, -8.0]])


def test_quantize_int8_rows():
    n = np.zeros((3, 256))
    n[0, 0], n[2, 7] = 16.0, np.inf
    q, s = O.quantize_int8(n)
    assert (q[0] == 127).all() and s[0] == np.float32(1) / np.float32(127) and s[1] == 0 and np.isnan(s[2])
    assert not q[1:].any()


# ------------------------------------------------------------------- refusals

def test_exports_every_declared_symbol(L):
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = set(re.findall(r"\bconvrot_status (convrot_[a-z0-9_]+)\s*\(", text))
    assert declared == set(norms._NORM_SIGNATURES)
    for name in declared:
        assert hasattr(L, name)


def _desc(kind=2, eps=1e-6, weight=C, bias=D):
    return norms._DESC.pack(kind, eps, weight or 0, bias or 0)


def _mod(scale=E, shift=F, gate=G, ss=512, hs=512, gs=512, dtype=0, rows=2, index=None):
    return norms._MOD.pack(scale or 0, shift or 0, gate or 0, ss, hs, gs, dtype, rows, index or 0)


def _out(kind=0, values=H, scales=I):
    return norms._OUT.pack(kind, values or 0, scales or 0)


def _call(L, residual, x=A, xs=512, y=B, ys=512, dtype=0, m=4, d=512, norm=_desc(), post=None, mod=_mod(), out=_out(),
          h=J):
    if not residual:
        return L.convrot_norm(x, xs, dtype, m, d, norm, mod, out, None)
    return L.convrot_residual_norm(x, xs, y, ys, dtype, m, d, 1.0, post, norm, mod, h, out, None)


@pytest.mark.parametrize("residual", [False, True])
def test_refusals(L, residual):
    def call(**kw):
        return _call(L, residual, **kw)

    for m, d in ((-1, 512), ((1 << 24) + 1, 8), (4, 0), (4, -1), (4, 16385), (1 << 22, 16384)):
        assert call(m=m, d=d) == SHAPE, (m, d)
    assert call(dtype=2) == INVALID and call(dtype=-1) == INVALID
    assert call(norm=None) == INVALID and call(out=None) == INVALID
    for bad in (dict(kind=0), dict(kind=3), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(norm=_desc(**bad)) == INVALID, bad
    assert call(norm=_desc(weight=C + 2)) == ALIGN and call(norm=_desc(bias=D + 1)) == ALIGN
    assert call(out=_out(kind=3)) == INVALID and call(out=_out(kind=-1)) == INVALID
    assert call(out=_out(kind=1), d=520) == SHAPE and call(out=_out(kind=2), d=264) == SHAPE
    assert call(xs=-1) == SHAPE and call(xs=1 << 31) == SHAPE
    for bad in (dict(rows=0), dict(rows=3), dict(rows=1 << 30), dict(ss=-1), dict(hs=1 << 31), dict(gs=-5)):
        assert call(mod=_mod(**bad)) == SHAPE, bad
    assert call(mod=_mod(dtype=1)) == INVALID and call(mod=_mod(dtype=3)) == INVALID
    assert call(m=0, x=None, y=None, h=None, out=_out(values=None)) == OK
    assert call(x=None) == INVALID and call(out=_out(values=None)) == INVALID
    assert call(out=_out(kind=1, scales=None)) == INVALID
    assert call(x=A + 1) == ALIGN and call(out=_out(values=H + 1)) == ALIGN
    assert call(out=_out(kind=1, values=H + 8)) == ALIGN and call(out=_out(kind=2, scales=I + 4)) == ALIGN
    assert call(mod=_mod(scale=E + 1)) == ALIGN and call(mod=_mod(dtype=2, shift=F + 2)) == ALIGN
    assert call(mod=_mod(index=K + 2)) == ALIGN
    for at in (A, C, D, E, F):                     # the output over an input
        assert call(out=_out(values=at)) == INVALID, at
    assert call(mod=_mod(index=H), out=_out()) == INVALID
    assert call(out=_out(kind=2, scales=H + 16)) == INVALID
    assert call(out=_out(values=A + 2 * 3 * 1024, scales=None), xs=1024) == INVALID     # the last row's start


def test_residual_refusals(L):
    def call(**kw):
        return _call(L, True, **kw)

    assert call(post=_desc(kind=7)) == INVALID and call(post=_desc(eps=-1.0)) == INVALID
    assert call(post=_desc(weight=C + 1)) == ALIGN
    assert call(ys=-1) == SHAPE and call(ys=1 << 31) == SHAPE
    assert call(y=None) == INVALID and call(h=None) == INVALID
    assert call(y=B + 1) == ALIGN and call(h=J + 1) == ALIGN and call(mod=_mod(gate=G + 1)) == ALIGN
    for at in (A + 2, B + 1024, C, D, E, F, G, H):  # h over an input or the other output
        assert call(h=at) == INVALID, at
    assert call(h=A, xs=1024) == INVALID and call(h=B, ys=520) == INVALID      # in place only where that is dense
    assert call(h=A, y=A, ys=1024) == INVALID
    assert call(h=A, mod=_mod(gate=A)) == INVALID
    assert call(out=_out(values=B)) == INVALID


def test_binding_refuses_before_the_library():
    x = torch.zeros((2, 256))
    for call in (lambda t: cr.norm(t), lambda t: cr.norm_quant(t, bits=4), lambda t: cr.residual_norm(t, t),
                 lambda t: cr.residual_norm_quant(t, t, bits=8)):
        with pytest.raises(TypeError):
            call(x)
        with pytest.raises(ValueError, match="GPU"):
            call(x.half())
        with pytest.raises(TypeError):
            call([1.0])
    with pytest.raises(ValueError, match="kind"):
        norms._desc("batch", 0.0, None, None, 256, -1)
    with pytest.raises(TypeError):
        norms._desc("rms", 0.0, x[0].half(), None, 256, -1)
    with pytest.raises(ValueError):
        norms._desc("rms", 0.0, x[0, :5], None, 256, -1)
    with pytest.raises(ValueError, match="bits"):
        norms._quantised(2, 256, 5, x)
    with pytest.raises(ValueError, match="multiple"):
        norms._quantised(2, 300, 8, x)
    with pytest.raises(ValueError):
        norms._alike(x, x[:1])
    with pytest.raises(ValueError):
        norms._alike(x, x.half())


def test_structures_are_packed_as_c_lays_them_out():
    class Desc(ctypes.Structure):
        _fields_ = [("kind", ctypes.c_int), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p)]

    class Mod(ctypes.Structure):
        _fields_ = [*((n, ctypes.c_void_p) for n in ("scale", "shift", "gate")),
                    *((n, ctypes.c_int64) for n in ("a", "b", "c")), ("dtype", ctypes.c_int), ("rows", ctypes.c_int64),
                    ("index", ctypes.c_void_p)]

    class Out(ctypes.Structure):
        _fields_ = [("kind", ctypes.c_int), ("values", ctypes.c_void_p), ("scales", ctypes.c_void_p)]

    for kind, packer, values in ((Desc, norms._DESC, (2, 0.5, 1 << 40, 5)), (Out, norms._OUT, (1, 3 << 40, 7)),
                                 (Mod, norms._MOD, (1, 2 << 40, 3, 4, 5 << 33, 6, 2, 7 << 34, 8))):
        raw = packer.pack(*values)
        assert len(raw) == ctypes.sizeof(kind)
        got = kind.from_buffer_copy(raw)
        assert tuple(getattr(got, f[0]) for f in kind._fields_) == values


def test_binding_checks_the_modulation():
    x = torch.zeros((6, 8), dtype=torch.float16)
    two, three = torch.zeros((2, 8), dtype=torch.float16), torch.zeros((3, 8), dtype=torch.float16)

    def call(scale=None, shift=None, gate=None, index=None):
        raw, kept = norms._modulation(x, 6, 8, scale, shift, gate, index)
        return None if raw is None else norms._MOD.unpack(raw)

    at = two.data_ptr()
    assert call(two, two) == (at, at, 0, 8, 8, 0, 0, 2, 0)
    assert call(two.float())[6] == 2 and call(two[0])[7] == 1 and call() is None
    wide = torch.zeros((2, 24), dtype=torch.float16)
    assert call(wide[:, 8:16])[:4] == (wide.data_ptr() + 16, 0, 0, 24)
    assert call(two[:1].expand(6, 8))[3] == 0
    for bad in ((two, three), (two, two.float()), (two[:, :4],), (torch.zeros((4, 8)).half(),), (two.bfloat16(),)):
        with pytest.raises((ValueError, TypeError)):
            call(*bad)
    index = torch.zeros(6, dtype=torch.int32)
    assert call(two, index=index)[8] == index.data_ptr()
    for bad in (index.long(), index[:5]):
        with pytest.raises((ValueError, TypeError)):
            call(two, index=bad)
    with pytest.raises(ValueError):
        call(index=index)
