"""Codes and scales of the quantising norms are the formula's.

The kernels are fp64 up to u = fp32(n H), so a code or scale may differ from the
64-bit oracle's only where the rotated value R lies within
  d = 2^-43 (|R| + sum(T) / 16)
of a border, T the sizes that meet in an element of n: a sum over a row passes at
most 16 + 6 + 16 additions (a lane, the lanes, the wavefronts) of 2^-53, so mu and
r are within 2^-47; an element has 7 roundings and its rotation 8, less than 2^-49
of the sum of its sizes; the oracle's rotation has 256 additions, 2^-45.  With
fp32 arithmetic d would be 2^24 times as wide.
"""

import numpy as np
import pytest
import torch

import rotation_quantized_int8_amd as cr
from oracle import mx_oracle as MX
from oracle import norm_oracle as O
from oracle.convrot_oracle import hadamard256

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cr.lib()
    torch.cuda.set_device(0)


def _np(t):
    return t.detach().to(torch.float64).cpu().numpy() if t.is_floating_point() else t.detach().cpu().numpy()


def _between(n, size):
    """The fp32 values that u may have: lowest and highest."""
    u = (n.reshape(-1, 256) @ hadamard256()).reshape(n.shape)
    total = np.broadcast_to(size, n.shape).reshape(-1, 256).sum(1).repeat(256).reshape(n.shape)
    d = 2.0 ** -43 * (np.abs(u) + total / 16)
    with np.errstate(over="ignore"):
        return (u - d + 0.0).astype(np.float32), (u + d + 0.0).astype(np.float32)


def _sizes(low, high):
    """Smallest and largest |u| of values between low and high."""
    least = np.where((low <= 0) & (high >= 0), np.float32(0), np.minimum(np.abs(low), np.abs(high)))
    return least, np.maximum(np.abs(low), np.abs(high))


def _equal8(q, s, n, size):
    low, high = _between(n, size)
    least, most = _sizes(low, high)
    q, s = _np(q), s.cpu().numpy()
    k = np.float32(127)
    assert ((s >= least.max(1) / k) & (s <= most.max(1) / k)).all()
    safe = np.where(s > 0, s, np.float32(1))[:, None]
    a, b = (np.where(s[:, None] > 0, np.rint(v / safe), 0) for v in (low, high))
    assert ((q >= a) & (q <= b)).all(), np.argwhere((q < a) | (q > b))[:4]
    return (a != b).mean()                         # the share that a border leaves open


def _equal4(q, s, n, size):
    low, high = _between(n, size)
    least, most = _sizes(low, high)
    m, k = n.shape
    c, e = MX.unpack(_np(q), _np(s))
    a, b = (MX.exponent(v.reshape(m, k // 32, 32).max(-1)) + 127 for v in (least, most))
    assert ((e >= a) & (e <= b)).all(), np.argwhere((e < a) | (e > b))[:4]
    p = np.repeat(2.0 ** (e - 127.0), 32, 1)
    a, b = (MX.decode(MX.encode(v.astype(np.float64) / p)) for v in (low, high))
    c = MX.decode(c)
    assert ((c >= a) & (c <= b)).all(), np.argwhere((c < a) | (c > b))[:4]
    return (a != b).mean()


def _x(gen, m, d, dtype):
    x = torch.randn((m, d), generator=gen)
    x[:, ::83] *= 20
    return (x * (0.5 + torch.rand((m, 1), generator=gen))).to(dtype)


SHAPES = [(512, 256), (513, 768), (300, 1024), (512, 2048), (100, 2304), (64, 8192), (17, 16384)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("m,d", SHAPES)
def test_codes_are_the_formulas(m, d, kind, dtype):
    gen = torch.Generator().manual_seed(1000 * m + d)
    x, y = _x(gen, m, d, dtype), _x(gen, m, d, dtype)
    w, b = 1 + 0.2 * torch.randn((d,), generator=gen), 0.1 * torch.randn((d,), generator=gen)
    pw, pb = 1 + 0.2 * torch.randn((d,), generator=gen), 0.1 * torch.randn((d,), generator=gen)
    mod = (0.3 * torch.randn((1, 3 * d), generator=gen)).to(dtype if kind == "layer" else F32)
    shift, scale, gate = mod.split(d, 1)

    def normed(v, extra=0.0):
        n = O.norm(v, kind, EPS, _np(w), _np(b))
        spread = np.sqrt(((v - (v.mean(1, keepdims=True) if kind == "layer" else 0)) ** 2).mean(1, keepdims=True) + EPS)
        size = np.abs(n) + 2 * (np.abs(v).max(1, keepdims=True) + extra) / spread + 1
        return O.modulate(n, _np(scale), _np(shift)), (1 + np.abs(_np(scale))) * size + np.abs(_np(shift))

    how = dict(kind=kind, eps=EPS, weight=w.to(DEV), bias=b.to(DEV), scale=scale.to(DEV), shift=shift.to(DEV))
    n, size = normed(_np(x))
    assert _equal8(*cr.norm_quant(x.to(DEV), bits=8, **how), n, size) < 1e-5
    assert _equal4(*cr.norm_quant(x.to(DEV), bits=4, **how), n, size) < 1e-5
    for post in (None, "layer", "rms"):
        v = O.residual(_np(x), _np(y), 0.5, _np(gate), post and (post, EPS, _np(pw), _np(pb)))
        # what meets in h: y, or a normed one below sqrt(d), with weights and gate below 3
        n, size = normed(v, np.abs(_np(x)).max() + 3 * np.abs(_np(y)).max() + 9 * d ** 0.5)
        more = dict(how, gate=gate.to(DEV), residual_scale=0.5, post=post, post_eps=EPS)
        if post:
            more.update(post_weight=pw.to(DEV), post_bias=pb.to(DEV))
        h, q, s = cr.residual_norm_quant(x.to(DEV), y.to(DEV), bits=8, **more)
        assert _equal8(q, s, n, size) < 1e-5
        h4, q, s = cr.residual_norm_quant(x.to(DEV), y.to(DEV), bits=4, **more)
        assert _equal4(q, s, n, size) < 1e-5
        # h: to fp32 (2^-24) and to its type (half a step, in the subnormals half of the smallest)
        tiny = {F16: 2.0 ** -25, BF16: 2.0 ** -134}[dtype]
        far = (torch.finfo(dtype).eps / 2 + 2.0 ** -23) * np.abs(v) + tiny + 2.0 ** -40
        assert torch.equal(h, h4) and (np.abs(_np(h) - v) <= far).all()


def test_spread_far_below_the_mean():
    """Rows whose mean is far above their spread: their codes are those of the spread."""
    d = 1024
    gen = torch.Generator().manual_seed(5)
    x = torch.full((4, d), 60000.0)
    x[0, 17] = x[1, 5] = 60032.0
    x[2, ::2] = 60032.0
    x[3] += 32 * torch.randint(-2, 3, (d,), generator=gen)
    x = x.to(F16)
    n = O.norm(_np(x), "layer", EPS)
    # differences of values are exact in 64 bits but for the mean's rounding, 2^-53 of 60000
    size = np.abs(n) + 1 + 2.0 ** -9 * 60000
    _equal8(*cr.norm_quant(x.to(DEV), bits=8, eps=EPS), n, size)
    _equal4(*cr.norm_quant(x.to(DEV), bits=4, eps=EPS), n, size)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_values_up_to_the_end_of_fp32(dtype):
    """Rotated values of nearly 2^128 have their codes; past it the block is not a number."""
    gen = torch.Generator().manual_seed(6)
    x = torch.sign(torch.randn((6, 256), generator=gen)).to(dtype)
    for up in (0, 3, 5):
        w = torch.full((256,), 2.0 ** (122 + up))
        n = O.norm(_np(x), "rms", 0.0, _np(w))
        u = MX.rotate_f32(n)
        assert np.isfinite(u).all() == (up < 5) and np.abs(u).max() > 2.0 ** (122 + up)
        q, s = cr.norm_quant(x.to(DEV), bits=4, kind="rms", eps=0.0, weight=w.to(DEV))
        want = MX.pack(*MX.quantize(u))
        assert np.array_equal(_np(q), want[0]) and np.array_equal(_np(s), want[1]), up
        q, s = cr.norm_quant(x.to(DEV), bits=8, kind="rms", eps=0.0, weight=w.to(DEV))
        want = O.quantize_int8(n)
        assert np.array_equal(_np(q), want[0]) and np.array_equal(s.cpu().numpy(), want[1], equal_nan=True), up


@pytest.mark.parametrize("d", [768, 49 * 256])
def test_rows_of_one_value(d):
    """They give 0 under any eps above 0, also behind a residual whose sums round."""
    x = torch.tensor([0.0, 1.0, -3.140625, 2.0 ** -14, 6e4, 0.01])[:, None].expand(-1, d).contiguous().to(F16).to(DEV)
    for eps in (1e-6, 1e-30, 1e-44):
        q, s = cr.norm_quant(x, bits=8, eps=eps)
        assert not q.any() and not s.any()
        h, q, s = cr.residual_norm_quant(x, x, bits=4, eps=eps, residual_scale=0.1, post="rms", post_eps=eps,
                                         gate=torch.full((1, d), 0.3, device=DEV))
        assert not q.any() and not s.any()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_no_eps_and_sizes_at_the_ends(dtype):
    """Rows of the type's smallest and largest values have the codes of their quotients."""
    gen = torch.Generator().manual_seed(7)
    base = torch.randn((3, 512), generator=gen)
    for f in ((2.0 ** -18, 2.0 ** 12) if dtype is F16 else (2.0 ** -126, 2.0 ** -100, 2.0 ** 124)):
        x = (base.double() * f).to(dtype)
        for kind in ("layer", "rms"):
            n = O.norm(_np(x), kind, 0.0)
            q, s = cr.norm_quant(x.to(DEV), bits=4, kind=kind, eps=0.0)
            _equal4(q, s, n, np.abs(n) + 8)
