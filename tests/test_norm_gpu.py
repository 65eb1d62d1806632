"""The norms around the linears on the GPU against their oracle in 64 bits.

16-bit outputs: |d| <= h (1 + 2^-11) |n| + tiny + 2^-40 T, h = eps / 2 of the
type (its one rounding, of a value rounded to fp32 before: 2^-24 next to 2^-9
or 2^-12, inside the 2^-11) and tiny half its smallest step (plus fp32's, which
is less); T the sum of the sizes that meet in n, whose fp64 roundings and sums
(2^-53 times some hundred) the last term covers.  Codes and scales are compared
bit for bit.
"""

import numpy as np
import pytest
import torch

import rotation_quantized_int8_amd as cr
from oracle import mx_oracle as MX
from oracle import norm_oracle as O

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


def _gen(*key):
    return torch.Generator().manual_seed(hash(key) % (1 << 31))


def _x(gen, m, d, dtype):
    x = torch.randn((m, d), generator=gen)
    x[:, ::83] *= 20
    return (x * (0.5 + torch.rand((m, 1), generator=gen))).to(dtype)


def _close(got, want, size, what=""):
    h = torch.finfo(got.dtype).eps / 2
    tiny = {F16: 2.0 ** -25, BF16: 2.0 ** -133}[got.dtype]
    err, bound = np.abs(_np(got) - want), h * (1 + 2.0 ** -11) * np.abs(want) + tiny + 2.0 ** -40 * size
    at = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), (what, at, err[at], bound[at], want[at])


def _equal8(q, s, want):
    wq, ws = want
    assert np.array_equal(s.cpu().numpy().view(np.uint32), ws.view(np.uint32)) or np.array_equal(_np(s), ws, equal_nan=True)
    assert np.array_equal(_np(q), wq), np.argwhere(_np(q) != wq)[:4]


def _equal4(q, s, n):
    """Codes and scales bit for bit, but for the sign of a 0: fp64 sums leave what is 0 exactly (a row of +-c)
    within 2^-50 of it on either side, and both codes of 0 stand for the same."""
    wc, ws = MX.quantize(MX.rotate_f32(n))
    c, e = MX.unpack(_np(q), _np(s))
    assert np.array_equal(e, ws) and np.array_equal(np.where(c == 8, 0, c), np.where(wc == 8, 0, wc)), \
        np.argwhere((c != wc) & ((c | wc) != 8))[:4]


class _Case:
    """Rows, modulation and weights of a call, and the oracle's answers."""

    def __init__(self, m, d, dtype, images=1, mod=None, affine=True, kind="layer", index=None, key=0):
        gen = _gen(m, d, images, kind, key)
        self.kind, self.x, self.y = kind, _x(gen, m, d, dtype), _x(gen, m, d, dtype)
        self.weight = 1 + 0.2 * torch.randn((d,), generator=gen) if affine else None
        self.bias = 0.1 * torch.randn((d,), generator=gen) if affine else None
        self.post_weight = 1 + 0.2 * torch.randn((d,), generator=gen)
        side = 0.3 * torch.randn((images, 3 * d + 5), generator=gen)       # odd offsets and stride
        self.scale = self.shift = self.gate = None
        if mod is not None:
            self.all = side.to(mod).to(DEV)
            self.shift, self.scale, self.gate = self.all[:, 1:d + 1], self.all[:, d + 1:2 * d + 1], self.all[:, 2 * d + 2:3 * d + 2]
        self.index = index
        self.of = np.asarray(index) if index is not None else np.arange(m) // (m // images)
        self.alive = (self.of >= 0) & (self.of < images)

    def gpu(self, *names):
        out = {n: getattr(self, n) for n in names}
        out = {n: t.to(DEV) if t is not None else None for n, t in out.items()}
        if self.index is not None:
            out["index"] = torch.tensor(self.index, dtype=torch.int32, device=DEV)
        return out

    def rows_of(self, t):
        return None if t is None else _np(t)[np.where(self.alive, self.of, 0)]

    def normed(self, v):
        """(n, sizes)."""
        n = O.norm(v, self.kind, EPS, None if self.weight is None else _np(self.weight),
                   None if self.bias is None else _np(self.bias))
        sc, sh = self.rows_of(self.scale), self.rows_of(self.shift)
        size = np.abs(n) + np.abs(v).max(1, keepdims=True) / np.sqrt((v * v).mean(1, keepdims=True) + EPS) + 1
        big = (1 + np.abs(sc) if sc is not None else 1) * size + (np.abs(sh) if sh is not None else 0)
        return O.modulate(n, sc, sh), big

    def h(self, post, residual_scale):
        p = None if post is None else (post, EPS, _np(self.post_weight), None)
        g = self.rows_of(self.gate)
        return O.residual(_np(self.x), _np(self.y), residual_scale, g, p)


NAMES = ("weight", "bias", "scale", "shift")
SIZES = [(1, 1), (2, 7), (5, 8), (3, 33), (4, 255), (64, 512), (9, 513), (7, 1001), (30, 1024), (6, 2048), (5, 2049),
         (3, 4096), (2, 5003), (2, 8192), (1, 16384), (2, 32768), (1, 32767)]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,d", SIZES)
def test_norm(m, d, dtype, kind):
    for mod, affine in ((None, False), (None, True), (dtype, False), (F32, True)):
        c = _Case(m, d, dtype, images=m if m % 2 else m // 2, mod=mod, affine=affine, kind=kind)
        n = cr.norm(c.x.to(DEV), kind=kind, eps=EPS, **c.gpu(*NAMES))
        _close(n, *c.normed(_np(c.x)), what=(mod, affine))


@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,d", SIZES)
def test_residual_norm(m, d, dtype, post):
    c = _Case(m, d, dtype, images=m, mod=dtype, affine=True, kind="rms" if post == "layer" else "layer")
    how = dict(residual_scale=0.5, post=post, post_eps=EPS, post_weight=c.post_weight.to(DEV) if post else None)
    h, n = cr.residual_norm(c.x.to(DEV), c.y.to(DEV), kind=c.kind, eps=EPS, **c.gpu(*NAMES, "gate"), **how)
    want = c.h(post, 0.5)
    hs = np.abs(want) + np.abs(_np(c.x)) + 2 * np.abs(_np(c.y)) + 40
    _close(h, want, hs, "h")
    wn, size = c.normed(want)
    _close(n, wn, size + hs / np.sqrt((want * want).mean(1, keepdims=True) + EPS), "n")
    h2, none = cr.residual_norm(c.x.to(DEV), c.y.to(DEV), kind=None, gate=c.gate, **how)
    assert none is None and torch.equal(h2, h)


QUANT = [(1, 256), (5, 512), (6, 768), (4, 1024), (9, 1280), (16, 2048), (3, 2304), (2, 4096), (3, 8192), (1, 16384),
         (2, 32768)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,d", QUANT)
def test_quantised_bit_exact(m, d, dtype):
    for kind, mod, affine in (("layer", dtype, False), ("rms", F32, True)):
        c = _Case(m, d, dtype, images=1, mod=mod, affine=affine, kind=kind)
        n, _ = c.normed(_np(c.x))
        how = dict(kind=kind, eps=EPS, **c.gpu(*NAMES))
        _equal8(*cr.norm_quant(c.x.to(DEV), bits=8, **how), O.quantize_int8(n))
        _equal4(*cr.norm_quant(c.x.to(DEV), bits=4, **how), n)
        post = "rms" if kind == "layer" else None
        how.update(gate=c.gate, residual_scale=0.5, post=post, post_weight=c.post_weight.to(DEV) if post else None)
        want = c.h(post, 0.5)
        n, _ = c.normed(want)
        h, q, s = cr.residual_norm_quant(c.x.to(DEV), c.y.to(DEV), bits=8, **how)
        _equal8(q, s, O.quantize_int8(n))
        h4, q, s = cr.residual_norm_quant(c.x.to(DEV), c.y.to(DEV), bits=4, **how)
        _equal4(q, s, n)
        h16, _ = cr.residual_norm(c.x.to(DEV), c.y.to(DEV), **how)
        assert torch.equal(h, h16) and torch.equal(h4, h16)


@pytest.mark.parametrize("d", [40, 512, 4096])
def test_index_and_padding_rows(d):
    """Rows in any order of the modulation's; rows out of range keep what the outputs held."""
    index = [2, 0, -1, 1, 3, 2, 1 << 30, 0, -(1 << 31), 1, 0]
    c = _Case(len(index), d, BF16, images=3, mod=BF16, affine=False, index=index)
    x, y, how = c.x.to(DEV), c.y.to(DEV), c.gpu("scale", "shift")
    out = torch.full_like(x, 7.0)
    assert cr.norm(x, eps=EPS, out=out, **how) is out
    dead = torch.from_numpy(~c.alive).to(DEV)
    assert (out[dead] == 7).all()
    n, size = c.normed(_np(c.x))
    _close(out[~dead], n[c.alive], size[c.alive])
    h, n16 = torch.full_like(x, 5.0), torch.full_like(x, 6.0)
    cr.residual_norm(x, y, eps=EPS, gate=c.gate, out=(h, n16), **how)
    assert (h[dead] == 5).all() and (n16[dead] == 6).all()
    want = c.h(None, 1.0)
    _close(h[~dead], want[c.alive], (np.abs(want) + 100)[c.alive])
    if d % 256 == 0:
        q, s = cr.norm_quant(x, bits=4, eps=EPS, **how)
        alive = np.flatnonzero(c.alive)
        _equal4(q[~dead], s[:, ~dead], n[alive])
        q, s = cr.norm_quant(x, bits=8, eps=EPS, **how)
        _equal8(q[~dead], s[~dead], O.quantize_int8(n[alive]))


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_that_go_wrong_elsewhere(kind, dtype):
    """Constant rows, rows of zeros, rows whose squares or sums pass fp32, a mean far above the spread."""
    big = 6e4 if dtype is F16 else 3e38
    x = torch.zeros((8, 768))
    x[1] = 3.140625
    x[2] = big * torch.sign(torch.randn(768, generator=_gen(1)))
    x[3] = big
    x[4] = 1000 + torch.arange(768) % 2 * 8
    x[5] = 2.0 ** -24 if dtype is F16 else 2.0 ** -133
    x[6, 5] = big
    x[7] = torch.randn(768, generator=_gen(2)) * 1e-4
    x = x.to(dtype)
    v = _np(x)
    want = O.norm(v, kind, EPS)
    size = np.abs(v).max(1, keepdims=True) / np.sqrt(((v - (v.mean(1, keepdims=True) if kind == "layer" else 0)) ** 2
                                                      ).mean(1, keepdims=True) + EPS) + 1
    _close(cr.norm(x.to(DEV), kind=kind, eps=EPS), want, size)
    assert torch.isfinite(cr.norm(x.to(DEV), kind=kind, eps=EPS)).all()
    if kind == "layer":
        assert not cr.norm(x[[0, 1, 3]].to(DEV), eps=EPS).any()
    else:
        _equal8(*cr.norm_quant(x.to(DEV), bits=8, kind=kind, eps=EPS), O.quantize_int8(want))
        _equal4(*cr.norm_quant(x.to(DEV), bits=4, kind=kind, eps=EPS), want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_shows_in_its_row_alone(bad):
    x = _x(_gen(3), 6, 1024, BF16)
    x[2, 77] = bad
    n = cr.norm(x.to(DEV)).cpu()
    assert torch.isnan(n[2, 77]) and torch.isfinite(n[[0, 1, 3, 4, 5]]).all()
    q, s = cr.norm_quant(x.to(DEV), bits=8)
    assert torch.isnan(s[2]) and not q[2].any() and torch.isfinite(s[[0, 1, 3, 4, 5]]).all()
    v = cr.mx_dequantize(*cr.norm_quant(x.to(DEV), bits=4)).cpu()
    assert torch.isnan(v[2]).any() and torch.isfinite(v[[0, 1, 3, 4, 5]]).all()
    y = x.flip(0)
    h, n = cr.residual_norm(_x(_gen(4), 6, 1024, BF16).to(DEV), y.to(DEV), post="rms")
    assert not torch.isfinite(h[3, 77]) and torch.isfinite(n[[0, 1, 2, 4, 5]]).all()


def test_tiny_rows_in_int8():
    """A row whose scale leaves fp32's normal range still has the codes of its quotients."""
    w = torch.full((512,), 2.0 ** -126) * (1 + torch.arange(512) % 7)
    x = _x(_gen(5), 4, 512, BF16)
    n = O.norm(_np(x), "rms", EPS, _np(w))
    for f in (1.0, 2.0 ** -10, 2.0 ** -20, 2.0 ** -23):
        sc = torch.full((1, 512), f - 1.0)
        q, s = cr.norm_quant(x.to(DEV), bits=8, kind="rms", eps=EPS, weight=w.to(DEV), scale=sc.to(DEV))
        u = MX.rotate_f32(n * (1 + _np(sc)))
        ws = (np.abs(u).max(1) / np.float32(127)).astype(np.float32)
        with np.errstate(divide="ignore", invalid="ignore"):
            wq = np.clip(np.rint((u / ws[:, None]).astype(np.float32)), -127, 127)
        wq = np.where(ws[:, None] > 0, wq, 0)
        assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(_np(q), wq)


@pytest.mark.parametrize("m,d", [(5, 40), (6, 2048), (3, 4096)])
def test_in_place_and_strides(m, d):
    """h over x or y; rows read from slices and broadcast modulations in place."""
    c = _Case(m, d, F16, images=1, mod=F16, affine=True)
    x, y, how = c.x.to(DEV), c.y.to(DEV), c.gpu(*NAMES, "gate")
    h, n = cr.residual_norm(x, y, post="rms", **how)
    for k in range(2):
        a, b = x.clone(), y.clone()
        out = (a, b)[k]
        got = cr.residual_norm(a, b, post="rms", out=(out, torch.empty_like(n)), **how)
        assert got[0] is out and torch.equal(out, h) and torch.equal(got[1], n)
    wide = torch.full((m, d + 11), float("nan"), dtype=F16, device=DEV)
    wide[:, 3:d + 3] = x
    assert torch.equal(cr.norm(wide[:, 3:d + 3], **c.gpu(*NAMES)), cr.norm(x, **c.gpu(*NAMES)))
    each = {k: v.expand(m, -1) if k in ("scale", "shift", "gate") else v for k, v in how.items()}    # stride 0
    assert torch.equal(cr.residual_norm(x, y, post="rms", **each)[1], n)
    assert torch.equal(cr.norm(x.view(1, m, d), scale=c.scale[0]).view(m, d), cr.norm(x, scale=c.scale))


def test_block_together():
    """norm -> 4-bit linear -> gated residual and the next norm -> int8 linear, against 64 bits on the same codes."""
    gen = _gen(6)
    c = _Case(300, 1024, BF16, images=3, mod=BF16, affine=False)
    x, w1, w2 = c.x.to(DEV), *((torch.randn((1024, 1024), generator=gen) * 0.03 for _ in range(2)))
    q1, s1 = cr.mx_quantize_weights(w1.to(DEV))
    q2, s2 = cr.quantize_weights(w2.to(DEV))
    mod = c.gpu("scale", "shift")
    q, s = cr.norm_quant(x, bits=4, eps=EPS, **mod)
    y = cr.mx_gemm(q, s, q1, s1, out_dtype=BF16)
    h, a, b = cr.residual_norm_quant(x, y, bits=8, eps=EPS, gate=c.gate, **mod)
    z = cr.gemm_i8_f16(a, b, q2, s2)

    n, _ = c.normed(_np(c.x))
    xv, wv = MX.values(*MX.quantize(MX.rotate_f32(n))), MX.values(*MX.unpack(_np(q1), _np(s1)))
    wy, terms = MX.product(xv, wv)
    h16 = torch.finfo(BF16).eps / 2                     # the product's bound: half a step, 2^-8 of a value, and its sums
    assert (np.abs(_np(y) - wy) <= h16 * np.abs(wy) + 1028 * 2.0 ** -23 * terms + 2.0 ** -133).all()
    c.y = y
    want = c.h(None, 1.0)
    _close(h, want, np.abs(want) + 100)
    wq, ws = O.quantize_int8(c.normed(want)[0])
    _equal8(a, b, (wq, ws))
    wz = (wq.astype(np.float64) @ _np(q2).astype(np.float64).T).astype(np.float32) * (ws[:, None] * _np(s2).astype(np.float32))
    assert np.array_equal(_np(z), wz.astype(np.float16).astype(np.float64))


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_graph_and_streams(bits):
    c = _Case(260, 2048, BF16, images=2, mod=BF16, affine=False)
    x, y, how = c.x.to(DEV), c.y.to(DEV), c.gpu("scale", "shift", "gate")

    def call():
        return cr.residual_norm(x, y, **how) if bits == 16 else cr.residual_norm_quant(x, y, bits=bits, **how)

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = call()
        for _ in range(4):
            for t in got:
                t.zero_()
            graph.replay()
            eager = call()
            side.synchronize()
            assert all(torch.equal(a, b) and torch.equal(a, e) for a, b, e in zip(want, got, eager))
    torch.cuda.current_stream().wait_stream(side)


def test_empty():
    assert cr.norm(torch.empty((0, 40), dtype=F16, device=DEV)).shape == (0, 40)
    q, s = cr.norm_quant(torch.empty((0, 256), dtype=F16, device=DEV), bits=4)
    assert q.shape == (0, 128) and s.shape == (1, 0, 8)
