"""The norms around the linears on the GPU against their oracle in 64 bits.

All arithmetic between the loads and the one rounding of an output is fp32.
With T the sum of the sizes that meet in an element of n (or h):
  16-bit outputs  |d| <= h |n| + tiny + 2^-18 T, h = eps / 2 of the type (its one
                  rounding) and tiny half its smallest step.  Up to 6 roundings
                  of an element are 6 2^-24; a sum passes at most 3 + 4 + 6 + 16
                  additions (a chunk, a lane's units, the lanes, the wavefronts),
                  so r is within 32 2^-24 / 2 + 2^-23, and mu, whose rounding the
                  second sum takes out, within 2^-19 of the spread: together less
                  than 2^-18.
  quantised       the rotated value u is within
                  d = 2^-19 |u| + 2^-20 sum(T) / 16 + 2^-142
                  of the oracle's (r errs for the whole row alike; 6 roundings of
                  each of its group's 256 terms and 8 additions, the last term
                  for results in fp32's subnormals: 2^-149 for each), so a scale
                  must be that of some value within d of the largest and a code
                  that of some value within d of u, under the scale that was
                  given.  Both are the oracle's own but next to a border.
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


def _gen(*key):
    return torch.Generator().manual_seed(hash(key) % (1 << 31))


def _x(gen, m, d, dtype):
    x = torch.randn((m, d), generator=gen)
    x[:, ::83] *= 20
    return (x * (0.5 + torch.rand((m, 1), generator=gen))).to(dtype)


def _close(got, want, size, what=""):
    h = torch.finfo(got.dtype).eps / 2
    tiny = {F16: 2.0 ** -25, BF16: 2.0 ** -134}[got.dtype]
    err, bound = np.abs(_np(got) - want), h * np.abs(want) + tiny + 2.0 ** -18 * size
    at = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), (what, at, err[at], bound[at], want[at])


def _turned(n, size):
    """u in 64 bits and how far an fp32 result may be from it."""
    u = (n.reshape(-1, 256) @ hadamard256()).reshape(n.shape)
    d = 2.0 ** -19 * np.abs(u).reshape(-1, 256) + 2.0 ** -20 * size.reshape(-1, 256).sum(1, keepdims=True) / 16
    return u, d.reshape(n.shape) + 2.0 ** -142


def _equal8(q, s, n, size):
    u, d = _turned(n, np.broadcast_to(size, n.shape))
    q, s = _np(q), _np(s)
    low, high = (np.abs(u) - d).max(1) / 127, (np.abs(u) + d).max(1) / 127
    assert ((s >= low * (1 - 2.0 ** -23) - 2.0 ** -149) & (s <= high * (1 + 2.0 ** -23) + 2.0 ** -149)).all(), (s, low, high)
    safe = np.where(s > 0, s, 1)[:, None]
    for bound, ok in ((u - d, np.less_equal), (u + d, np.greater_equal)):
        want = np.where(s[:, None] > 0, np.clip(np.rint(bound / safe), -127, 127), 0)
        assert ok(want, q).all(), np.argwhere(~ok(want, q))[:4]


def _equal4(q, s, n, size):
    u, d = _turned(n, np.broadcast_to(size, n.shape))
    c, e = MX.unpack(_np(q), _np(s))
    m, k = u.shape
    for bound, ok in (((np.abs(u) - d), np.less_equal), ((np.abs(u) + d), np.greater_equal)):
        want = MX.exponent(bound.reshape(m, k // 32, 32).max(-1).clip(0)) + 127
        assert ok(want, e).all(), (np.argwhere(~ok(want, e))[:4], want, e)
    p = np.repeat(2.0 ** (e - 127.0), 32, 1)
    for bound, ok in ((u - d, np.less_equal), (u + d, np.greater_equal)):
        want = MX.decode(MX.encode(bound / p))
        assert ok(want, MX.decode(c)).all(), np.argwhere(~ok(want, MX.decode(c)))[:4]


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


    def h_size(self, want):
        """Sizes that meet in h: gate and post weight below 3, a normed y below sqrt(D)."""
        return np.abs(want) + np.abs(_np(self.x)) + 3 * np.abs(_np(self.y)) + 9 * min(40, want.shape[1] ** 0.5)


NAMES = ("weight", "bias", "scale", "shift")
SIZES = [(1, 1), (2, 7), (5, 8), (3, 33), (4, 255), (64, 512), (9, 513), (7, 1001), (30, 1024), (6, 2048), (5, 2049),
         (3, 4096), (2, 5003), (2, 8192), (3, 8200), (2, 16384), (1, 16383)]


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
    hs = c.h_size(want)
    _close(h, want, hs, "h")
    wn, size = c.normed(want)
    _close(n, wn, size + hs / np.sqrt((want * want).mean(1, keepdims=True) + EPS), "n")
    h2, none = cr.residual_norm(c.x.to(DEV), c.y.to(DEV), kind=None, gate=c.gate, **how)
    assert none is None and torch.equal(h2, h)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,d", [(2100, 1000), (2052, 1024), (4100, 513), (1030, 2041), (1026, 2048), (520, 4096),
                                 (516, 4095), (5000, 40)])
def test_many_rows(m, d, dtype):
    """The variants with two units a lane, which many rows take."""
    c = _Case(m, d, dtype, images=2, mod=dtype, affine=True)
    _close(cr.norm(c.x.to(DEV), eps=EPS, **c.gpu(*NAMES)), *c.normed(_np(c.x)))
    h, n = cr.residual_norm(c.x.to(DEV), c.y.to(DEV), eps=EPS, post="layer", post_eps=EPS,
                            post_weight=c.post_weight.to(DEV), **c.gpu(*NAMES, "gate"))
    want = c.h("layer", 1.0)
    hs = c.h_size(want)
    _close(h, want, hs, "h")
    wn, size = c.normed(want)
    _close(n, wn, size + hs / np.sqrt((want * want).mean(1, keepdims=True) + EPS), "n")
    h2, _ = cr.residual_norm(c.x.to(DEV), c.y.to(DEV), kind=None, post="layer", post_eps=EPS,
                             post_weight=c.post_weight.to(DEV), gate=c.gate)
    assert torch.equal(h2, h)


@pytest.mark.parametrize("m,d", [(8, 1280), (64, 768), (4096, 256), (1000, 2304)])
def test_many_quantised_rows(m, d):
    """Grids of a whole number of workgroups an XCD (their rows go side by side), and others."""
    c = _Case(m, d, BF16, images=1, mod=BF16, affine=False)
    n, size = c.normed(_np(c.x))
    _equal4(*cr.norm_quant(c.x.to(DEV), bits=4, eps=EPS, **c.gpu("scale", "shift")), n, size)


QUANT = [(1, 256), (5, 512), (6, 768), (4, 1024), (9, 1280), (16, 2048), (3, 2304), (2, 4096), (3, 8192), (2, 8448),
         (2, 16384)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,d", QUANT)
def test_quantised(m, d, dtype):
    for kind, mod, affine in (("layer", dtype, False), ("rms", F32, True)):
        c = _Case(m, d, dtype, images=1, mod=mod, affine=affine, kind=kind)
        n, size = c.normed(_np(c.x))
        how = dict(kind=kind, eps=EPS, **c.gpu(*NAMES))
        _equal8(*cr.norm_quant(c.x.to(DEV), bits=8, **how), n, size)
        _equal4(*cr.norm_quant(c.x.to(DEV), bits=4, **how), n, size)
        post = "rms" if kind == "layer" else None
        how.update(gate=c.gate, residual_scale=0.5, post=post, post_weight=c.post_weight.to(DEV) if post else None)
        want = c.h(post, 0.5)
        n, size = c.normed(want)
        size = size + c.h_size(want) / np.sqrt((want * want).mean(1, keepdims=True) + EPS)
        h, q, s = cr.residual_norm_quant(c.x.to(DEV), c.y.to(DEV), bits=8, **how)
        _equal8(q, s, n, size)
        h4, q, s = cr.residual_norm_quant(c.x.to(DEV), c.y.to(DEV), bits=4, **how)
        _equal4(q, s, n, size)
        assert torch.equal(h, h4)
        _close(h, want, c.h_size(want))


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
        _equal4(q[~dead], s[:, ~dead], n[alive], size[alive])
        q, s = cr.norm_quant(x, bits=8, eps=EPS, **how)
        _equal8(q[~dead], s[~dead], n[alive], size[alive])


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
        _equal8(*cr.norm_quant(x.to(DEV), bits=8, kind=kind, eps=EPS), want, size)
        _equal4(*cr.norm_quant(x.to(DEV), bits=4, kind=kind, eps=EPS), want, size)


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


def test_tiny_rows():
    """Rows whose scale leaves fp32's normal range still have the codes of their quotients."""
    w = torch.full((512,), 2.0 ** -118) * (1 + torch.arange(512) % 7)
    x = _x(_gen(5), 4, 512, BF16)
    n = O.norm(_np(x), "rms", EPS, _np(w))
    for f in (1.0, 2.0 ** -8, 2.0 ** -12, 2.0 ** -16, 2.0 ** -20, 2.0 ** -23):
        how = dict(kind="rms", eps=EPS, weight=w.to(DEV), scale=torch.full((1, 512), f - 1.0).to(DEV))
        _equal8(*cr.norm_quant(x.to(DEV), bits=8, **how), n * f, np.abs(n))
        _equal4(*cr.norm_quant(x.to(DEV), bits=4, **how), n * f, np.abs(n))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [40, 768, 4096])
def test_no_eps(d, dtype):
    """eps 0: rows of any size come out alike, also those whose squares vanish in fp32."""
    x = _x(_gen(7, d), 3, d, dtype)
    small = [2.0 ** -14] if dtype is F16 else [2.0 ** -60, 2.0 ** -100]
    for f in (1.0, *small):
        y = (x.double() * f).to(dtype)
        want = O.norm(_np(y), "layer", 0.0)
        _close(cr.norm(y.to(DEV), eps=0.0), want, np.abs(want) + 2)


@pytest.mark.parametrize("eps", [1e-6, 1e-20, 1e-30, 1e-38, 1e-44])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [24, 512, 4096])
def test_rows_without_spread(d, dtype, eps):
    """Rows of one value of any size give 0 with any eps above 0, and their rms norm a row of one value."""
    big = 6e4 if dtype is F16 else 1e30
    x = torch.tensor([0.0, 1.0, -3.140625, 2.0 ** -14, big, -big, 0.01])[:, None].expand(-1, d).contiguous().to(dtype).to(DEV)
    zero = torch.zeros_like(x)
    assert not cr.norm(x, eps=eps).any()
    h, n = cr.residual_norm(x, zero, eps=eps, post="layer", post_eps=eps)
    assert torch.equal(h, x) and not n.any()
    v = _np(x)
    want = v / np.sqrt(v * v + max(eps, 2.0 ** -126))
    for n in (cr.norm(x, kind="rms", eps=eps), cr.residual_norm(x, zero, kind="rms", eps=eps)[1]):
        _close(n, want, np.abs(want))


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

    _equal4(q, s, *c.normed(_np(c.x)))
    xv, wv = MX.values(*MX.unpack(_np(q), _np(s))), MX.values(*MX.unpack(_np(q1), _np(s1)))
    wy, terms = MX.product(xv, wv)
    h16 = torch.finfo(BF16).eps / 2                     # the product's bound: half a step, 2^-8 of a value, and its sums
    assert (np.abs(_np(y) - wy) <= h16 * np.abs(wy) + 1028 * 2.0 ** -23 * terms + 2.0 ** -133).all()
    c.y = y
    want = c.h(None, 1.0)
    _close(h, want, np.abs(want) + 100)
    n, size = c.normed(want)
    _equal8(a, b, n, size + c.h_size(want) / np.sqrt((want * want).mean(1, keepdims=True) + EPS))
    sums = (_np(a).astype(np.float64) @ _np(q2).astype(np.float64).T).astype(np.float32)
    wz = sums * (_np(b).astype(np.float32)[:, None] * _np(s2).astype(np.float32))
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
