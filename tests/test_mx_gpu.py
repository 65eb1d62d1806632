"""The 4-bit linear on the GPU against its oracle in 64 bits.

Codes, scales and the read-back are compared bit for bit.  A product is
compared on its operands' own codes, per element, with
  |dy| <= h |y| + tiny + (K + 4) 2^-23 S,
h = eps / 2 of the output type (its one rounding) and tiny half its smallest
step, S the sum of the terms' sizes (products, bias, residual): the products
are exact in fp32 (4 significant bits), K + 1 additions in an order that the
matrix cores choose err by at most 2^-23 S each, whether they round or cut.
"""

import numpy as np
import pytest
import torch

import rotation_quantized_int8_amd as cr
from oracle import convrot_oracle as base
from oracle import mx_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


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


def _x(gen, m, k, dtype):
    x = torch.randn((m, k), generator=gen)
    x[:, ::83] *= 20
    return x.to(dtype)


def _random4(gen, rows, k, low=110, high=130):
    """Codes and scales of any values that a file may hold."""
    return (torch.randint(0, 256, (rows, k // 2), generator=gen, dtype=torch.uint8).to(DEV),
            torch.randint(low, high, (k // 256, rows, 8), generator=gen, dtype=torch.uint8).to(DEV))


def _step(dtype):
    return {F16: 2.0 ** -25, BF16: 2.0 ** -134}[dtype]


def _check_product(y, want, size, k, dtype, what=""):
    h = torch.finfo(dtype).eps / 2
    err = np.abs(_np(y) - want)
    bound = h * np.abs(want) + _step(dtype) + (k + 4) * 2.0 ** -23 * size
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), (what, worst, err[worst], bound[worst], want[worst])


def _equal4(codes, scales, want):
    q, s = O.pack(*want)
    assert np.array_equal(_np(scales), s), np.argwhere(_np(scales) != s)[:4]
    assert np.array_equal(_np(codes), q), np.argwhere(_np(codes) != q)[:4]


# ------------------------------------------------------------------ quantisers

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,k", [(1, 256), (3, 512), (17, 768), (64, 2048), (5, 8192), (2, 131072)])
def test_activations_bit_exact(m, k, dtype):
    x = _x(_gen(1, m, k), m, k, dtype)
    _equal4(*cr.mx_act_quant(x.to(DEV)), O.quantize(O.rotate_f32(_np(x))))


@pytest.mark.parametrize("n,k", [(1, 256), (19, 512), (33, 2048), (4, 8192)])
def test_weights_bit_exact(n, k):
    w = torch.randn((n, k), generator=_gen(2, n, k)) * 0.02
    _equal4(*cr.mx_quantize_weights(w.to(DEV)), O.quantize(base.rotate_weights_f32(w.numpy())))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantise_by_hand(dtype):
    """Rows whose rotation is known: one element of 16 gives +-1 everywhere, ties and borders of the codes."""
    x = torch.zeros((9, 256))
    x[0, 0] = 16.0                                    # u = 1: e = -2, codes of 4
    x[1, 7] = -24.0                                   # u = -+1.5: e = -2, codes of 6
    x[2, 0] = 28.0                                    # 1.75 2^2 = 7: past 6
    signs = torch.from_numpy(base.hadamard256_pm1()).float()
    for r, u in ((3, [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]), (4, [-4, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5])):
        x[r] = (torch.tensor(u).repeat(32) @ signs) / 16      # exact in each type: few bits
    x[5, 0] = 2.0 ** -20
    x[6, 0] = -0.0
    x[7] = torch.arange(256) % 5 - 2.0
    if dtype is not F16:
        x[8, 3] = 2.0 ** -120
    q, s = (cr.mx_quantize_weights if dtype is F32 else cr.mx_act_quant)(x.to(dtype).to(DEV))
    _equal4(q, s, O.quantize(O.rotate_f32(x.to(dtype).double().numpy())))
    c, e = O.unpack(_np(q), _np(s))
    assert (O.decode(c[0]) == 4 * np.sign(O.decode(c[0]))).all() and (e[0] == 125).all()
    assert (np.abs(O.decode(c[2])) == 6).all()
    if x[3].to(dtype).float().equal(x[3]):
        assert O.decode(c[3])[:8].tolist() == [4, 0, 1, 1, 2, 2, 4, 4]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantise_extreme_sizes(dtype):
    """Scales down to the smallest and values that pass fp32."""
    gen = _gen(3)
    x = torch.randn((300, 256), generator=gen, dtype=torch.float64)
    x = (x * 2.0 ** (torch.arange(300, dtype=torch.float64)[:, None] - 150)).float().to(dtype)   # up to past fp32
    q, s = (cr.mx_quantize_weights if dtype is F32 else cr.mx_act_quant)(x.to(DEV))
    _equal4(q, s, O.quantize(O.rotate_f32(_np(x))))
    assert 0 in _np(s) and 255 in _np(s)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantise_not_finite_shows_in_its_group_alone(dtype, bad):
    x = torch.ones((3, 512)).to(dtype)
    x[1, 300] = bad
    q, s = (cr.mx_quantize_weights if dtype is F32 else cr.mx_act_quant)(x.to(DEV))
    s, v = _np(s), cr.mx_dequantize(q, s, BF16)
    assert (s[1, 1] == 255).all() and (s != 255).sum() == s.size - 8
    assert torch.isnan(v[1, 256:]).all() and torch.isfinite(v[1, :256]).all() and torch.isfinite(v[[0, 2]]).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,k", [(1, 256), (7, 768), (40, 2048)])
def test_dequantize_bit_exact(rows, k, dtype):
    q, s = _random4(_gen(4, rows, k), rows, k)
    want = torch.from_numpy(O.dequantize(*O.unpack(_np(q), _np(s))).astype(np.float32)).to(dtype)
    assert torch.equal(cr.mx_dequantize(q, s, dtype).cpu(), want)


@pytest.mark.parametrize("low,high", [(120, 121), (120, 132), (120, 133), (8, 20), (7, 19), (228, 239), (230, 240), (0, 254)])
def test_dequantize_spans_of_scales(low, high):
    """Groups whose scales lie close together, far apart and at either end, with blocks of zeros among them."""
    gen = _gen(14, low, high)
    q, s = _random4(gen, 50, 768, low, high + 1)
    q.view(50, 24, 16)[torch.rand((50, 24), generator=gen).to(DEV) < 0.2] = 0x80
    s[torch.rand(s.shape, generator=gen).to(DEV) < 0.3] = low
    s[:, 3, 2], s[:, 4, 1] = 0, 254
    q.view(50, 24, 16)[3, 2::8] = q.view(50, 24, 16)[4, 1::8] = 0
    got, held = cr.mx_dequantize(q, s, BF16), O.unpack(_np(q), _np(s))
    exact = O.dequantize(*held)
    with np.errstate(over="ignore", invalid="ignore"):
        want = torch.from_numpy(exact.astype(np.float32)).to(BF16)
    if high - low <= 45:
        assert torch.equal(got.cpu().nan_to_num(), want.nan_to_num())
    else:   # past 45 binades the fp64 sums round: 8 additions, each 2^-53 of what has met so far
        size = np.abs(O.values(*held)).reshape(50, 3, 256).sum(-1).repeat(256, 1) / 16
        fits = np.abs(exact) < 3e38
        err = np.abs(_np(got) - exact)[fits]
        assert (err <= (2.0 ** -8 * np.abs(exact) + 2.0 ** -50 * size + _step(BF16))[fits]).all()


def test_dequantize_extreme_scales():
    s = torch.arange(256, dtype=torch.uint8)[None, :, None].expand(1, 256, 8).contiguous().to(DEV)
    q = torch.full((256, 128), 0xF7, dtype=torch.uint8, device=DEV)            # 6, -6
    v = O.dequantize(*O.unpack(_np(q), _np(s)))
    with np.errstate(over="ignore", invalid="ignore"):
        want = torch.from_numpy(v.astype(np.float32)).to(BF16)
    got = cr.mx_dequantize(q, s, BF16).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(), want.nan_to_num())


# ------------------------------------------------------------------- products

SIZES = [(1, 16, 256), (1, 1, 256), (1, 2048, 2048), (3, 40, 512), (16, 64, 768), (17, 33, 256), (24, 1000, 2048),
         (32, 16, 8192), (33, 64, 256), (64, 64, 512), (65, 63, 768), (100, 130, 1024), (128, 2048, 256),
         (200, 1003, 768), (777, 1003, 768), (1024, 256, 2048), (2049, 1030, 512), (4100, 4200, 256)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(m, n, k, dtype):
    gen = _gen(5, m, n, k)
    (qx, sx), (qw, sw) = _random4(gen, m, k, 120, 126), _random4(gen, n, k, 118, 124)
    bias = torch.randn((n,), generator=gen).to(DEV)
    res = torch.randn((m, n), generator=gen).to(dtype).to(DEV)
    y = cr.mx_gemm(qx, sx, qw, sw, bias=bias, residual=res, out_dtype=dtype)
    plain = cr.mx_gemm(qx, sx, qw, sw, out_dtype=dtype)
    rows = np.arange(m) if m * n * k < 1 << 28 else np.unique(np.r_[0:8, m // 2:m // 2 + 8, m - 8:m, 250:262])
    x = O.values(*O.unpack(_np(qx), _np(sx)))[rows]
    w = O.values(*O.unpack(_np(qw), _np(sw)))
    _check_product(y[rows], *O.product(x, w, _np(bias), _np(res)[rows]), k, dtype, "extras")
    _check_product(plain[rows], *O.product(x, w), k, dtype, "plain")
    if len(rows) < m:                                  # the rest: equal rows give equal rows
        q2, s2 = qx.flip(0).contiguous(), sx.flip(1).contiguous()
        assert torch.equal(cr.mx_gemm(q2, s2, qw, sw, out_dtype=dtype).flip(0), plain)


@pytest.mark.parametrize("m", [1, 20, 40, 300])
def test_product_one_hot(m):
    """Each output one product: rows, columns, blocks and scales meet as they should, exactly."""
    k, n = 1024, 1024
    qx = torch.zeros((m, k // 2), dtype=torch.uint8)
    sx = torch.full((k // 256, m, 8), 127, dtype=torch.uint8)
    hot = (torch.arange(m) * 37 + 5) % k
    for i, h in enumerate(hot.tolist()):
        qx[i, h // 2] = 2 if h % 2 == 0 else 0x20       # 1.0
        sx[h // 256, i, (h % 256) // 32] = 127 + i % 5
    gen = _gen(6, m)
    qw, sw = _random4(gen, n, k, 122, 130)
    y = _np(cr.mx_gemm(qx.to(DEV), sx.to(DEV), qw, sw))
    w = O.values(*O.unpack(_np(qw), _np(sw)))
    assert np.array_equal(y, (w[:, hot.numpy()] * 2.0 ** (np.arange(m) % 5)).T)


@pytest.mark.parametrize("m", [2, 50, 300])
def test_product_nan_scale_shows_in_its_row_alone(m):
    gen = _gen(7, m)
    (qx, sx), (qw, sw) = _random4(gen, m, 512), _random4(gen, 100, 512)
    sx[1, m - 1, 3] = 255
    sw[0, 7, 0] = 255
    qx.view(m, -1)[m - 1, 128 + 48:128 + 64] = 0       # as the quantiser leaves such a block
    y = cr.mx_gemm(qx, sx, qw, sw, out_dtype=BF16)
    nan = torch.zeros((m, 100), dtype=torch.bool)
    nan[m - 1], nan[:, 7] = True, True
    assert torch.equal(torch.isnan(y).cpu(), nan)


@pytest.mark.parametrize("m", [4, 200])
def test_product_extreme_scales(m):
    """2^-127 times 2^127 and the like: a scale is a power of two at either end of its range."""
    qx = torch.full((m, 128), 0x22, dtype=torch.uint8, device=DEV)             # 1.0
    qw = torch.full((64, 128), 0x22, dtype=torch.uint8, device=DEV)
    for a, b, want in ((0, 254, 256.0), (254, 0, 256.0), (127, 127, 256.0), (30, 100, 256.0 * 2.0 ** -124)):
        sx = torch.full((1, m, 8), a, dtype=torch.uint8, device=DEV)
        sw = torch.full((1, 64, 8), b, dtype=torch.uint8, device=DEV)
        y = _np(cr.mx_gemm(qx, sx, qw, sw, out_dtype=BF16))
        assert (y == want).all(), (a, b, y.ravel()[:2], want)


@pytest.mark.parametrize("m", [1, 24, 300])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_linear_is_its_stages(m, dtype):
    gen = _gen(8, m)
    x = _x(gen, m, 1024, dtype).view(1, m, 1024)
    qw, sw = cr.mx_quantize_weights((torch.randn((200, 1024), generator=gen) * 0.02).to(DEV))
    bias = torch.randn((200,), generator=gen).to(DEV)
    other = BF16 if dtype is F16 else F16
    y = cr.mx_linear(x.to(DEV), qw, sw, bias=bias, out_dtype=other)
    assert y.shape == (1, m, 200) and y.dtype is other
    staged = cr.mx_gemm(*cr.mx_act_quant(x.to(DEV)), qw, sw, bias=bias, out_dtype=other)
    assert torch.equal(y[0], staged)
    xv = O.values(*O.quantize(O.rotate_f32(_np(x[0]))))
    _check_product(y[0], *O.product(xv, O.values(*O.unpack(_np(qw), _np(sw))), _np(bias)), 1024, other)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 40, 256), (1, 1000, 8192), (4, 33, 2048), (16, 64, 512), (5, 17, 1536), (3, 16, 2560),
                                   (2, 16400, 4096)])
def test_one_launch_is_its_stages(m, n, k, dtype):
    """Few short rows: every workgroup quantises them itself, to the same bits."""
    gen = _gen(13, m, n, k)
    x = _x(gen, m, k, dtype).to(DEV)
    qw, sw = _random4(gen, n, k, 116, 122)
    res = torch.randn((m, n), generator=gen).to(dtype).to(DEV)
    want = cr.mx_gemm(*cr.mx_act_quant(x), qw, sw, residual=res, out_dtype=dtype)
    assert torch.equal(cr.mx_linear(x, qw, sw, residual=res), want)
    xv, wv = O.values(*O.quantize(O.rotate_f32(_np(x)))), O.values(*O.unpack(_np(qw), _np(sw)))
    _check_product(want, *O.product(xv, wv, None, _np(res)), k, dtype)


@pytest.mark.parametrize("m", [3, 24, 300, 2100])
def test_residual_in_place_and_out(m):
    gen = _gen(9, m)
    x, res = _x(gen, m, 512, F16).to(DEV), torch.randn((m, 1048), generator=gen).to(F16).to(DEV)
    qw, sw = _random4(gen, 1048, 512, 116, 120)
    want = cr.mx_linear(x, qw, sw, residual=res)
    ws = torch.empty(cr.mx_workspace_bytes(m, 1048, 512), dtype=torch.uint8, device=DEV)
    got = cr.mx_linear(x, qw, sw, residual=res, out=res, workspace=ws)
    assert got is res and torch.equal(res, want)


def test_empty_sizes():
    z = dict(dtype=torch.uint8, device=DEV)
    bias = torch.arange(5, dtype=F32, device=DEV)
    res = torch.full((3, 5), 0.5, dtype=F16, device=DEV)
    none = [torch.empty((r, 0), **z) for r in (3, 5)], [torch.empty((0, r, 8), **z) for r in (3, 5)]
    y = cr.mx_gemm(none[0][0], none[1][0], none[0][1], none[1][1], bias=bias, residual=res)
    assert torch.equal(y, (bias + 0.5).half().expand(3, 5))
    assert not cr.mx_linear(torch.empty((3, 0), dtype=F16, device=DEV), none[0][1], none[1][1]).any()
    qw, sw = _random4(_gen(10), 8, 256)
    assert cr.mx_linear(torch.empty((0, 256), dtype=BF16, device=DEV), qw, sw).shape == (0, 8)
    assert cr.mx_act_quant(torch.empty((0, 256), dtype=BF16, device=DEV))[0].shape == (0, 128)
    assert cr.mx_dequantize(torch.empty((0, 128), **z), torch.empty((1, 0, 8), **z)).shape == (0, 256)


@pytest.mark.parametrize("m", [1, 24, 700])
def test_graph_streams_and_repeats(m):
    """A captured linear replayed among eager ones, on another stream: the same bits each time."""
    gen = _gen(11, m)
    x = _x(gen, m, 2048, BF16).to(DEV)
    qw, sw = cr.mx_quantize_weights((torch.randn((520, 2048), generator=gen) * 0.02).to(DEV))
    want = cr.mx_linear(x, qw, sw)
    ws = torch.empty(cr.mx_workspace_bytes(m, 520, 2048), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cr.mx_linear(x, qw, sw, out=out, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            cr.mx_linear(x, qw, sw, out=out, workspace=ws)
        for _ in range(4):
            out.zero_()
            graph.replay()
            again = cr.mx_linear(x, qw, sw)
            side.synchronize()
            assert torch.equal(out, want) and torch.equal(again, want)
    torch.cuda.current_stream().wait_stream(side)


def test_views_and_strides():
    """Slices and transposes are copied as the other linears copy them."""
    gen = _gen(12)
    wide = _x(gen, 40, 1024, F16).to(DEV)
    x = wide[:, 256:768]
    qw, sw = _random4(gen, 48, 512, 118, 124)
    assert torch.equal(cr.mx_linear(x, qw, sw), cr.mx_linear(x.contiguous(), qw, sw))
    res = torch.randn((48, 40), generator=gen).half().to(DEV).t()
    assert torch.equal(cr.mx_linear(x, qw, sw, residual=res), cr.mx_linear(x, qw, sw, residual=res.contiguous()))
