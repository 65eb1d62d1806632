"""Rows of 16 bits out that go wrong more easily than others, against 64 bits.

The arithmetic is fp32: mu + e is within 2^-19 of the spread of the row's mean (e is
the mean of differences, whose sum passes at most 29 additions), r within 2^-19, an
element has up to 6 more roundings: with T the sizes that meet in it after the
mean is taken out, |d| <= h |n| + tiny + 2^-18 T (h half a step of the type, tiny half
of its smallest).
"""

import numpy as np
import pytest
import torch

import rotation_quantized_int8_amd as cr
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
    return t.detach().to(torch.float64).cpu().numpy()


def _close(got, want, size, what=""):
    h = torch.finfo(got.dtype).eps / 2
    tiny = {F16: 2.0 ** -25, BF16: 2.0 ** -134}[got.dtype]
    err, bound = np.abs(_np(got) - want), h * np.abs(want) + tiny + 2.0 ** -18 * size
    at = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), (what, at, err[at], bound[at], want[at])


SIZES = [24, 1000, 1003, 2048, 4096, 8200, 16384]


def _far(d, dtype):
    """Rows whose mean is far above their spread: steps of the type near a large value."""
    gen = torch.Generator().manual_seed(d)
    big, step = (60000.0, 32.0) if dtype is F16 else (2.0 ** 20 + 2.0 ** 15, 2.0 ** 13)
    x = torch.full((6, d), big, dtype=torch.float64)
    x[0, d // 2] += step
    x[1, 0] += step
    x[2, ::2] += step
    x[3] += step * torch.randint(-2, 3, (d,), generator=gen)
    x[4] = -x[0]
    x[5, -1] -= step
    assert x.to(dtype).double().equal(x)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", SIZES)
def test_mean_far_above_the_spread(d, dtype):
    x = _far(d, dtype)
    want = O.norm(_np(x), "layer", EPS)
    _close(cr.norm(x.to(DEV), eps=EPS), want, np.abs(want) + 1)
    zero = torch.zeros_like(x)
    h, n = cr.residual_norm(zero.to(DEV), x.to(DEV), kind="layer", eps=EPS, post="layer", post_eps=EPS)
    _close(h, want, np.abs(want) + 1, "h")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", SIZES)
def test_residual_whose_mean_is_far_above_its_spread(d, dtype):
    """h exact in fp32: a value of few bits and steps of 2^-4 and less next to 2^14."""
    gen = torch.Generator().manual_seed(d + 1)
    x = torch.full((3, d), 2.0 ** 14)
    y = torch.zeros((3, d))
    y[0, d // 3] = 2.0 ** -4
    y[1] = torch.randint(-8, 9, (d,), generator=gen) * 2.0 ** -6
    y[2, ::3] = 2.0 ** -8
    v = x.double().numpy() + y.double().numpy()
    want = O.norm(v, "layer", 1e-12)
    h, n = cr.residual_norm(x.to(dtype).to(DEV), y.to(dtype).to(DEV), eps=1e-12)
    # a row whose spread is that of one step has its mean within 2^-20 of a step
    spread = np.sqrt(v.var(1, keepdims=True) + 1e-12)
    _close(n, want, np.abs(want) + 1 + np.abs(y.numpy()).max(1, keepdims=True) / spread)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", SIZES)
def test_any_size_of_row_without_eps(d, dtype):
    """Rows of the type's smallest and largest values, far means and none, under eps 0."""
    gen = torch.Generator().manual_seed(d + 2)
    base = torch.randn((4, d), generator=gen, dtype=torch.float64)
    base[2:] += 64
    for f in ((2.0 ** -14, 1.0, 2.0 ** 9) if dtype is F16 else (2.0 ** -118, 2.0 ** -64, 1.0, 2.0 ** 40, 2.0 ** 119)):
        x = (base * f).to(dtype)
        want = O.norm(_np(x), "layer", 0.0)
        _close(cr.norm(x.to(DEV), eps=0.0), want, np.abs(want) + 1, f)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("d", [40, 1024, 4099, 8192])
def test_not_finite_as_the_formula_has_it(d, kind, dtype):
    """A NaN makes its row's statistics and so the whole row NaN; an infinity makes r 0 (rms) or the mean infinite."""
    gen = torch.Generator().manual_seed(d + 3)
    x = torch.randn((5, d), generator=gen).to(dtype)
    x[1, d // 2], x[2, 3], x[3, 0] = float("nan"), float("inf"), float("-inf")
    n = cr.norm(x.to(DEV), kind=kind, eps=EPS).cpu()
    with np.errstate(invalid="ignore"):
        want = O.norm(_np(x), kind, EPS)
    assert torch.equal(torch.isnan(n), torch.from_numpy(np.isnan(want)))
    assert torch.isnan(n[1]).all() and not n[2:4].nan_to_num().any()
    y = torch.zeros_like(x).to(DEV)
    h, n2 = cr.residual_norm(x.to(DEV), y, kind=kind, eps=EPS)
    assert torch.equal(torch.isnan(n2).cpu(), torch.isnan(n)) and torch.equal(h.cpu().nan_to_num(), x.nan_to_num())
    h, n3 = cr.residual_norm(y, x.to(DEV), kind=None, post=kind, post_eps=EPS)
    assert n3 is None and torch.equal(torch.isnan(h).cpu(), torch.isnan(n))
    if d % 256 == 0:
        q, s = cr.norm_quant(x.to(DEV), bits=4, kind=kind, eps=EPS)
        assert (s[:, 1] == 255).all() and not q[1].any()
        q, s = cr.norm_quant(x.to(DEV), bits=8, kind=kind, eps=EPS)
        assert torch.isnan(s).tolist() == [False, True, True, True, False] and not q[1:4].any()


@pytest.mark.parametrize("m,d", [(600, 5000), (1030, 8190)])
def test_many_long_rows(m, d):
    """The variant of two units a lane and eight wavefronts a row."""
    gen = torch.Generator().manual_seed(m)
    x, y = (torch.randn((m, d), generator=gen).to(BF16) for _ in range(2))
    want = O.norm(_np(x), "layer", EPS)
    _close(cr.norm(x.to(DEV), eps=EPS), want, np.abs(want) + 1)
    v = _np(x) + O.norm(_np(y), "rms", EPS)
    h, n = cr.residual_norm(x.to(DEV), y.to(DEV), eps=EPS, post="rms", post_eps=EPS)
    _close(h, v, np.abs(v) + np.abs(_np(x)) + 1, "h")
    want = O.norm(v, "layer", EPS)
    _close(n, want, 3 * np.abs(want) + 10, "n")
    h2, _ = cr.residual_norm(x.to(DEV), y.to(DEV), kind=None, post="rms", post_eps=EPS)
    assert torch.equal(h2, h)


def test_more_rows_than_a_grid_of_1024_threads_each():
    """2^22 rows and one of 4104: every one is written (one row in memory, read with stride 0)."""
    m, d = (1 << 22) + 1, 4104
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 34 GB of GPU memory")
    x = torch.randn((1, d), generator=torch.Generator().manual_seed(1)).to(F16).to(DEV)
    out = torch.zeros((m, d), dtype=F16, device=DEV)
    cr.norm(x.expand(m, d), eps=EPS, out=out)
    want = O.norm(_np(x), "layer", EPS)
    _close(out[:1], want, np.abs(want) + 1)
    for a in range(0, m, 1 << 18):
        assert (out[a:a + (1 << 18)] == out[0]).all(), a
    del out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("post", ["layer", "rms"])
@pytest.mark.parametrize("m,d", [(5, 33), (3, 1001), (4, 2048), (2, 8200), (2100, 1000)])
def test_weight_and_bias_of_the_norm_of_y(m, d, post, dtype):
    gen = torch.Generator().manual_seed(1000 * m + d)
    x, y = (torch.randn((m, d), generator=gen).to(dtype) for _ in range(2))
    w, b = 1 + 0.2 * torch.randn((d,), generator=gen), torch.randn((d,), generator=gen)
    for weight, bias in ((w, b), (None, b), (w, None)):
        h, _ = cr.residual_norm(x.to(DEV), y.to(DEV), kind=None, residual_scale=0.5, post=post, post_eps=EPS,
                                post_weight=None if weight is None else weight.to(DEV),
                                post_bias=None if bias is None else bias.to(DEV))
        p = O.norm(_np(y), post, EPS, None if weight is None else _np(weight), None if bias is None else _np(bias))
        _close(h, 0.5 * _np(x) + p, np.abs(p) + np.abs(_np(x)) + 2 * np.abs(_np(b)) + 4)
