"""The 4-bit linear where its kernels' loops turn: bit for bit, or with the bound of
its products, |dy| <= h |y| + tiny + (K + 4) 2^-23 S, S the sum of the terms' sizes
(the products are exact in fp32, each of K + 1 additions errs by at most 2^-23 S;
h half a step of the output type, tiny half its smallest)."""

import numpy as np
import pytest
import torch

import rotation_quantized_int8_amd as cr
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


def _random4(gen, rows, k, low, high):
    return (torch.randint(0, 256, (rows, k // 2), generator=gen, dtype=torch.uint8).to(DEV),
            torch.randint(low, high, (k // 256, rows, 8), generator=gen, dtype=torch.uint8).to(DEV))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("low,high", [(100, 121), (105, 136)])
def test_dequantize_rounds_to_fp32_and_then_to_the_type(low, high, dtype):
    """Groups whose scales are far apart: some of their values round otherwise at once."""
    q, s = _random4(torch.Generator().manual_seed(high), 1000, 1024, low, high)
    exact = O.dequantize(*O.unpack(_np(q), _np(s)))
    want = torch.from_numpy(exact.astype(np.float32)).to(dtype)
    assert torch.equal(cr.mx_dequantize(q, s, dtype).cpu(), want)
    if dtype is F16:
        assert (exact.astype(np.float16) != want.numpy()).any()


def _values(q, s):
    return torch.from_numpy(O.values(*O.unpack(_np(q), _np(s)))).to(DEV)


# by tile: sizes that take it, and slices (of 256) before, at and past the depth of its ring, odd and even
TILES = [(4100, 4200, (1, 2, 3, 4, 5, 8)),        # 256 x 256, two stages
         (2305, 2817, (1, 2, 3, 4, 5, 8)),        # 128 x 128, two stages
         (2049, 1030, (1, 2, 3, 4, 5, 6, 9, 10)),  # 128 x 64, three stages
         (777, 1003, (1, 3, 4, 5, 6, 9, 10))]     # 64 x 64, four stages


@pytest.mark.parametrize("m,n,slices", [(m, n, g) for m, n, all_of in TILES for g in all_of])
def test_product_over_slices(m, n, slices):
    """Every output of every tile, with ragged edges."""
    k = 256 * slices
    gen = torch.Generator().manual_seed(1000 * m + slices)
    (qx, sx), (qw, sw) = _random4(gen, m, k, 120, 126), _random4(gen, n, k, 118, 124)
    bias = torch.randn((n,), generator=gen).to(DEV)
    x, w = _values(qx, sx), _values(qw, sw)
    want, size = x @ w.t(), x.abs() @ w.abs().t()
    for dtype in (F16, BF16):
        res = torch.randn((m, n), generator=gen).to(dtype).to(DEV)
        for b, r in ((None, None), (bias, res)):
            y = cr.mx_gemm(qx, sx, qw, sw, bias=b, residual=r, out_dtype=dtype).double()
            v, t = want, size
            if b is not None:
                v, t = v + b.double() + r.double(), t + b.double().abs() + r.double().abs()
            tiny = {F16: 2.0 ** -25, BF16: 2.0 ** -134}[dtype]
            bound = torch.finfo(dtype).eps / 2 * v.abs() + tiny + (k + 4) * 2.0 ** -23 * t
            assert ((y - v).abs() <= bound).all(), (dtype, b is not None, ((y - v).abs() / bound).max())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m,k", [(8195, 2048), (1029, 8192), (65551, 256), (70, 131072)])
def test_activations_past_the_resident_groups(m, k, dtype):
    """More groups than workgroups in work hold: the same bits as few rows at a time, and the oracle's."""
    gen = torch.Generator().manual_seed(m)
    x = torch.randn((m, k), generator=gen)
    x[:, ::83] *= 20
    x = x.to(dtype).to(DEV)
    q, s = cr.mx_act_quant(x)
    step = max(1, 4096 * 256 // k)                  # 4096 groups a call: no workgroup takes a second
    for a in range(0, m, step):
        q1, s1 = cr.mx_act_quant(x[a:a + step].contiguous())
        assert torch.equal(q[a:a + step], q1) and torch.equal(s[:, a:a + step], s1), a
    some = torch.tensor([0, 1, m // 2, m - 2, m - 1])
    want = O.pack(*O.quantize(O.rotate_f32(_np(x[some.to(DEV)]))))
    assert np.array_equal(_np(q)[some], want[0]) and np.array_equal(_np(s)[:, some], want[1])
