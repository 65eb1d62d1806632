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
