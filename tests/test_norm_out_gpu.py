"""Outputs given to the quantising norms, and the rows that they leave as they were."""

import pytest
import torch

import rotation_quantized_int8_amd as cr

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cr.lib()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [256, 2048, 16384])
def test_padding_rows_keep_what_the_outputs_held(d, bits):
    index = [1, -1, 0, 0, 7, 1, 1 << 30, -(1 << 31), 0]
    m, dead = len(index), torch.tensor([not 0 <= i < 2 for i in index], device=DEV)
    gen = torch.Generator().manual_seed(d + bits)
    x, y = (torch.randn((m, d), generator=gen).to(BF16).to(DEV) for _ in range(2))
    scale, shift, gate = (0.3 * torch.randn((3, 2, d), generator=gen)).to(BF16).to(DEV)
    how = dict(bits=bits, scale=scale, shift=shift, index=torch.tensor(index, dtype=torch.int32, device=DEV))

    def rows(s):                                    # scales by rows
        return s.transpose(0, 1) if bits == 4 else s

    q0, s0 = cr.norm_quant(x, **how)
    out = torch.full_like(q0, 77), torch.full_like(s0, 99)
    got = cr.norm_quant(x, out=out, **how)
    assert got[0] is out[0] and got[1] is out[1]
    assert (out[0][dead] == 77).all() and (rows(out[1])[dead] == 99).all()
    assert torch.equal(out[0][~dead], q0[~dead]) and torch.equal(rows(out[1])[~dead], rows(s0)[~dead])

    h0, q0, s0 = cr.residual_norm_quant(x, y, gate=gate, **how)
    h = torch.full_like(x, 5.0)
    out = h, torch.full_like(q0, 77), torch.full_like(s0, 99)
    got = cr.residual_norm_quant(x, y, gate=gate, out=out, **how)
    assert all(a is b for a, b in zip(got, out))
    assert (h[dead] == 5).all() and (out[1][dead] == 77).all() and (rows(out[2])[dead] == 99).all()
    assert torch.equal(h[~dead], h0[~dead]) and torch.equal(out[1][~dead], q0[~dead])
    assert torch.equal(rows(out[2])[~dead], rows(s0)[~dead])
    place = x.clone()
    got = cr.residual_norm_quant(place, y, gate=gate, out=(place, None, None), **how)
    assert got[0] is place and torch.equal(place[~dead], h0[~dead]) and torch.equal(place[dead], x[dead])
    place = y.clone()
    assert cr.residual_norm_quant(x, place, gate=gate, out=place, **how)[0] is place
    assert torch.equal(place[~dead], h0[~dead])


def test_refusals():
    x = torch.zeros((4, 512), dtype=BF16, device=DEV)
    q, s = cr.norm_quant(x, bits=4)
    for bad in ((q[:3], s), (q.int(), s), (q, s[:1]), (q, s.float()), (q.t().contiguous().t(), s), (q.cpu(), s)):
        with pytest.raises(ValueError, match="out's"):
            cr.norm_quant(x, bits=4, out=bad)
        with pytest.raises(ValueError, match="out's"):
            cr.residual_norm_quant(x, x, bits=4, out=(None, *bad))
    with pytest.raises(ValueError, match="out's h"):
        cr.residual_norm_quant(x, x, bits=4, out=(x[:2], q, s))
    wide = torch.zeros(4 * 512 + 16, dtype=torch.int8, device=DEV)
    with pytest.raises(ValueError, match="aligned"):
        cr.norm_quant(x, bits=8, out=(wide[8:8 + 2048].view(4, 512), None))
