"""What the bounds of test_kv_precision_gpu.py tell apart, without a GPU: the
attention kernels' roundings in numpy pass them, and mistakes planted there do not.
"""

from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import kv_oracle as O
from test_kv_precision_gpu import F16, _check


def _cache(k, v, bits):
    """A cache on the host, one head, pages of 16, page i at place i."""
    n, d = k.shape
    parts = []
    for x in (k, v):
        c, s = O.quantize(np.pad(x, ((0, -n % 16), (0, 0))), bits)
        parts += [torch.from_numpy(O.pack(c, bits)).view(-1, 1, 16, d * bits // 8), torch.from_numpy(s).view(-1, 1, 16)]
    pages = parts[0].shape[0]
    return SimpleNamespace(k_codes=parts[0], k_scale=parts[1], v_codes=parts[2], v_scale=parts[3], pages=pages, heads=1,
                           page_size=16, head_dim=d, bits=bits), torch.arange(pages, dtype=torch.int32)[None]


def _emulate(cache, q, m, scale, few, weights=2, queries=2, shared=False):
    """The outputs of fp16 queries [n, D] over m tokens, not causal; weights, queries: fp16 numbers of each."""
    d = q.shape[1]
    c, s = [], []
    for codes, scales in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        c.append(O.unpack(codes.reshape(-1, codes.shape[-1]).numpy(), cache.bits)[:m].astype(np.float64))
        s.append(scales.reshape(-1).numpy()[:m].astype(np.float64))
    x = (q.double().numpy() @ O.signs(d)).astype(np.float32).astype(np.float64)
    top = np.abs(x).max(-1, keepdims=True)
    if few:
        x = np.rint(x * (32512 / top)) * (top / 32512)
    else:
        unit = 2.0 ** (np.floor(np.log2(top.max() if shared else top)) + (1 if shared else -9))
        y = x / unit
        z = y.astype(np.float16).astype(np.float64)
        if queries == 2:
            z += (y - z).astype(np.float16)
        x = z * unit
    score = (x @ c[0].T) * s[0] * (scale * d ** -0.5 * np.log2(np.e))
    best = (score + np.log2(s[1])).max(-1, keepdims=True)
    p = 2.0 ** (score - best + 8)
    w = p * s[1]
    r = w.astype(np.float16).astype(np.float64)
    if weights == 2:
        r += (w - r).astype(np.float16)
    o = (r @ c[1]) / p.sum(-1, keepdims=True) @ O.signs(d) * d ** -0.5
    return torch.from_numpy(o).to(F16)[:, None]


def _passes(cache, table, q, m, got, scale):
    try:
        _check(cache, q[:, None], table, [len(q)], [m], False, got, scale=scale)
    except AssertionError:
        return False
    return True


@pytest.mark.parametrize("d,bits", [(64, 4), (128, 8), (256, 4)])
def test_one_fp16_number_for_weights_is_seen(d, bits):
    m = 400
    k, v = np.zeros((m, d)), np.full((m, d), np.float16(1.99), dtype=np.float64)
    k[0, 0] = 1.0
    cache, table = _cache(k, v, bits)
    q = torch.zeros((3, d), dtype=F16)
    q[:, 0] = 1.0
    seen = []
    for part in (0.9, -0.9, 0.5, -0.5):
        scale = float(np.log(2.0 / (1.0 + part * 2.0 ** -11)))
        assert _passes(cache, table, q, m, _emulate(cache, q, m, scale, True), scale)
        seen.append(not _passes(cache, table, q, m, _emulate(cache, q, m, scale, True, weights=1), scale))
    assert any(seen)


@pytest.mark.parametrize("d,bits", [(64, 4), (64, 8), (128, 4), (128, 8)])
def test_one_fp16_number_for_queries_is_seen(d, bits):
    rows, scale = 140, 1.0 / 15.0
    k, v = np.zeros((2, d)), np.random.default_rng(d).normal(size=(2, d))
    k[0, 0], k[1, 1] = 1.0, np.float16(1501.0 / 600.0)
    cache, table = _cache(k, v, bits)
    q = torch.zeros((rows, d))
    q[:, 0], q[:, 1] = 1501.0 + 2.0 * (torch.arange(rows) % 8), 600.0
    q = q.half()
    assert _passes(cache, table, q, 2, _emulate(cache, q, 2, scale, False, weights=1), scale)
    assert not _passes(cache, table, q, 2, _emulate(cache, q, 2, scale, False, weights=1, queries=1), scale)


@pytest.mark.parametrize("bits", [4, 8])
def test_a_unit_shared_by_rows_is_seen(bits):
    rows, m, d = 140, 300, 128
    r = np.random.default_rng(bits)
    cache, table = _cache(r.normal(size=(m, d)), r.normal(size=(m, d)), bits)
    q = torch.from_numpy(r.normal(size=(rows, d)) * 2.0 ** -7)
    q[5] *= 2.0 ** 20
    q = q.half()
    scale = 2.0 ** 7 * d ** -0.5
    assert _passes(cache, table, q, m, _emulate(cache, q, m, scale, False, weights=1), scale)
    assert not _passes(cache, table, q, m, _emulate(cache, q, m, scale, False, weights=1, shared=True), scale)


@pytest.mark.parametrize("few", [True, False])
def test_the_sign_of_the_scale_is_seen(few):
    rows, m, d = 140 if not few else 100, 200, 64
    r = np.random.default_rng(3)
    cache, table = _cache(r.normal(size=(m, d)), r.normal(size=(m, d)), 8)
    q = torch.from_numpy(r.normal(size=(rows, d))).half()
    assert _passes(cache, table, q, m, _emulate(cache, q, m, -0.1, few), -0.1)
    assert not _passes(cache, table, q, m, _emulate(cache, q, m, 0.1, few), -0.1)
