"""Attention over the key/value cache against 64 bits, with the terms of the
kernel that runs (test_kv_gpu.py allows every kernel the roundings of all).

A score is off by at most  delta = |scale| max|k| (e + 2^-20 |q|)  (2-norms),
2^-20 for the fp32 arithmetic of a score and e for the rotated query as it
enters the matrix cores; with top = max |q W| of the row (W the +-1 matrix):
  up to 128 rows per key head: 16-bit fixed point of the row's own maximum,
          half a step of top / 32512, and fp32 butterflies:
          e = top / 65024 + 2^-21 sqrt(D) |q|;
  more rows, fp16: two fp16 numbers (2^-22, and the end of fp16's range, 2^-30
          of the row's maximum), and fp32 sums of the rotation:
          e = 2^-21 top + 2^-19 sqrt(D) |q|;
  more rows, bf16: one fp16 number: 2^-11 |q| more.
A weight is off, through itself and the sum, by 2 delta of itself, and by its
rounding: 2^-11 for one fp16 number, 2^-21 for two (fp16, up to 128 rows).
The sums over n tokens: up to 128 rows a wavefront adds 32 tokens at a time to
sums that hold the codes' offset (up to 15, or 255, where a row's codes have a
2-norm of at least 2, or 32, sqrt(D) in these tests: 8 times the value, 2^-23
each), 4 wavefronts and their join; more rows, 16 tokens at a time without an
offset.  With both,
  rel = expm1(2 delta) + rounding + (n / 128 + 16) 2^-20       (up to 128 rows)
  rel = expm1(2 delta) + rounding + (n / 16 + 64) 2^-22        (more).
H keeps 2-norms, so the error of an output row before its own rounding has a
2-norm of at most rel sum_j p_j |v_j|, and so has each element; the rounding
adds half a step of the output, to an element and in the 2-norm.
"""

import numpy as np
import pytest
import torch

import rotation_quantized_int8_amd as cr
from oracle import kv_oracle as O
from test_kv_gpu import BF16, DEV, F16, _check_attention, _gen, _host_rows, _np, _random_cache, _say, _sequences

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cr.lib()
    torch.cuda.set_device(0)


def _half_step(x, dtype):
    """Half the distance of dtype's neighbours at |x|."""
    f = torch.finfo(dtype)
    return 2.0 ** np.floor(np.log2(np.maximum(np.abs(x), f.smallest_normal))) * f.eps / 2


def _check(cache, q, table, q_lens, kv_lens, causal, got, scale=None, tell=""):
    d, group = cache.head_dim, q.shape[1] // cache.heads
    scale = d ** -0.5 if scale is None else scale
    few, fp16 = max(q_lens) * group <= 128, q.dtype == F16
    at, worst = 0, 0.0
    for b, (n, m) in enumerate(zip(q_lens, kv_lens)):
        k, v, here = _host_rows(cache, table[b].cpu().numpy(), m)
        assert here.all()
        qb = _np(q[at:at + n])
        o, spread = O.attention(qb, k, v, scale, causal)
        size = np.linalg.norm(qb, axis=-1)
        top = np.abs(qb @ O.signs(d)).max(-1)
        if few:
            e = top / 65024 + 2.0 ** -21 * d ** 0.5 * size
        else:
            e = 2.0 ** -21 * top + 2.0 ** -19 * d ** 0.5 * size + (0.0 if fp16 else 2.0 ** -11 * size)
        delta = abs(scale) * (np.linalg.norm(k, axis=-1).max() if m else 0.0) * (e + 2.0 ** -20 * size)
        rel = np.expm1(np.minimum(2 * delta, 3.0)) + (2.0 ** -21 if few and fp16 else 2.0 ** -11)
        rel += (m / 128 + 16) * 2.0 ** -20 if few else (m / 16 + 64) * 2.0 ** -22
        room = rel * spread[..., 0]
        y = _np(got[at:at + n])
        assert np.isfinite(y).all(), tell
        off, step = np.abs(y - o), _half_step(y, got.dtype)
        for share in (off / (step + room[..., None]),
                      np.linalg.norm(off, axis=-1) / (np.linalg.norm(step, axis=-1) + room)):
            if share.size:
                worst = max(worst, float(share.max()))
                assert share.max() <= 1.0, (tell, b, n, m, float(share.max()), np.argwhere(share > 1.0)[:4].tolist())
        at += n
    _say("   largest share of the bound:", tell, round(worst, 3))


def _plain_table(m, page=16):
    return (torch.arange(-(-m // page), dtype=torch.int32, device=DEV)[None],
            torch.tensor([m], dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("dtype,loud", [(F16, 2.0 ** 6), (F16, 2.0 ** 12), (BF16, 2.0 ** 6), (BF16, 2.0 ** 12),
                                        (BF16, 2.0 ** 20), (BF16, 2.0 ** -20)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [40, 300])
def test_a_loud_row_leaves_its_neighbours_alone(rows, d, bits, dtype, loud):
    """One query row far above (or below) the others of its tile, in another query and another head."""
    _say("loud row", rows, d, bits, dtype, loud)
    g = _gen(d, bits, rows)
    m = 600
    cache = _random_cache(g, -(-m // 16), 16, 1, d, bits)
    table, lens = _sequences(g, cache, [m])
    q = torch.randn((rows // 2, 2, d), generator=g)
    q[7, 1] *= loud
    q = q.to(dtype).to(DEV)
    got = cr.kv_attention(cache, q, table, lens)
    assert got.isfinite().all()
    _check_attention(cache, q, table, [rows // 2], [m], True, got)
    _check(cache, q, table, [rows // 2], [m], True, got)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows", [40, 300])
def test_rows_of_all_sizes_in_one_tile(rows, bits, dtype):
    _say("rows of all sizes", rows, bits, dtype)
    g = _gen(bits, rows)
    m, d = 600, 128
    cache = _random_cache(g, -(-m // 16), 16, 1, d, bits)
    table, lens = _sequences(g, cache, [m])
    size = torch.exp2(torch.linspace(*((-8, 12) if dtype == F16 else (-20, 20)), rows))
    q = (torch.randn((rows, 1, d), generator=g) * size[torch.randperm(rows, generator=g)][:, None, None]).to(dtype)
    q[3] = 0
    q = q.to(DEV)
    got = cr.kv_attention(cache, q, table, lens, causal=False)
    _check_attention(cache, q, table, [rows], [m], False, got)
    _check(cache, q, table, [rows], [m], False, got)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows", [40, 140, 300])
def test_queries_whose_rounding_tells_two_keys_apart(rows, bits, d):
    """q = X e0 + Y e1 with X + Y odd above 2048, so that one fp16 number of the rotated query is off by 1, and keys
    along e0 and e1 whose scores, near 100, balance: with one number a weight would be off by a hundredth."""
    _say("queries' second number", rows, bits, d)
    g = _gen(rows, bits, d)
    table, lens = _plain_table(2)
    cache = cr.KVCache.empty(1, 16, 1, d, bits, DEV)
    k, v = torch.zeros((2, 1, d)), torch.randn((2, 1, d), generator=g)
    k[0, 0, 0], k[1, 0, 1] = 1.0, 1501.0 / 600.0
    cr.kv_append(cache, k.half().to(DEV), v.half().to(DEV), torch.arange(2, device=DEV))
    q = torch.zeros((rows, 1, d))
    q[:, 0, 0], q[:, 0, 1] = 1501.0 + 2.0 * (torch.arange(rows) % 8), 600.0
    q = q.half().to(DEV)
    got = cr.kv_attention(cache, q, table, lens, scale=1.0 / 15.0, causal=False)
    _check(cache, q, table, [rows], [2], False, got, scale=1.0 / 15.0)


@pytest.mark.parametrize("bits", [4, 8])
def test_many_even_tokens_in_one_workgroup(bits):
    """131072 tokens of equal scores, so many heads that a workgroup walks them all; 16 heads are compared.  The mean
    of the values is 1 / 362 of one, and the sums that hold the codes' offset are 8 (128) times one: restarted every
    64 steps of 32 tokens their rounding (2 products a step of at most 2^-24 of a sum that grows to 15, 255 times the
    weights, independent) comes to 3e-5 of the mean; 4 times that, and the output's own rounding, are allowed."""
    _say("many even tokens", bits)
    d, heads, page, m = 64, 1024, 256, 131072
    dev = torch.Generator(device=DEV)
    dev.manual_seed(bits)
    shape = (m // page, heads, page)
    if bits == 4:                                          # nibbles 9 .. 15, 0 .. 7
        v = torch.randint(0, 15, (*shape, d // 2), dtype=torch.uint8, device=DEV, generator=dev).add_(9).bitwise_and_(15)
        high = torch.randint(0, 15, (*shape, d // 2), dtype=torch.uint8, device=DEV, generator=dev).add_(9).bitwise_and_(15)
        v.bitwise_or_(high.mul_(16))
        del high
    else:
        v = torch.randint(-127, 128, (*shape, d), dtype=torch.int8, device=DEV, generator=dev)
    scale = torch.rand(shape, device=DEV, generator=dev).mul_(0.01).add_(0.01)
    cache = cr.KVCache(torch.zeros_like(v), scale, v, scale)
    table = torch.arange(m // page, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([m], dtype=torch.int32, device=DEV)
    got = cr.kv_attention(cache, torch.zeros((1, heads, d), dtype=F16, device=DEV), table, lens)
    h = torch.tensor(O.signs(d), device=DEV)
    for a in range(0, heads, 64):
        raw = v[:, a].reshape(m, -1)
        if bits == 4:
            b = raw.int()
            raw = torch.stack([((b & 15) ^ 8) - 8, ((b >> 4) ^ 8) - 8], -1).flatten(-2)
        mean = (raw.double() * scale[:, a].reshape(m, 1).double()).mean(0)
        o = ((mean[None] @ h)[0] / d ** 0.5).cpu()
        y = got[0, a].double().cpu()
        off, own, size = (y - o).norm().item(), (o.half().double() - o).norm().item(), o.norm().item()
        _say("   error", off / size, "of it the output's rounding", own / size)
        assert off <= (1.1 * own ** 2 + (2.0 ** -13 * size) ** 2) ** 0.5


@pytest.mark.parametrize("d,bits", [(64, 8), (128, 4), (256, 4)])
@pytest.mark.parametrize("rows,m", [(1, 90), (24, 90), (24, 900), (150, 210), (150, 900)])
def test_a_nan_shows_under_a_weight_of_nothing(rows, m, d, bits):
    """A value of NaN whose score lies 300 below the others': the queries that see it show it, the others do not."""
    _say("NaN far below", rows, m, d, bits)
    g = _gen(rows, m, d)
    table, lens = _plain_table(m)
    k, v = torch.randn((m, 1, d), generator=g) * 0.1, torch.randn((m, 1, d), generator=g)
    q = torch.randn((rows, 1, d), generator=g) * 0.1
    q[..., 0] = 10.0
    for at in (m - 1 - rows // 2, m - rows, 3):
        kk, vv = k.clone(), v.clone()
        kk[at, 0, 0], vv[at, 0, 5] = -30.0, float("nan")
        cache = cr.KVCache.empty(table.numel(), 16, 1, d, bits, DEV)
        cr.kv_append(cache, kk.half().to(DEV), vv.half().to(DEV), torch.arange(m, device=DEV))
        got = cr.kv_attention(cache, q.half().to(DEV), table, lens, scale=1.0)
        sees = m - rows + torch.arange(rows) >= at
        assert got[sees.to(DEV)].isnan().all()
        assert got[~sees.to(DEV)].isfinite().all()


@pytest.mark.parametrize("dtype,loud,key", [(F16, 2.0 ** 12, 2.0 ** 13), (BF16, 2.0 ** 25, 1.0), (BF16, 2.0 ** 28, 1.0),
                                            (BF16, -2.0 ** 32, 1.0), (BF16, 2.0 ** 60, 2.0 ** 20), (BF16, 2.0 ** 80, 2.0 ** -40)])
@pytest.mark.parametrize("d,bits", [(64, 8), (128, 4), (256, 8)])
@pytest.mark.parametrize("rows,m", [(1, 600), (24, 600), (40, 600), (300, 600), (2, 9000), (24, 5000), (200, 5000)])
def test_scores_past_the_steps_of_fp32(rows, m, d, bits, dtype, loud, key):
    """Scores so large that fp32 holds them in steps of more than 1: where the largest is clear of the others by more
    than the query's own rounding, its token has all the weight."""
    _say("large scores", rows, m, d, bits, dtype, loud, key)
    g = _gen(rows, d, bits)
    table, lens = _plain_table(m)
    cache = cr.KVCache.empty(table.numel(), 16, 1, d, bits, DEV)
    k, v = torch.randn((m, 1, d), generator=g) * key, torch.randn((m, 1, d), generator=g)
    v[::3] *= 2.0 ** -8
    cr.kv_append(cache, k.to(dtype).to(DEV), v.to(dtype).to(DEV), torch.arange(m, device=DEV))
    q = torch.randn((rows, 1, d), generator=g) * loud
    if rows > 1:
        q[rows // 2] /= loud                               # an ordinary row among them
    q = q.to(dtype).to(DEV)
    got = cr.kv_attention(cache, q, table, lens, causal=False)
    _check(cache, q, table, [rows], [m], False, got)
    got = _np(got)[:, 0]
    kk, vv, _ = _host_rows(cache, table[0].cpu().numpy(), m)
    s = _np(q)[:, 0] @ kk[:, 0].T * d ** -0.5
    size = np.linalg.norm(_np(q)[:, 0], axis=-1) * np.linalg.norm(kk[:, 0], axis=-1).max() * d ** -0.5
    order = np.sort(s, axis=-1)
    clear = (order[:, -1] - order[:, -2] > 2.0 ** -10 * size) & (size > 2.0 ** 22)
    assert rows < 3 or clear.sum() > rows // 2
    one = vv[s.argmax(-1), 0]                              # off by its weight's rounding to fp16 at most
    off = np.abs(got - one)
    assert (off <= _half_step(got, dtype) + 2.0 ** -11 * np.linalg.norm(one, axis=-1)[:, None])[clear].all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,bits", [(64, 8), (128, 4), (256, 4)])
@pytest.mark.parametrize("rows", [1, 24, 100, 150])
def test_scales_of_both_signs(rows, d, bits, dtype):
    _say("signs of the scale", rows, d, bits, dtype)
    g = _gen(rows, d)
    m = 500
    cache = _random_cache(g, -(-m // 16), 16, 1, d, bits)
    table, lens = _sequences(g, cache, [m])
    q = torch.randn((rows, 1, d), generator=g).to(dtype).to(DEV)
    for scale in (-0.1, 0.1, -0.01, 0.0):
        got = cr.kv_attention(cache, q, table, lens, scale=scale)
        _check(cache, q, table, [rows], [m], True, got, scale=scale, tell=str(scale))


@pytest.mark.parametrize("d,bits", [(64, 4), (128, 8), (256, 4)])
@pytest.mark.parametrize("rows", [1, 20, 128])
def test_weights_that_all_round_one_way(rows, d, bits):
    """One token's weight is twice the others', less 0.9 half steps of fp16, and all have one value: rounded once to
    fp16 the weights would cost an output of fp16 a step."""
    _say("weights that round one way", rows, d, bits)
    m = 400
    table, lens = _plain_table(m)
    cache = cr.KVCache.empty(table.numel(), 16, 1, d, bits, DEV)
    k, v = torch.zeros((m, 1, d)), torch.full((m, 1, d), 1.99)
    k[0, 0, 0] = 1.0
    cr.kv_append(cache, k.half().to(DEV), v.half().to(DEV), torch.arange(m, device=DEV))
    q = torch.zeros((rows, 1, d), dtype=F16)
    q[..., 0] = 1.0
    q = q.to(DEV)
    for part in (0.9, -0.9, 0.5, -0.5):
        scale = float(np.log(2.0 / (1.0 + part * 2.0 ** -11)))
        got = cr.kv_attention(cache, q, table, lens, scale=scale, causal=False)
        _check(cache, q, table, [rows], [m], False, got, scale=scale, tell=str(part))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_lowest_codes(d, bits):
    """Codes of -8 and -128, which kv_append does not write, in rows of nothing else and among others."""
    _say("lowest codes", d, bits)
    low = -8 if bits == 4 else -128
    r = np.random.default_rng(d)
    h = O.signs(d)
    c = np.stack([np.full(d, low), np.where(h[1] > 0, low, -low - 1), np.where(h[d - 1] < 0, low, -low - 1), h[3] * (low + 1)]
                 + list(r.integers(low, -low, (28, d)))).astype(np.int8)
    scale = r.uniform(0.01, 0.02, 32).astype(np.float32)
    raw = torch.from_numpy(O.pack(c, bits)).view(2, 1, 16, -1).to(DEV)
    scales = torch.from_numpy(scale).view(2, 1, 16).to(DEV)
    cache = cr.KVCache(raw, scales, raw.clone(), scales.clone())
    want = O.read_f32(c, scale)
    for dtype in (F16, BF16):
        for got in cr.kv_read(cache, torch.arange(32, device=DEV), dtype=dtype):
            assert torch.equal(got[:, 0].cpu(), torch.from_numpy(want).to(dtype))
    table, lens = _plain_table(32)
    for rows in (1, 40, 140):
        q = torch.randn((rows, 1, d), generator=_gen(rows, d)).half().to(DEV)
        got = cr.kv_attention(cache, q, table, lens, causal=False)
        _check(cache, q, table, [rows], [32], False, got)


@pytest.mark.parametrize("loud", [2.0 ** 22, 2.0 ** 26, 2.0 ** 31, -2.0 ** 31, 2.0 ** 50])
@pytest.mark.parametrize("d,bits", [(64, 8), (128, 4), (256, 4)])
@pytest.mark.parametrize("rows,m", [(1, 600), (5, 4336), (40, 600), (300, 600), (200, 5000)])
def test_large_scores_over_values_of_all_sizes(rows, m, d, bits, loud):
    """As above, bf16, with values whose sizes differ by 2^24: the largest score's token has all the weight."""
    _say("large scores, values of all sizes", rows, m, d, bits, loud)
    g = _gen(rows, d, bits, 7)
    table, lens = _plain_table(m)
    cache = cr.KVCache.empty(table.numel(), 16, 1, d, bits, DEV)
    k, v = torch.randn((m, 1, d), generator=g), torch.randn((m, 1, d), generator=g)
    v *= torch.exp2(torch.randint(-8, 17, (m, 1, 1), generator=g).float())
    cr.kv_append(cache, k.bfloat16().to(DEV), v.bfloat16().to(DEV), torch.arange(m, device=DEV))
    q = (torch.randn((rows, 1, d), generator=g) * loud).bfloat16().to(DEV)
    got = _np(cr.kv_attention(cache, q, table, lens, causal=False))[:, 0]
    assert np.isfinite(got).all()
    kk, vv, _ = _host_rows(cache, table[0].cpu().numpy(), m)
    s = _np(q)[:, 0] @ kk[:, 0].T * d ** -0.5
    size = np.linalg.norm(_np(q)[:, 0], axis=-1) * np.linalg.norm(kk[:, 0], axis=-1).max() * d ** -0.5
    order = np.sort(s, axis=-1)
    clear = order[:, -1] - order[:, -2] > 2.0 ** -10 * size
    assert rows < 8 or clear.sum() > rows // 2
    one = vv[s.argmax(-1), 0]
    # a weight of fp16 that is up to 2^24 below the largest possible is off by 2^-25 of that
    room = 2.0 ** -11 * np.linalg.norm(one, axis=-1) + 2.0 ** -33 * np.linalg.norm(vv[:, 0], axis=-1).max()
    off = np.abs(got - one)
    assert (off <= _half_step(got, BF16) + room[:, None])[clear].all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,bits", [(64, 8), (128, 4), (256, 8)])
@pytest.mark.parametrize("rows,m", [(5, 90), (40, 3000), (300, 90), (300, 3000)])
def test_a_query_without_finite_scores_shows_alone(rows, m, d, bits, dtype):
    """Queries with an infinity or a NaN, or whose rotation passes fp32, give NaN where they see a token, zeros where
    they see none, and leave the other rows as they are without them."""
    _say("queries that are not finite", rows, m, d, bits, dtype)
    g = _gen(rows, m, d)
    cache = _random_cache(g, -(-m // 16), 16, 1, d, bits)
    table, lens = _sequences(g, cache, [m])
    q = torch.randn((rows, 1, d), generator=g).to(dtype)
    clean = q.clone()
    bad = torch.zeros(rows, dtype=torch.bool)
    for i, value in enumerate((float("nan"), float("inf"), float("-inf"))):
        q[i + 1, 0, 5 * i] = value
        clean[i + 1] = 0
        bad[i + 1] = True
    if dtype == BF16:
        q[rows - 1] = 3e38
        clean[rows - 1] = 0
        bad[rows - 1] = True
    for causal in (True, False):
        got = cr.kv_attention(cache, q.to(DEV), table, lens, causal=causal).cpu()[:, 0]
        sees = torch.ones(rows, dtype=torch.bool) if not causal else m - rows + torch.arange(rows) >= 0
        assert got[bad & sees].isnan().all() and not got[~sees].any()
        fine = clean.to(DEV)
        want = cr.kv_attention(cache, fine, table, lens, causal=causal)
        _check(cache, fine, table, [rows], [m], causal, want)
        got[bad] = want[:, 0].cpu()[bad]
        _check(cache, fine, table, [rows], [m], causal, got[:, None].to(DEV))
