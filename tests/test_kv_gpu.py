"""The key/value cache on the GPU against its oracle in 64 bits.

Codes and scales are compared bit for bit, and so is the read-back.  Attention
is compared on the cache's own codes, per element, with
  |do| <= h |o| + tiny + (2^-11 + 2 (2^-11 + 2^-20) S + (n + D) 2^-22) spread,
h = eps / 2 of the output type (its one rounding) and tiny half its smallest
step; spread = sum_j p_j |v_j| (2-norms; H keeps them, so an error of the
rotated elements reaches an element of the output at most by its norm):
  2^-11           a softmax weight rounded once to fp16 (weights that leave
                  fp16's normal range carry 2^-39 of the largest at most, in
                  the sum over n tokens inside the last term),
  2 * 2^-11 * S   the rotated query rounded once to fp16, S = scale |q| max |k|:
                  a score moves by at most 2^-11 S, and a weight, through
                  itself and the sum, by twice that (2^-20: fp32 scores),
  (n + D) 2^-22   fp32 sums over tokens and elements, in any order, and exp.
That holds for errors that all add up.  They are independent, so the 2-norm
over a call's outputs is also held to
  |do|_2 <= h |o|_2 + (2^-11 + 2^-11 2 S / sqrt(D) + (n + D) 2^-22) |even|_2,
even = sqrt(sum_j p_j^2 |v_j|^2): independent errors of the weights add in
squares, and of the rotated query, whose elements are all of one size, a score
takes S / sqrt(D) 2^-11; every term is a largest error where its standard
deviation, 1 / sqrt(3) of it, would do.
"""

import numpy as np
import pytest
import torch

import rotation_quantized_int8_amd as cr
from oracle import kv_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cr.lib()
    torch.cuda.set_device(0)


def _say(*a):
    print(*a, flush=True)


def _np(t):
    return t.detach().to(torch.float64).cpu().numpy() if t.is_floating_point() else t.detach().cpu().numpy()


def _values(gen, shape, dtype):
    """Rows with loud channels, as a model's keys have them."""
    x = torch.randn(shape, generator=gen)
    x[..., ::37] *= 8
    return x.to(dtype)


def _gen(*key):
    g = torch.Generator()
    g.manual_seed(hash(key) % (1 << 31))
    return g


def _bits32(a):
    return np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)


# ------------------------------------------------------------- write and read

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,heads,page", [(1, 1, 16), (37, 3, 32), (515, 2, 256)])
def test_append_and_read_bit_exact(tokens, heads, page, d, bits, dtype):
    _say("append/read", tokens, heads, page, d, bits, dtype)
    g = _gen(tokens, heads, page, d, bits)
    k, v = _values(g, (tokens, heads, d), dtype), _values(g, (tokens, heads, d), dtype)
    pages = -(-tokens // page) + 2
    cache = cr.KVCache.empty(pages, page, heads, d, bits, DEV)
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(0x55)
    cache.k_scale.fill_(-3.0)
    cache.v_scale.fill_(-3.0)
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    cr.kv_append(cache, k.to(DEV), v.to(DEV), slots.to(DEV))
    touched = np.zeros(pages * page, dtype=bool)
    touched[slots.numpy()] = True
    got = cr.kv_read(cache, slots.to(DEV), dtype=dtype)
    for x, codes, scale, back in ((k, cache.k_codes, cache.k_scale, got[0]), (v, cache.v_codes, cache.v_scale, got[1])):
        c, s = O.quantize(_np(x), bits)
        raw = codes.transpose(1, 2).reshape(pages * page, heads, -1).cpu().numpy()
        sc = scale.transpose(1, 2).reshape(pages * page, heads).cpu().numpy()
        assert np.array_equal(_bits32(sc[slots.numpy()]), _bits32(s))
        assert np.array_equal(raw[slots.numpy()], O.pack(c, bits))
        assert (raw[~touched] == 0x55).all() and (sc[~touched] == -3.0).all()
        want = torch.from_numpy(O.read_f32(c, s)).to(dtype)
        assert torch.equal(back.cpu(), want)


def _special_rows(d, dtype):
    x = torch.zeros((9, d))
    x[1, 3] = 1.0
    x[2] = 65504.0 if dtype == F16 else 1e30
    x[3, :2] = torch.tensor([65504.0, -65504.0])
    x[4] = 2.0 ** -24 if dtype == F16 else 2.0 ** -130   # subnormal steps
    x[5, 7] = float("inf")
    x[6, 7], x[6, 8] = float("inf"), float("-inf")
    x[7, 9] = float("nan")
    x[8] = torch.arange(d) % 15 - 7.0                    # small integers: ties
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_special_rows(d, bits, dtype):
    _say("special rows", d, bits, dtype)
    x = _special_rows(d, dtype)[:, None]
    cache = cr.KVCache.empty(1, 16, 1, d, bits, DEV)
    slots = torch.arange(9, device=DEV)
    cr.kv_append(cache, x.to(DEV), x.to(DEV).flip(0), slots)
    c, s = O.quantize(_np(x), bits)
    for codes, scale, order in ((cache.k_codes, cache.k_scale, 1), (cache.v_codes, cache.v_scale, -1)):
        got = scale[0, 0, :9].cpu().numpy()
        want = s[::order, 0]
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(_bits32(np.nan_to_num(got)), _bits32(np.nan_to_num(want)))
        assert np.array_equal(codes[0, 0, :9].cpu().numpy(), O.pack(c[::order, 0], bits))
    k, _ = cr.kv_read(cache, slots, dtype=dtype)
    assert torch.equal(k.cpu().isnan().all(-1)[:, 0], torch.from_numpy(np.isnan(s[:, 0])))


def test_append_strides_padding_and_bad_slots():
    _say("append strides, padding, bad slots")
    g = _gen(3)
    n, h, d = 40, 3, 128
    fused = _values(g, (n, 5 * h, d), F16).to(DEV)
    k, v = fused[:, h:2 * h], fused[:, 4 * h:]
    odd_k = torch.empty((n, h, d + 1), dtype=F16, device=DEV)[..., 1:].copy_(k)      # copied by the binding
    turned = v.transpose(0, 1).contiguous().transpose(0, 1)                           # heads outermost
    slots = torch.arange(n) * 2
    slots[5], slots[9], slots[11], slots[12] = -1, 96, -(1 << 40), 1 << 50
    kept = (slots >= 0) & (slots < 96)
    a, b = (cr.KVCache.empty(6, 16, h, d, 4, DEV) for _ in range(2))
    cr.kv_append(a, k, v, slots.to(DEV))
    cr.kv_append(b, odd_k, turned, slots.to(DEV))
    ka, va = cr.kv_read(a, slots.to(DEV))
    for x, y in ((a.k_codes, b.k_codes), (a.k_scale, b.k_scale), (a.v_codes, b.v_codes), (a.v_scale, b.v_scale)):
        assert torch.equal(x, y)
    for got, x in ((ka, k), (va, v)):
        c, s = O.quantize(_np(x), 4)
        want = torch.from_numpy(O.read_f32(c, s)).half()
        want[~kept] = 0
        assert torch.equal(got.cpu(), want)
    # a broadcast input: one row for every token
    one = _values(g, (1, h, d), F16).to(DEV).expand(n, h, d)
    cr.kv_append(a, one, one, torch.arange(n, device=DEV))
    k2, v2 = cr.kv_read(a, torch.arange(n, device=DEV))
    assert torch.equal(k2, k2[:1].expand(n, h, d)) and torch.equal(k2, v2)
    # into given outputs
    out = (torch.empty((n, h, d), dtype=F16, device=DEV), torch.empty((n, h, d), dtype=F16, device=DEV))
    assert cr.kv_read(a, torch.arange(n, device=DEV), out=out)[0] is out[0] and torch.equal(out[0], k2)


def test_empty_calls():
    cache = cr.KVCache.empty(2, 16, 2, 64, 4, DEV)
    none = torch.empty((0, 2, 64), dtype=F16, device=DEV)
    cr.kv_append(cache, none, none, torch.empty(0, dtype=torch.int64, device=DEV))
    assert cr.kv_read(cache, torch.empty(0, dtype=torch.int64, device=DEV))[0].shape == (0, 2, 64)
    table = torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    assert cr.kv_attention(cache, none, table, table[:, 0]).shape == (0, 2, 64)
    # sequences without a token, and a table without columns
    q = torch.ones((3, 2, 64), dtype=F16, device=DEV)
    for width in (0, 1):
        table = torch.zeros((3, width), dtype=torch.int32, device=DEV)
        o = cr.kv_attention(cache, q, table, torch.zeros(3, dtype=torch.int32, device=DEV))
        assert not o.any()


# ------------------------------------------------------------------- attention

def _random_cache(g, pages, page, heads, d, bits):
    cache = cr.KVCache.empty(pages, page, heads, d, bits, DEV)
    n = pages * page
    for codes, scale in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        c, s = O.quantize(_np(_values(g, (n, heads, d), F16)), bits)
        raw = torch.from_numpy(O.pack(c, bits)).view(pages, page, heads, -1).transpose(1, 2)
        codes.copy_(raw)
        scale.copy_(torch.from_numpy(s).view(pages, page, heads).transpose(1, 2))
    return cache


def _host_rows(cache, pages, kv):
    """Float64 keys and values [kv, heads, D] of a sequence, and which are present."""
    p = cache.page_size
    idx = np.arange(kv)
    page = np.asarray(pages)[idx // p]
    here = (page >= 0) & (page < cache.pages)
    page = np.where(here, page, 0)
    out = []
    for codes, scale in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        raw = codes[torch.from_numpy(page), :, torch.from_numpy(idx % p)].cpu().numpy()
        s = scale[torch.from_numpy(page), :, torch.from_numpy(idx % p)].cpu().numpy()
        out.append(O.rows(O.unpack(raw, cache.bits), s))
    return out[0], out[1], here


def _check_attention(cache, q, table, q_lens, kv_lens, causal, got, scale=None, tell=""):
    d = cache.head_dim
    scale = d ** -0.5 if scale is None else scale
    h = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * h
    at, worst, norms = 0, 0.0, np.zeros(2)
    for b, (n, m) in enumerate(zip(q_lens, kv_lens)):
        k, v, here = _host_rows(cache, table[b].cpu().numpy(), m)
        qb = _np(q[at:at + n])
        if here.all():
            o, spread = O.attention(qb, k, v, scale, causal)
        else:   # the positions count all tokens; the absent ones are left out
            o, spread = np.zeros(qb.shape), np.zeros((*qb.shape[:2], 2))
            for i in range(n):
                see = here & (np.arange(m) <= (m - n + i if causal else m))
                o[i:i + 1], spread[i:i + 1] = O.attention(qb[i:i + 1], k[see], v[see], scale, False)
        big = scale * np.linalg.norm(qb, axis=-1) * (np.linalg.norm(k, axis=-1).max() if m else 0.0)
        bound = h * np.abs(o) + tiny + ((2.0 ** -11 + 2 * (2.0 ** -11 + 2.0 ** -20) * big + (m + d) * 2.0 ** -22)
                                        * spread[..., 0])[..., None]
        off = np.abs(_np(got[at:at + n]) - o)
        even = (2.0 ** -11 * (1 + 2 * big / np.sqrt(d)) + (m + d) * 2.0 ** -22) * spread[..., 1]
        norms += [(off ** 2).sum(), (h * h * o ** 2).sum() + (even ** 2).sum() + o.size * tiny ** 2]
        if off.size:
            worst = max(worst, float((off / bound).max()))
        assert (off <= bound).all(), (b, n, m, float((off / bound).max()))
        at += n
    share = float(np.sqrt(norms[0] / norms[1])) if norms[1] else float(norms[0] > 0)
    _say("   largest share of the bound:", tell, round(worst, 3), "in the 2-norm:", round(share, 3))
    assert share <= 1.0


def _sequences(g, cache, kv_lens, spare=0):
    """Tables of distinct pages in random order."""
    p = cache.page_size
    need = [-(-m // p) for m in kv_lens]
    order = torch.randperm(cache.pages, generator=g)
    table, at = torch.full((len(kv_lens), max(need + [1]) + spare), -7, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.to(DEV), torch.tensor(kv_lens, dtype=torch.int32, device=DEV)


def _spoil_unused(cache, table, kv_lens):
    """NaN scales and arbitrary codes in every slot that no sequence holds."""
    p = cache.page_size
    used = torch.zeros(cache.pages * p, dtype=torch.bool)
    for b, m in enumerate(kv_lens):
        i = torch.arange(m)
        used[table[b].cpu().long()[i // p] * p + i % p] = True
    free = ~used.view(cache.pages, 1, p).to(DEV)
    for codes, scale in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        scale.masked_fill_(free, float("nan"))
        codes.masked_fill_(free[..., None], 0x77)


def _starts(q_lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device=DEV)


# (queries, cached tokens) of each sequence, key heads, group, head size, bits, dtype, page, causal
ATTENTION = [
    # single tokens: lengths around tile borders, zero and one
    ([1] * 8, [0, 1, 2, 15, 16, 17, 31, 33], 2, 1, 128, 4, F16, 16, True),
    ([1] * 6, [63, 64, 65, 127, 128, 130], 3, 4, 128, 4, BF16, 32, True),
    ([1] * 3, [255, 257, 512], 1, 8, 64, 4, F16, 64, True),
    ([1] * 3, [1, 300, 77], 2, 5, 256, 4, BF16, 16, True),
    ([1] * 3, [100, 0, 333], 2, 3, 64, 8, BF16, 32, True),
    ([1] * 4, [9, 48, 160, 401], 2, 2, 128, 8, F16, 128, True),
    ([1] * 2, [259, 1030], 1, 7, 256, 8, F16, 256, True),
    # one long sequence (split and joined), next to a short one and an empty one
    ([1, 1, 1], [9001, 40, 0], 2, 4, 128, 4, F16, 16, True),
    ([1], [20000], 1, 1, 64, 4, BF16, 64, True),
    ([1, 1], [5003, 4999], 1, 2, 256, 8, F16, 32, True),
    # groups of more than one tile of rows
    ([1, 1], [200, 31], 1, 17, 128, 4, F16, 16, True),
    ([1, 1], [500, 64], 1, 40, 64, 8, BF16, 16, True),
    # a few tokens at once
    ([2, 3, 4, 5], [100, 3, 4, 3000], 2, 4, 128, 4, F16, 16, True),
    ([3, 0, 1, 2], [64, 64, 1, 1], 1, 3, 256, 4, BF16, 32, True),
    # more queries than tokens: the first see none
    ([7, 40, 3], [2, 33, 0], 2, 2, 128, 4, F16, 16, True),
    ([300], [270], 1, 1, 64, 8, BF16, 16, True),
    # prompts and chunks
    ([33, 64], [33, 64], 2, 1, 128, 4, F16, 16, True),
    ([129, 1, 200], [129, 500, 900], 2, 2, 128, 4, BF16, 64, True),
    ([257], [257], 2, 3, 64, 4, F16, 32, True),
    ([130], [411], 1, 2, 256, 4, F16, 128, True),
    ([70, 90], [170, 90], 1, 5, 256, 8, BF16, 16, True),
    ([255, 17], [255, 1000], 1, 4, 128, 8, F16, 256, True),
    ([48], [6000], 1, 2, 128, 4, F16, 16, True),          # few rows, a long context: split
    # enough rows of 128 for workgroups of 256, lengths that leave tiles and groups of 16 part empty
    ([512, 499, 3, 290], [600, 499, 300, 777], 8, 4, 128, 4, BF16, 32, True),
    ([400, 513], [450, 100], 16, 4, 128, 8, F16, 16, False),
    # many rows over a longer context: split; rows around the border between the two kernels
    ([150, 141], [4000, 2222], 1, 2, 64, 4, F16, 16, True),
    ([150, 141], [4000, 2222], 1, 2, 128, 8, F16, 16, True),
    ([200, 130], [100, 128], 2, 2, 128, 4, BF16, 16, True),
    ([200, 130], [77, 1], 2, 2, 64, 4, F16, 32, False),
    ([700], [3000], 2, 2, 128, 4, BF16, 16, True),
    ([700], [3000], 2, 2, 64, 8, F16, 64, True),
    ([200, 130], [129, 2048], 1, 1, 64, 4, BF16, 16, False),
    ([128, 100], [300, 900], 2, 1, 128, 4, BF16, 16, True),
    ([129, 128], [300, 900], 2, 1, 256, 8, F16, 32, True),
    ([127, 33], [2000, 1029], 3, 1, 64, 8, F16, 16, False),
    # about a sequence and key head for each CU: workgroups of 16 wavefronts, single ones for a whole sequence
    ([1] * 20, [2040, 0, 1] + [97 * i + 13 for i in range(17)], 8, 2, 128, 4, F16, 32, True),
    ([2] * 26, [1500, 3, 1] + [53 * i for i in range(23)], 7, 2, 64, 8, BF16, 16, True),
    ([1] * 9, [1024, 1, 999, 1000, 31, 0, 512, 513, 768], 2, 3, 256, 8, F16, 64, True),
    ([9] * 40, [900 - 17 * i for i in range(40)], 4, 3, 128, 8, BF16, 16, True),
    # states of another length
    ([100, 64], [77, 1], 2, 1, 128, 4, F16, 16, False),
    ([1, 1, 5], [77, 513, 0], 2, 4, 64, 4, BF16, 32, False),
    ([260], [45], 1, 2, 256, 8, F16, 16, False),
    ([40, 0, 3], [0, 10, 200], 1, 6, 128, 8, BF16, 16, False),
]


@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention(case):
    q_lens, kv_lens, heads, group, d, bits, dtype, page, causal = ATTENTION[case]
    _say("attention", ATTENTION[case])
    g = _gen(case)
    cache = _random_cache(g, sum(-(-m // page) for m in kv_lens) + 2, page, heads, d, bits)
    table, lens = _sequences(g, cache, kv_lens, spare=1)
    _spoil_unused(cache, table, kv_lens)
    q = torch.randn((sum(q_lens), heads * group, d), generator=g).to(dtype).to(DEV)
    even = len(set(q_lens)) == 1
    got = cr.kv_attention(cache, q, table, lens, q_start=None if even else _starts(q_lens), causal=causal)
    _check_attention(cache, q, table, q_lens, kv_lens, causal, got, tell="default bounds")
    tight = cr.kv_attention(cache, q, table, lens, q_start=_starts(q_lens), max_q=max(q_lens), max_kv=max(kv_lens),
                            causal=causal)
    _check_attention(cache, q, table, q_lens, kv_lens, causal, tight, tell="tight bounds")


@pytest.mark.parametrize("batch", [63, 64, 65, 130, 256])
def test_attention_of_many_sequences(batch):
    """Units cut over all sequences: idle ones, short ones, a few long ones."""
    _say("many sequences", batch)
    g = _gen(batch, 11)
    kv_lens = [int(x) for x in torch.randint(0, 90, (batch,), generator=g)]
    kv_lens[0], kv_lens[batch // 2], kv_lens[-1], kv_lens[1] = 3000, 1700, 700, 0
    cache = _random_cache(g, sum(-(-m // 16) for m in kv_lens), 16, 2, 64, 4)
    table, lens = _sequences(g, cache, kv_lens)
    q = torch.randn((batch, 6, 64), generator=g).half().to(DEV)
    got = cr.kv_attention(cache, q, table, lens)
    _check_attention(cache, q, table, [1] * batch, kv_lens, True, got)
    # some sequences without a query, some with two
    q_lens = [int(x) for x in torch.randint(0, 3, (batch,), generator=g)]
    q = torch.randn((sum(q_lens), 6, 64), generator=g).half().to(DEV)
    got = cr.kv_attention(cache, q, table, lens, q_start=_starts(q_lens), max_q=2)
    _check_attention(cache, q, table, q_lens, kv_lens, True, got)


def test_attention_of_more_sequences_than_are_balanced():
    """Over 256 sequences and a wide table: fixed chunks of 2048 tokens, of 16384 where the heads fill the card."""
    for heads, most in ((1, 9001), (4, 33001)):
        _say("300 sequences", heads)
        _more_sequences(heads, most)


def _more_sequences(heads, most):
    g = _gen(12)
    kv_lens = [int(x) for x in torch.randint(0, 40, (300,), generator=g)]
    kv_lens[7] = most
    cache = _random_cache(g, sum(-(-m // 16) for m in kv_lens), 16, heads, 64, 8)
    table, lens = _sequences(g, cache, kv_lens)
    q = torch.randn((300, 3 * heads, 64), generator=g).bfloat16().to(DEV)
    got = cr.kv_attention(cache, q, table, lens)
    _check_attention(cache, q, table, [1] * 300, kv_lens, True, got)


@pytest.mark.parametrize("n,m,heads,d", [(1, 9001, 1024, 64), (3, 8700, 1100, 128), (40, 5003, 1600, 64),
                                         (36, 4500, 1100, 128), (33, 4300, 600, 256), (136, 4500, 600, 128),
                                         (140, 4300, 1600, 64), (133, 4100, 300, 256)])
def test_attention_walks_long_contexts_alone(n, m, heads, d):
    """So many heads that one workgroup walks a context past its 64 remembered pages; three heads are compared."""
    _say("long and alone", n, m, heads, d)
    g = _gen(n, m)
    page, pages = 16, -(-m // 16)
    dev = torch.Generator(device=DEV)
    dev.manual_seed(m)
    shape = (pages, heads, page)
    cache = cr.KVCache(*(f() for _ in range(2) for f in (
        lambda: torch.randint(0, 256, (*shape, d // 2), dtype=torch.uint8, device=DEV, generator=dev),
        lambda: torch.rand(shape, device=DEV, generator=dev) * 0.1)))
    for codes in (cache.k_codes, cache.v_codes):       # codes of -8 are not written by kv_append
        codes[(codes & 0xF) == 8] = 0
        codes[(codes >> 4) == 8] = 0
    table, lens = _sequences(g, cache, [m])
    q = torch.randn((n, heads, d), generator=g).half().to(DEV)
    got = cr.kv_attention(cache, q, table, lens, max_kv=m)
    some = torch.tensor([0, heads // 2 + 1, heads - 1])
    part = cr.KVCache(*(t[:, some].contiguous() for t in (cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale)))
    _check_attention(part, q[:, some], table, [n], [m], True, got[:, some])


@pytest.mark.parametrize("n,heads,group,d,batch", [(18, 512, 1, 64, 2), (17, 520, 1, 128, 2), (11, 448, 2, 64, 4),
                                                   (5, 1100, 1, 128, 3), (19, 300, 1, 256, 3), (20, 512, 1, 64, 2)])
@pytest.mark.parametrize("q_each", [False, True])
def test_attention_joins_rows_that_share_a_wavefront(n, heads, group, d, batch, q_each):
    """Units of equal work over unequal lengths, and so many rows that the join puts four into a wavefront: a tile's
    rows end inside one where their number is no multiple of four.  Three heads are compared."""
    _say("join of shared wavefronts", n, heads, group, d, batch, q_each)
    g = _gen(n, heads, d)
    kv_lens = [5003, 300, 2700, 1][:batch]
    pages = sum(-(-m // 16) for m in kv_lens)
    dev = torch.Generator(device=DEV)
    dev.manual_seed(n)
    shape = (pages, heads, 16)
    codes = [torch.randint(-7, 8, (*shape, d), dtype=torch.int8, device=DEV, generator=dev) for _ in range(2)]
    scales = [torch.rand(shape, device=DEV, generator=dev) * 0.1 for _ in range(2)]
    packed = [((c[..., 0::2] & 15) | (c[..., 1::2] << 4)).view(torch.uint8) for c in codes]
    cache = cr.KVCache(packed[0], scales[0], packed[1], scales[1])
    table, lens = _sequences(g, cache, kv_lens)
    q_lens = [n - (i % 3 if q_each else 0) for i in range(batch)]
    q = torch.randn((sum(q_lens), heads * group, d), generator=g).half().to(DEV)
    got = cr.kv_attention(cache, q, table, lens, q_start=_starts(q_lens) if q_each else None, max_q=n,
                          max_kv=max(kv_lens), out=torch.full_like(q, float("nan")))
    some = torch.tensor([0, heads // 2 + 1, heads - 1])
    rows = (some[:, None] * group + torch.arange(group)).flatten()
    part = cr.KVCache(*(t[:, some].contiguous() for t in (cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale)))
    assert got.isfinite().all()
    _check_attention(part, q[:, rows], table, q_lens, kv_lens, True, got[:, rows])


@pytest.mark.parametrize("rows", [1, 40, 140])
@pytest.mark.parametrize("bits", [4, 8])
def test_attention_value_rows_of_all_sizes(rows, bits):
    """Values of zero under the largest weight, and values whose scales span fp32."""
    _say("value sizes", rows, bits)
    m, d = 400, 64
    g = _gen(rows, bits)
    k, v = _values(g, (m, 1, d), BF16), _values(g, (m, 1, d), BF16)
    table = torch.arange(25, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([m], dtype=torch.int32, device=DEV)
    q = torch.randn((rows, 1, d), generator=g).bfloat16().to(DEV)
    slots = torch.arange(m, device=DEV)
    for change in ("sink", "first tiles zero", "all zero", "tiny", "large", "rising"):
        kk, vv = k.clone(), v.clone()
        if change == "sink":                            # its score is far above the others, its value is zero
            kk[0] = q[0, 0].cpu() * 30
            vv[0] = 0
        elif change == "first tiles zero":
            vv[:200] = 0
        elif change == "all zero":
            vv[:] = 0
        elif change == "tiny":
            vv *= 2.0 ** -60
        elif change == "large":
            vv *= 2.0 ** 60
        else:
            vv *= torch.exp2(torch.linspace(-70, 60, m))[:, None, None].bfloat16()
        cache = cr.KVCache.empty(25, 16, 1, d, bits, DEV)
        cr.kv_append(cache, kk.to(DEV), vv.to(DEV), slots)
        got = cr.kv_attention(cache, q, table, lens)
        _check_attention(cache, q, table, [rows], [m], True, got, tell=change)
        if change == "all zero":
            assert not got.any()


@pytest.mark.parametrize("n,m", [(1, 5000), (20, 700), (150, 700)])
def test_attention_is_repeatable_on_streams_and_buffers(n, m):
    _say("streams", n, m)
    g = _gen(n, m)
    cache = _random_cache(g, 2 * (-(-m // 16)), 16, 2, 128, 4)
    table, lens = _sequences(g, cache, [m, m - 3])
    base = torch.randn((2 * n, 24, 128), generator=g).half().to(DEV)
    q = base[:, 8:16]                                     # a slice of a fused projection, read in place
    want = cr.kv_attention(cache, q.contiguous(), table, lens)
    _check_attention(cache, q, table, [n, n], [m, m - 3], True, want)
    out = torch.full((2 * n, 8, 128), float("nan"), dtype=F16, device=DEV)
    need = cr.kv_workspace_bytes(cache, 2 * n, 8, 2, n, table.shape[1] * 16)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert cr.kv_attention(cache, q, table, lens, out=out, workspace=ws) is out
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    assert (ws[need:] == 0xFF).all()
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)   # heads outermost
    assert torch.equal(cr.kv_attention(cache, turned, table, lens), want)
    odd = torch.empty((2 * n, 8, 129), dtype=F16, device=DEV)[..., 1:].copy_(q)
    assert torch.equal(cr.kv_attention(cache, odd, table, lens), want)


@pytest.mark.parametrize("n,m", [(1, 3000), (17, 300), (70, 300), (30, 300)])
def test_attention_absent_pages_and_extreme_scores(n, m):
    _say("absent pages", n, m)
    g = _gen(n, m, 1)
    cache = _random_cache(g, 2 * (-(-m // 32)), 32, 1, 64, 4)
    table, lens = _sequences(g, cache, [m, m])
    table[0, 1], table[0, 3], table[1, 0] = -1, cache.pages, -(1 << 31)
    table[1, 2:] = (1 << 31) - 1                          # only its second page is there
    q = torch.randn((2 * n, 4, 64), generator=g).half().to(DEV)
    for causal in (True, False):
        got = cr.kv_attention(cache, q, table, lens, causal=causal)
        _check_attention(cache, q, table, [n, n], [m, m], causal, got)
    table.fill_(-1)
    assert not cr.kv_attention(cache, q, table, lens).any()
    # lengths out of range are clamped; scores far from zero
    table, _ = _sequences(g, cache, [m, m])
    wild = torch.tensor([1 << 30, -5], dtype=torch.int32, device=DEV)
    got = cr.kv_attention(cache, q, table, wild, causal=False)
    full = table.shape[1] * 32
    _check_attention(cache, q, table, [n, n], [full, 0], False, got)
    for scale in (0.0, 40.0, -40.0):
        got = cr.kv_attention(cache, q, table, lens, scale=scale, causal=False)
        assert got.isfinite().all()
        if scale == 0.0:
            _check_attention(cache, q, table, [n, n], [m, m], False, got, scale=0.0)
    # one sharp weight among many
    got = cr.kv_attention(cache, q, table, lens, scale=1.0, causal=False)
    _check_attention(cache, q, table, [n, n], [m, m], False, got, scale=1.0)


def test_attention_sums_a_long_even_tail():
    """One loud token and 60000 even ones far below it that weigh as much together."""
    _say("long even tail")
    m, d = 60001, 64
    pages = -(-m // 64)
    cache = cr.KVCache.empty(pages, 64, 1, d, 4, DEV)
    k = torch.zeros((m, 1, d))
    k[0, 0, 0] = 1.0
    v = torch.full((m, 1, d), 1.0)
    v[0] = -1.0
    slots = torch.arange(m, device=DEV)
    cr.kv_append(cache, k.half().to(DEV), v.half().to(DEV), slots)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([m], dtype=torch.int32, device=DEV)
    q = torch.zeros((1, 1, d), dtype=F16)
    q[..., 0] = 1.0
    for rows in (1, 40, 140):
        x = q.expand(rows, 1, d).contiguous().to(DEV)
        got = cr.kv_attention(cache, x, table, lens, scale=float(np.log(60000.0)), causal=False)
        _check_attention(cache, x, table, [rows], [m], False, got, scale=float(np.log(60000.0)))


@pytest.mark.parametrize("rows", [1, 20, 40, 150])
@pytest.mark.parametrize("step", [8, 16, 32, 64, 128])
def test_attention_scores_that_keep_rising(rows, step):
    """Every `step` tokens the scores rise, so that the running maximum does too."""
    _say("rising scores", rows, step)
    m, d = 777, 128
    g = _gen(step)
    k = torch.zeros((m, 1, d))
    k[:, 0, 0] = (torch.arange(m) // step).float()
    cache = cr.KVCache.empty(-(-m // 16), 16, 1, d, 4, DEV)
    cr.kv_append(cache, k.half().to(DEV), _values(g, (m, 1, d), F16).to(DEV), torch.arange(m, device=DEV))
    table = torch.arange(cache.pages, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([m], dtype=torch.int32, device=DEV)
    q = torch.zeros((rows, 1, d), dtype=F16)
    q[..., 0] = torch.linspace(0.01, 1.0, rows)[:, None]
    for scale in (0.3, 3.0, 8.0):
        got = cr.kv_attention(cache, q.to(DEV), table, lens, scale=scale)
        _check_attention(cache, q, table, [rows], [m], True, got, scale=scale)


def test_attention_shows_a_nan_that_is_seen_only():
    _say("NaN rows")
    g = _gen(8)
    for n, m in ((1, 700), (50, 100), (80, 100)):
        cache = _random_cache(g, -(-m // 16), 16, 2, 128, 4)
        table, lens = _sequences(g, cache, [m])
        q = torch.randn((n, 4, 128), generator=g).half().to(DEV)
        page = int(table[0, (m - 1) // 16])
        cache.v_scale[page, 1, (m - 1) % 16] = float("nan")   # the last token, seen by the last query alone
        got = cr.kv_attention(cache, q, table, lens)
        assert got[-1, 2:].isnan().all() and got[-1, :2].isfinite().all()
        assert n == 1 or got[:-1].isfinite().all()


@pytest.mark.parametrize("n", [1, 64, 20])
def test_graph_replays_write_and_attend(n):
    """Write, attend and read inside one graph, replayed with new inputs and
    eager work between the replays; each replay equals the eager calls."""
    _say("graph", n)
    g = _gen(n, 5)
    m = 2000
    caches = [_random_cache(_gen(1), 2 * (m // 16), 16, 2, 128, 4) for _ in range(2)]
    table, lens = _sequences(g, caches[0], [m, m - 70])
    at = lens.long()[:, None] - n + torch.arange(n, device=DEV)
    slots = (torch.gather(table.long(), 1, at // 16) * 16 + at % 16).reshape(-1)
    q = torch.empty((2 * n, 8, 128), dtype=F16, device=DEV)
    k, v = (torch.empty((2 * n, 2, 128), dtype=F16, device=DEV) for _ in range(2))

    def step(cache):
        cr.kv_append(cache, k, v, slots)
        return (cr.kv_attention(cache, q, table, lens), *cr.kv_read(cache, slots))

    for x in (q, k, v):
        x.copy_(torch.randn(x.shape, generator=g))
    step(caches[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(caches[0])
    for _ in range(4):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g))
        graph.replay()
        want = step(caches[1])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        (torch.ones(1 << 20, device=DEV) * 2).sum().item()


def test_offsets_past_32_bits():
    """A cache whose codes pass 4 GiB, its last pages in use."""
    _say("large cache")
    free, _ = torch.cuda.mem_get_info()
    if free < 30 << 30:
        pytest.skip("needs 30 GiB of free GPU memory")
    heads, page, d = 8, 256, 256
    pages = (5 << 30) // (heads * page * d)                # 5 GiB of 8-bit codes for the keys, as much for the values
    shape = (pages, heads, page)
    cache = cr.KVCache(torch.empty((*shape, d), dtype=torch.int8, device=DEV),
                       torch.empty(shape, dtype=torch.float32, device=DEV),
                       torch.empty((*shape, d), dtype=torch.int8, device=DEV),
                       torch.empty(shape, dtype=torch.float32, device=DEV))
    g = _gen(6)
    n = 600
    k, v = _values(g, (n, heads, d), F16), _values(g, (n, heads, d), F16)
    first = (pages - 3) * page
    slots = torch.arange(first, first + n, device=DEV)
    cr.kv_append(cache, k.to(DEV), v.to(DEV), slots)
    for got, x in zip(cr.kv_read(cache, slots), (k, v)):
        c, s = O.quantize(_np(x), 8)
        assert torch.equal(got.cpu(), torch.from_numpy(O.read_f32(c, s)).half())
    table = torch.arange(pages - 3, pages, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    for rows in (1, 40, 140):
        q = torch.randn((rows, heads, d), generator=g).half().to(DEV)
        got = cr.kv_attention(cache, q, table, lens)
        _check_attention(cache, q, table, [rows], [n], True, got)


def test_binding_refusals():
    cache = cr.KVCache.empty(4, 16, 2, 64, 4, DEV)
    x = torch.zeros((3, 2, 64), dtype=F16, device=DEV)
    slots = torch.arange(3, device=DEV)
    for bad in (x.float(), x[:, :1], x[..., :32], x[:2], x.cpu()):
        with pytest.raises((TypeError, ValueError)):
            cr.kv_append(cache, x, bad, slots)
    with pytest.raises(ValueError):
        cr.kv_append(cache, x, x.bfloat16(), slots)
    for bad in (slots.int(), slots[:2], slots.cpu()):
        with pytest.raises((TypeError, ValueError)):
            cr.kv_append(cache, x, x, bad)
    with pytest.raises(TypeError):
        cr.kv_read(cache, slots, dtype=torch.float32)
    with pytest.raises(ValueError):
        cr.kv_read(cache, slots, out=(x, x[:2]))
    q = torch.zeros((2, 4, 64), dtype=F16, device=DEV)
    table, lens = torch.zeros((2, 2), dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    for over in (dict(q=q[:, :3]), dict(table=table.long()), dict(kv_lens=lens[:1]), dict(q_start=lens),
                 dict(max_kv=33), dict(max_kv=-1), dict(q=q[:1]), dict(q=q.float()), dict(out=q.bfloat16()),
                 dict(workspace=q)):
        with pytest.raises((TypeError, ValueError, cr.ConvRotError)):
            cr.kv_attention(**{**dict(cache=cache, q=q, table=table, kv_lens=lens), **over})
