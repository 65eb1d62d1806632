"""The attention block example: quantised projections around the quantised cache."""
import importlib.util
import os

import pytest
import torch

import rotation_quantized_int8_amd as cr
from test_kv_gpu import _check_attention

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
_spec = importlib.util.spec_from_file_location("attention_block", _PATH)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)

SIZES = [dict(width=512, heads=8, kv_heads=2, context=256, lengths=(37, 90), steps=5, page_size=16, bits=4,
              context_tokens=19),
         dict(width=1024, heads=8, kv_heads=8, context=512, lengths=(130, 1, 64), steps=40, page_size=32, bits=8,
              context_tokens=77)]


def _bytes(cache):
    return [t.clone() for t in (cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale)]


@pytest.mark.parametrize("sizes", SIZES)
def test_steps_in_a_graph_equal_eager_steps(sizes):
    one, two = example.main(**sizes, graphed=True), example.main(**sizes, graphed=False)
    assert one["last"].isfinite().all()
    assert torch.equal(one["first"], two["first"]) and torch.equal(one["last"], two["last"])
    for a, b in zip(one["caches"], two["caches"]):
        for x, y in zip(_bytes(a), _bytes(b)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("sizes", SIZES)
def test_prompt(sizes):
    """The prompt's attention against 64 bits; written in two chunks it fills the cache with the same bytes."""
    r = example.main(**sizes, graphed=False)
    block, cross, prompt, table, page = r["block"], r["cross"], r["prompt"], r["table"], sizes["page_size"]
    lengths = list(sizes["lengths"])
    sequence = torch.cat([torch.full((n,), b) for b, n in enumerate(lengths)]).cuda()
    position = torch.cat([torch.arange(n) for n in lengths]).cuda()
    slots = example.slots_of(table, page, sequence, position)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    start = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    cache = block.cache(r["caches"][0].pages, page, sizes["bits"])
    q = block.queries(cache, prompt, slots)
    o = cr.kv_attention(cache, q, table, lens, q_start=start)
    _check_attention(cache, q, table, lengths, lengths, True, o)
    y = cr.linear_w8a8_ex(o.view(len(prompt), -1), *block.out, residual=prompt)
    qc = cross.queries(r["caches"][1], y, None)
    oc = cr.kv_attention(r["caches"][1], qc, r["context_table"], r["context_lens"], q_start=start, causal=False)
    _check_attention(r["caches"][1], qc, r["context_table"], lengths, [sizes["context_tokens"]] * len(lengths), False, oc)
    assert torch.equal(cr.linear_w8a8_ex(oc.view(len(prompt), -1), *cross.out, residual=y), r["first"])
    parts = block.cache(cache.pages, page, sizes["bits"])
    cut = len(prompt) // 3
    for rows in (slice(cut, None), slice(0, cut)):
        block.queries(parts, prompt[rows], slots[rows])
    for x, z in zip(_bytes(cache), _bytes(parts)):
        assert torch.equal(x, z)
