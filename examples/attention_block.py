"""An attention block on the quantised path end to end: W8A8 projections
(rotated int8 weights) around attention over a rotated, quantised key/value
cache.

    x -> layer norm -> q, k, v (one W8A8 linear) -> kv_append -> kv_attention
      -> W8A8 out projection + residual -> y

Two sequences share one paged cache.  Their prompts of different lengths run
as one call; then tokens are fed one at a time, each step (projections, cache
write, attention, and the counting of the positions) one replay of a HIP
graph; a second cache holds states of another length (a text encoder's), which
the last step attends to without a causal mask.

    python examples/attention_block.py        # on an MI355X
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import rotation_quantized_int8_amd as cr  # noqa: E402


class AttentionBlock:
    """Weights of one block: `heads` query heads in groups over `kv_heads`."""

    def __init__(self, width: int, heads: int, kv_heads: int, context: int = 0, seed: int = 0, device="cuda"):
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, width // heads
        gen = torch.Generator().manual_seed(seed)

        def weights(n, k):
            return cr.quantize_weights((torch.randn((n, k), generator=gen) * k ** -0.5).to(device))

        kv = 2 * kv_heads * self.head_dim
        self.qkv = weights(width + kv, width) if not context else None
        self.q = weights(width, width) if context else None       # cross attention: the keys and values come
        self.kv = weights(kv, context) if context else None       # from states of width `context`
        self.out = weights(width, width)

    def cache(self, pages: int, page_size: int, bits: int, device="cuda") -> cr.KVCache:
        return cr.KVCache.empty(pages, page_size, self.kv_heads, self.head_dim, bits, device)

    def write_context(self, cache, states, slots) -> None:
        """Cross attention: the states' keys and values, once."""
        kv = cr.linear_w8a8(states, *self.kv).view(len(states), 2, self.kv_heads, self.head_dim)
        cr.kv_append(cache, kv[:, 0], kv[:, 1], slots)

    def queries(self, cache, x, slots):
        """The rows' queries; their keys and values go into `slots` of the cache."""
        h = torch.nn.functional.layer_norm(x, x.shape[-1:])
        if self.q is not None:
            return cr.linear_w8a8(h, *self.q).view(len(x), self.heads, self.head_dim)
        y = cr.linear_w8a8(h, *self.qkv).view(len(x), self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = y.split([self.heads, self.kv_heads, self.kv_heads], 1)   # read in place, no copies
        cr.kv_append(cache, k, v, slots)
        return q

    def __call__(self, cache, x, slots, table, kv_lens, **bounds):
        """x fp16 [tokens, width] -> [tokens, width]; bounds: q_start, max_q, max_kv, causal of kv_attention."""
        o = cr.kv_attention(cache, self.queries(cache, x, slots), table, kv_lens, **bounds)
        return cr.linear_w8a8_ex(o.view(len(x), -1), *self.out, residual=x)


def slots_of(table, page_size, sequence, position):
    """Slots of tokens (sequence, position), on the device."""
    page = table[sequence, torch.div(position, page_size, rounding_mode="floor")].long()
    return page * page_size + position % page_size


def generate(block, cross, caches, prompt, lengths, steps, table, context_table, context_lens, page_size,
             graphed=True):
    """The prompts (rows of both sequences, one after the other), then `steps`
    tokens of each, a step's output the next one's input (`graphed`: a step is
    one replay).  Returns the outputs of the prompt and of the last step."""
    device, batch = prompt.device, len(lengths)
    most = max(lengths) + steps
    lens = torch.tensor(lengths, dtype=torch.int32, device=device)
    start = torch.zeros(batch + 1, dtype=torch.int32, device=device)
    start[1:] = lens.cumsum(0)
    sequence = torch.cat([torch.full((n,), b) for b, n in enumerate(lengths)]).to(device)
    position = torch.cat([torch.arange(n) for n in lengths]).to(device)
    y = block(caches[0], prompt, slots_of(table, page_size, sequence, position), table, lens, q_start=start,
              max_q=max(lengths), max_kv=max(lengths))
    first = cross(caches[1], y, None, context_table, context_lens, q_start=start, max_q=max(lengths), causal=False)

    x = first[(start[1:] - 1).long()].clone()                     # each sequence's last row
    each = torch.arange(batch, device=device)

    def step():
        at = lens.clone()
        lens.add_(1)
        y = block(caches[0], x, slots_of(table, page_size, each, at.long()), table, lens, max_kv=most)
        x.copy_(cross(caches[1], y, None, context_table, context_lens, causal=False))

    if not graphed:
        for _ in range(steps):
            step()
        return first, x
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = lens.clone(), x.clone()
    with torch.cuda.stream(side):
        step()                                                    # warm up; its token is written again below
        lens.copy_(keep[0])
        x.copy_(keep[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps):
        graph.replay()
    return first, x


def main(width=2048, heads=16, kv_heads=4, context=1024, lengths=(700, 1024), steps=16, page_size=64, bits=4,
         context_tokens=77, graphed=True, device="cuda"):
    block = AttentionBlock(width, heads, kv_heads, seed=1, device=device)
    cross = AttentionBlock(width, heads, kv_heads, context=context, seed=2, device=device)
    gen = torch.Generator().manual_seed(3)
    batch, per = len(lengths), -(-(max(lengths) + steps) // page_size)
    table = torch.randperm(batch * per, generator=gen).to(torch.int32).view(batch, per).to(device)
    context_per = -(-context_tokens // page_size)
    context_table = torch.arange(batch * context_per, dtype=torch.int32, device=device).view(batch, context_per)
    context_lens = torch.full((batch,), context_tokens, dtype=torch.int32, device=device)
    caches = [block.cache(batch * per, page_size, bits, device),
              cross.cache(batch * context_per, page_size, 8, device)]

    states = torch.randn((batch * context_tokens, context), generator=gen).half().to(device)
    at = torch.arange(context_tokens, device=device).repeat(batch)
    sequence = torch.arange(batch, device=device).repeat_interleave(context_tokens)
    cross.write_context(caches[1], states, slots_of(context_table, page_size, sequence, at))

    prompt = torch.randn((sum(lengths), width), generator=gen).half().to(device)
    first, last = generate(block, cross, caches, prompt, list(lengths), steps, table, context_table, context_lens,
                           page_size, graphed)
    torch.cuda.synchronize()
    return dict(block=block, cross=cross, caches=caches, table=table, prompt=prompt, first=first, last=last,
                context_table=context_table, context_lens=context_lens)


if __name__ == "__main__":
    r = main()
    held = sum(t.numel() * t.element_size() for c in r["caches"] for t in (c.k_codes, c.k_scale, c.v_codes, c.v_scale))
    print(f"prompt outputs {list(r['first'].shape)}, last step {list(r['last'].shape)}, caches {held / 2 ** 20:.1f} MiB")
