"""The rotated, quantised key/value cache: what its operators are measured on.

A row x of head_dim values (one token, one head) is kept as u = x W with W the
+-1 Sylvester-Hadamard matrix of that size, s = max|u| / qmax, and
c = round_half_even(u / s) in [-qmax, qmax]; qmax is 7 (4 bits, two codes a
byte, the even element in the low half, two's complement) or 127 (8 bits).
The stored scale is s / sqrt(head_dim), so that c * scale is the row in the
orthonormal basis H = W / sqrt(head_dim), and the row itself is (c * scale) H.

Layout: codes [pages, heads, page, head_dim * bits / 8], scales fp32
[pages, heads, page]; a slot is page_index * page + offset.

Three operators:
  write      quantise new keys and values into their slots (with the read-back
             of these slots, since what is held in 4 or 8 bits is compared as
             the values it stands for)
  read       the rows of given slots as 16-bit tensors
  attention  softmax(q k^T / sqrt(head_dim)) v over the cached rows of each
             sequence through its table of pages: single tokens, prompts
             (causal, aligned at the end), and states of another length (not
             causal).  A query that sees no key gives zeros.
"""
import math
import random

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one generated token for each of four sequences: latency
        dict(name="write step", op="write", tokens=4, heads=8, head_dim=128, bits=4, dtype="fp16", page=16),
        # the prompt size of the linear sweep (1024 rows, 2048 columns = 16 heads of 128)
        dict(name="write prompt", op="write", tokens=1024, heads=16, head_dim=128, bits=4, dtype="bf16", page=64),
        # a packed batch of prompts, kept in 8 bits
        dict(name="write packed prompts", op="write", tokens=16384, heads=8, head_dim=128, bits=8, dtype="fp16",
             page=256),
        # a short shared prefix handed to a dense consumer, odd length, small heads
        dict(name="read prefix", op="read", tokens=4099, heads=4, head_dim=64, bits=4, dtype="bf16", page=32),
        # a long context read back whole
        dict(name="read context", op="read", tokens=65536, heads=8, head_dim=128, bits=4, dtype="fp16", page=128),
        # one token against a short context, a key head for each query head: latency
        dict(name="decode one", op="attention", batch=1, q_len=1, kv_len=1000, ragged=False, heads=16, group=1,
             head_dim=128, bits=4, dtype="fp16", page=16, causal=True),
        # a serving batch at mixed positions, grouped heads; one slot of the batch is idle (length 0)
        dict(name="decode batch", op="attention", batch=32, q_len=1, kv_len=8192, ragged=True, heads=8, group=4,
             head_dim=128, bits=4, dtype="bf16", page=64, causal=True),
        # two very long contexts: the split over the sequence
        dict(name="decode long", op="attention", batch=2, q_len=1, kv_len=131072, ragged=False, heads=4, group=8,
             head_dim=128, bits=4, dtype="bf16", page=256, causal=True),
        # wide heads in 8 bits, an odd group, odd lengths
        dict(name="decode wide int8", op="attention", batch=48, q_len=1, kv_len=2501, ragged=True, heads=4, group=5,
             head_dim=256, bits=8, dtype="fp16", page=32, causal=True),
        # a whole prompt
        dict(name="prompt", op="attention", batch=1, q_len=4096, kv_len=4096, ragged=False, heads=8, group=4,
             head_dim=128, bits=4, dtype="bf16", page=64, causal=True),
        # the next chunks of three prompts behind what is cached already, odd lengths, small heads in 8 bits
        dict(name="prompt chunks", op="attention", batch=3, q_len=701, kv_len=6007, ragged=True, heads=8, group=3,
             head_dim=64, bits=8, dtype="fp16", page=16, causal=True),
        # image latents against a text encoder's states, written once and read at every step
        dict(name="cross", op="attention", batch=2, q_len=1024, kv_len=512, ragged=False, heads=16, group=1,
             head_dim=128, bits=4, dtype="fp16", page=64, causal=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = [work(c) for c in listed()]
    most_bytes, most_flops = max(w["bytes"] for w in top), max(w["flops"] for w in top)
    while True:
        op = rng.choice(["write", "read", "attention", "attention", "attention"])
        c = dict(op=op, heads=rng.choice([1, 2, 3, 4, 6, 8, 12, 16]), head_dim=rng.choice([64, 128, 128, 256]),
                 bits=rng.choice([4, 4, 8]), dtype=rng.choice(["fp16", "bf16"]), page=rng.choice([16, 32, 64, 128, 256]))
        if op != "attention":
            c["tokens"] = _log_int(rng, 1, 65536)
        else:
            c["batch"] = _log_int(rng, 1, 64)
            c["group"] = rng.randint(1, 8)
            c["kv_len"] = _log_int(rng, 1, 131072)
            c["causal"] = rng.random() < 0.75
            c["q_len"] = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4096)
            if c["causal"]:
                c["q_len"] = min(c["q_len"], c["kv_len"] + 3)  # a few queries may see no key
            c["ragged"] = rng.random() < 0.6
            # the plain form holds every score of the padded batch in 32 bits, and every padded row
            if c["batch"] * c["heads"] * c["group"] * c["q_len"] * c["kv_len"] > 32 * 4096 * 4096:
                continue
            if c["batch"] * c["kv_len"] * c["heads"] * c["head_dim"] > 32 * 8192 * 8 * 128:
                continue
        w = work(c)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            return c


def _lengths(case):
    """Queries and cached keys of each sequence: whole lengths, or ragged ones (an idle slot among eight or more)."""
    n, q, kv = case["batch"], case["q_len"], case["kv_len"]
    if not case["ragged"]:
        return [q] * n, [kv] * n
    r = random.Random(n * 1000003 + q * 10007 + kv)
    qs = [q] + [r.randint((q + 1) // 2, q) for _ in range(n - 1)]
    kvs = [kv] + [max(r.randint((kv + 3) // 4, kv), min(qs[i + 1], kv) if case["causal"] else 0) for i in range(n - 1)]
    if n >= 8:
        kvs[n // 2] = 0
    return qs, kvs


def _row_bytes(case):
    return case["head_dim"] * case["bits"] // 8 + 4


def work(case):
    d, h = case["head_dim"], case["heads"]
    if case["op"] == "write":  # K and V in, codes and scales written, the values they stand for out
        rows = 2 * case["tokens"] * h
        return {"bytes": rows * (2 * d + _row_bytes(case) + 2 * d) + 8 * case["tokens"],
                "flops": rows * 2 * d * int(math.log2(d))}
    if case["op"] == "read":
        rows = 2 * case["tokens"] * h
        return {"bytes": rows * (_row_bytes(case) + 2 * d) + 8 * case["tokens"], "flops": rows * d * int(math.log2(d))}
    qs, kvs = _lengths(case)
    pairs = 0
    for q, kv in zip(qs, kvs):
        if case["causal"]:  # query i of q sees the first kv - q + i + 1 keys
            seen = min(q, kv)
            pairs += seen * kv - seen * (seen - 1) // 2
        else:
            pairs += q * kv
    hq = h * case["group"]
    return {"bytes": sum(kvs) * h * 2 * _row_bytes(case) + sum(qs) * hq * d * 4, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ the inputs

def _signs(d, device):
    w = torch.ones((1, 1), dtype=torch.float64, device=device)
    while w.shape[0] < d:
        w = torch.cat([torch.cat([w, w], 1), torch.cat([w, -w], 1)], 0)
    return w


def _rows(gen, n, heads, d, device):
    """Keys or values as a model makes them: a few channels of each head stand out."""
    x = torch.randn((n, heads, d), generator=gen, device=device)
    loud = torch.rand((heads, d), generator=gen, device=device) < 0.02
    return x * torch.where(loud, 8.0, 1.0)


def _filled(gen, pages, case, device):
    """Codes and scales of a cache whose every slot holds a quantised row."""
    h, d, p = case["heads"], case["head_dim"], case["page"]
    top = 7.0 if case["bits"] == 4 else 127.0
    shape = (pages, h, p, d * case["bits"] // 8)
    codes = torch.empty(shape, dtype=torch.uint8 if case["bits"] == 4 else torch.int8, device=device)
    scale = torch.empty((pages, h, p), dtype=torch.float32, device=device)
    w = _signs(d, device).float()
    step = max(1, (1 << 25) // (h * p * d))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        u = (_rows(gen, n * p, h, d, device) @ w).view(n, p, h, d).permute(0, 2, 1, 3)
        s = u.abs().amax(-1) / top
        c = torch.round(u / s[..., None]).clamp(-top, top).to(torch.int8)
        if case["bits"] == 4:
            c = ((c[..., 0::2] & 15) | (c[..., 1::2] << 4)).view(torch.uint8)
        codes[a:a + n] = c
        scale[a:a + n] = s / math.sqrt(d)
    return codes, scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 17)
    h, d, p = case["heads"], case["head_dim"], case["page"]
    st = {"case": case, "signs": _signs(d, dev)}
    st["signs32"] = st["signs"].float()
    if case["op"] == "attention":
        qs, kvs = _lengths(case)
        per = [-(-n // p) for n in kvs]
        width = max(per + [1])
        pages = sum(per) + 1
        st["k"], st["ks"] = _filled(gen, pages, case, dev)
        st["v"], st["vs"] = _filled(gen, pages, case, dev)
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        table = torch.zeros((len(kvs), width), dtype=torch.int32, device=dev)
        at = 0
        for i, n in enumerate(per):
            table[i, :n] = order[at:at + n]
            if kvs[i] % p:  # what lies past the end of a sequence's last page was never written
                st["ks"][order[at + n - 1].item(), :, kvs[i] % p:] = float("nan")
                st["vs"][order[at + n - 1].item(), :, kvs[i] % p:] = float("nan")
            at += n
        st["table"] = table
        st["kv_lens"] = torch.tensor(kvs, dtype=torch.int32, device=dev)
        start = [0]
        for n in qs:
            start.append(start[-1] + n)
        st["q_start"] = torch.tensor(start, dtype=torch.int32, device=dev)
        st["max_q"], st["max_kv"] = max(qs), max(kvs)
        st["q"] = torch.randn((start[-1], h * case["group"], d), generator=gen, device=dev).to(_DT[case["dtype"]])
        return st
    n = case["tokens"]
    pages = -(-n // p) + 2
    slots = torch.randperm(pages, generator=gen, device=dev)[:-(-n // p)]
    st["slots"] = (slots[:, None] * p + torch.arange(p, device=dev)).reshape(-1)[:n].contiguous()
    if case["op"] == "read":
        st["k"], st["ks"] = _filled(gen, pages, case, dev)
        st["v"], st["vs"] = _filled(gen, pages, case, dev)
        return st
    kind = torch.uint8 if case["bits"] == 4 else torch.int8
    for c, s in (("k", "ks"), ("v", "vs")):
        st[c] = torch.zeros((pages, h, p, d * case["bits"] // 8), dtype=kind, device=dev)
        st[s] = torch.zeros((pages, h, p), dtype=torch.float32, device=dev)
    # keys and values as a fused projection leaves them: side by side in one row of each token
    kv = torch.cat([_rows(gen, n, h, d, dev), _rows(gen, n, h, d, dev)], 1).to(_DT[case["dtype"]])
    st["new_k"], st["new_v"] = kv[:, :h], kv[:, h:]
    return st


# -------------------------------------------------------------- the plain form

def _write(codes, scale, x, slots, signs):
    """x [n, heads, d] into its slots; sums in 64 bits, since a code may lie next to a border."""
    d, p, packed = x.shape[-1], codes.shape[2], codes.dtype == torch.uint8
    top = 7.0 if packed else 127.0
    u = (x.double() @ signs).float()
    s = u.abs().amax(-1) / top
    c = torch.where(s[..., None] > 0, torch.round(u / s[..., None]), torch.zeros_like(u)).clamp(-top, top)
    c = c.to(torch.int8)
    if packed:
        c = ((c[..., 0::2] & 15) | (c[..., 1::2] << 4)).view(torch.uint8)
    page, off = slots // p, slots % p
    codes[page, :, off] = c
    scale[page, :, off] = s * float(torch.tensor(d, dtype=torch.float64).rsqrt().float())


def _values(codes, scale):
    """Codes and their scales as the rows in the rotated basis, 32 bits."""
    if codes.dtype == torch.uint8:
        b = codes.int()
        c = torch.stack([((b & 15) ^ 8) - 8, ((b >> 4) ^ 8) - 8], -1).flatten(-2)
    else:
        c = codes
    return c.float() * scale[..., None]


def _read(codes, scale, slots, signs32, dtype):
    p = codes.shape[2]
    page, off = slots // p, slots % p
    x = _values(codes[page, :, off], scale[page, :, off])
    return (x @ signs32 * x.shape[-1] ** -0.5).to(dtype)


def _attend(st):
    case, q = st["case"], st["q"]
    h, g, d = case["heads"], case["group"], case["head_dim"]
    n, t, width = case["batch"], q.shape[0], st["table"].shape[1] * case["page"]
    table, lens, start = st["table"].long(), st["kv_lens"].long(), st["q_start"].long()
    pos = torch.arange(width, device=q.device)
    alive = pos < lens[:, None]                                               # [n, width]

    def rows(codes, scale):
        c = codes[table].transpose(1, 2).flatten(2, 3)                       # [n, h, width, bytes]
        s = scale[table].transpose(1, 2).flatten(2, 3)
        return _values(c, torch.where(alive[:, None], s, torch.zeros_like(s)))

    rot = st["signs32"] * d ** -0.5
    i = torch.arange(st["max_q"], device=q.device)
    count = start[1:] - start[:-1]
    take = torch.where(i < count[:, None], start[:-1, None] + i, t)          # [n, max_q], t: no such query
    padded = torch.cat([q.float() @ rot, torch.zeros((1, h * g, d), device=q.device)])[take]
    padded = padded.view(n, -1, h, g, d).permute(0, 2, 3, 1, 4).reshape(n, h, -1, d)
    s = padded @ rows(st["k"], st["ks"]).transpose(2, 3).contiguous() * d ** -0.5
    seen = alive[:, None, :].expand(n, st["max_q"], width)
    if case["causal"]:
        seen = seen & (pos <= (lens - count)[:, None, None] + i[:, None])
    s = s.view(n, h, g, -1, width).masked_fill_(~seen[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m.isinf(), torch.zeros_like(m), m))
    total = e.sum(-1, keepdim=True)
    o = (e.view(n, h, -1, width) @ rows(st["v"], st["vs"])).view(n, h, g, -1, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)) @ rot
    which = torch.searchsorted(start[1:].contiguous(), torch.arange(t, device=q.device), right=True)
    return o.permute(0, 3, 1, 2, 4)[which, torch.arange(t, device=q.device) - start[which]].reshape(t, h * g, d).to(q.dtype)


def run(state):
    case = state["case"]
    if own:
        import rotation_quantized_int8_amd as cr

        cache = cr.KVCache(state["k"], state["ks"], state["v"], state["vs"])
        if case["op"] == "attention":
            return cr.kv_attention(cache, state["q"], state["table"], state["kv_lens"], q_start=state["q_start"],
                                   max_q=state["max_q"], max_kv=state["max_kv"], causal=case["causal"])
        if case["op"] == "write":
            cr.kv_append(cache, state["new_k"], state["new_v"], state["slots"])
        return cr.kv_read(cache, state["slots"], dtype=_DT[case["dtype"]])
    if case["op"] == "attention":
        return _attend(state)
    if case["op"] == "write":
        _write(state["k"], state["ks"], state["new_k"], state["slots"], state["signs"])
        _write(state["v"], state["vs"], state["new_v"], state["slots"], state["signs"])
    return (_read(state["k"], state["ks"], state["slots"], state["signs32"], _DT[case["dtype"]]),
            _read(state["v"], state["vs"], state["slots"], state["signs32"], _DT[case["dtype"]]))


# ------------------------------------------------------------------ in 64 bits

def _turn(x):
    """x W by butterflies over the last axis."""
    d, lead = x.shape[-1], x.shape[:-1]
    k = 1
    while k < d:
        y = x.reshape(*lead, d // (2 * k), 2, k)
        x = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(*lead, d)
        k *= 2
    return x


def _stored(codes, scale, page, off):
    """The rows that slots (page, off) stand for, in the basis of the inputs."""
    c, s = codes[page, :, off], scale[page, :, off].double()
    if c.dtype == torch.uint8:
        low, high = (c.to(torch.int8) << 4) >> 4, c.view(torch.int8) >> 4
        c = torch.cat([low[..., None], high[..., None]], -1).flatten(-2)
    return _turn(c.double() * s[..., None]) / math.sqrt(_width(c))


def _width(c):
    return c.shape[-1]


def exact(case, seed):
    st = prepare(case, seed)
    p, d = case["page"], case["head_dim"]
    if case["op"] == "read":
        page, off = st["slots"] // p, st["slots"] % p
        return _stored(st["k"], st["ks"], page, off), _stored(st["v"], st["vs"], page, off)
    if case["op"] == "write":
        top, out = (7.0 if case["bits"] == 4 else 127.0), []
        for x in (st["new_k"], st["new_v"]):
            u = _turn(x.double())
            s = u.abs().amax(-1, keepdim=True) / top
            c = torch.where(s > 0, u / s, torch.zeros_like(u)).round()
            out.append(_turn(c * s) / d)
        return tuple(out)
    g, qs, kvs = case["group"], *_lengths(case)
    out, at = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device), 0
    for b, (n, m) in enumerate(zip(qs, kvs)):
        key = torch.arange(m, device=out.device)
        page, off = st["table"][b].long()[key // p], key % p
        k, v = _stored(st["k"], st["ks"], page, off), _stored(st["v"], st["vs"], page, off)
        for h in range(case["heads"] * g if m else 0):
            kh, vh = k[:, h // g], v[:, h // g]
            for a in range(0, n, 1024):
                z = min(n, a + 1024)
                s = st["q"][at + a:at + z, h].double() @ kh.T.contiguous() / math.sqrt(d)
                if case["causal"]:
                    hidden = key[None] > (m - n + torch.arange(a, z, device=out.device))[:, None]
                    s = s.masked_fill(hidden, float("-inf"))
                w = torch.softmax(s, -1).nan_to_num(0.0)  # a query that sees no key
                out[at + a:at + z, h] = w @ vh
        at += n
    return out
