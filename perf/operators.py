"""The 4-bit paged KV cache, as it is measured: writing new keys and values into it, reading rows back as
values, and attention over it.

A cache is six tensors.  Codes are uint8 [pages][heads][page][dim / 2], two's-complement nibbles, dimension
2j in the low and 2j + 1 in the high half of byte j; steps are fp32 [pages][heads][page]; the first position
of a sequence (BOS) is kept at 8 bits in int8 [pages][heads][dim], indexed by the sequence's first page.
Sequence b of a batch owns the rows starts[b] .. starts[b + 1] of the token tensors, at its last positions.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
Q4, Q3, Q8 = math.sqrt(7.0), 3.0, 127.0


def listed():
    write = {"op": "write", "page": 64, "dim": 128, "bits": 4, "out": "fp32"}
    read = {"op": "read", "page": 64, "dim": 128}
    attend = {"op": "attend", "page": 64, "dim": 128, "dtype": "bf16", "window": 0, "causal": True, "lse": False}
    return [
        # one decode step of one sequence: latency alone
        {**write, "name": "write_step", "batch": 1, "new": 1, "new_to": 1, "len": 78, "len_to": 78, "kv": 8, "dtype": "bf16"},
        # a decode step of a ragged batch, in the 3-bit form
        {**write, "name": "write_batch", "batch": 96, "new": 1, "new_to": 1, "len": 33, "len_to": 8000, "kv": 8, "dim": 64,
         "bits": 3, "dtype": "fp32"},
        # the prompts of a prefill, all heads with keys of their own (32 heads of 128)
        {**write, "name": "write_prompt", "batch": 3, "new": 1500, "new_to": 6000, "len": 1500, "len_to": 6000, "kv": 32,
         "dtype": "bf16"},
        # a short prefix out of small pages
        {**read, "name": "read_prefix", "batch": 1, "new": 333, "new_to": 333, "len": 333, "len_to": 333, "kv": 5, "page": 16,
         "out": "fp32"},
        # whole caches of a batch, for a dense pass over them
        {**read, "name": "read_batch", "batch": 24, "new": 900, "new_to": 8192, "len": 900, "len_to": 8192, "kv": 8,
         "out": "bf16"},
        # one token after a short prompt: latency alone
        {**attend, "name": "attend_step", "batch": 1, "new": 1, "new_to": 1, "len": 500, "len_to": 500, "heads": 32, "kv": 8},
        # a decode step of a full ragged batch, four query heads to a key head
        {**attend, "name": "attend_batch", "batch": 64, "new": 1, "new_to": 1, "len": 256, "len_to": 8192, "heads": 32, "kv": 8},
        # decode at the far end of long contexts
        {**attend, "name": "attend_long", "batch": 2, "new": 1, "new_to": 1, "len": 100001, "len_to": 131072, "heads": 64, "kv": 8},
        # a head of keys to each query head, in fp32, 32 heads of 128 over 4096 positions
        {**attend, "name": "attend_heads", "batch": 4, "new": 1, "new_to": 1, "len": 4096, "len_to": 4096, "heads": 32, "kv": 32,
         "dtype": "fp32", "lse": True},
        # a few draft tokens of each sequence, behind a sliding window, small pages and heads
        {**attend, "name": "attend_draft", "batch": 16, "new": 1, "new_to": 6, "len": 700, "len_to": 5000, "heads": 40, "kv": 8,
         "dim": 64, "page": 16, "window": 1024, "lse": True},
        # ragged prompts from their first token
        {**attend, "name": "attend_prompt", "batch": 3, "new": 700, "new_to": 4100, "len": 700, "len_to": 4100, "heads": 32,
         "kv": 8},
        # the next chunk of prompts that already have a long cache
        {**attend, "name": "attend_chunk", "batch": 2, "new": 512, "new_to": 1024, "len": 12000, "len_to": 16500, "heads": 32,
         "kv": 8, "dim": 64},
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        top[c["op"]] = max(top.get(c["op"], 0.0), w["bytes"] + w["flops"] / 200)
    while True:
        c = {"op": rng.choice(("write", "read", "attend", "attend", "attend")), "page": rng.choice((16, 32, 64, 128, 256)),
             "dim": rng.choice((64, 128, 128, 256)), "kv": rng.choice((1, 2, 3, 5, 8, 16, 32))}
        c["batch"] = _between(rng, 1, 96)
        c["len"] = _between(rng, 1, 12000)
        c["len_to"] = _between(rng, c["len"], 3 * c["len"])
        if c["op"] == "write":
            c |= {"bits": rng.choice((3, 4, 4)), "dtype": rng.choice(("bf16", "fp32")), "out": rng.choice(("bf16", "fp32"))}
        elif c["op"] == "read":
            c |= {"out": rng.choice(("bf16", "fp32"))}
        else:
            c |= {"heads": c["kv"] * rng.choice((1, 2, 3, 4, 5, 8)), "dtype": rng.choice(("bf16", "bf16", "fp32")),
                  "lse": rng.random() < 0.5, "causal": rng.random() < 0.9}
            c["window"] = _between(rng, 1, 4096) if c["causal"] and rng.random() < 0.3 else 0
        kind = rng.choice(("step", "few", "all", "chunk"))
        if kind == "step":
            c["new"] = c["new_to"] = 1
        elif kind == "few":
            c["new"], c["new_to"] = 1, rng.randint(2, 9)
        elif kind == "all":
            c["new"], c["new_to"] = c["len"], c["len_to"]
        else:
            c["new"] = _between(rng, 1, c["len"])
            c["new_to"] = min(c["len_to"], 2 * c["new"])
        w = work(c)
        rows, longest = c["batch"] * max(_new(c)), max(_lengths(c))
        padded = rows * longest * c.get("heads", 0)  # the plain form's scores
        dense = c["batch"] * longest * c["kv"] * c["dim"]  # its keys
        if w["bytes"] + w["flops"] / 200 <= top[c["op"]] and padded <= 1.6e9 and dense <= 5.4e8 and rows * c["kv"] * c["dim"] <= 2e8:
            return c


def _spread(lo, hi, count, turn):
    """`count` whole numbers over lo .. hi, ragged and the same for every seed; the first is hi."""
    return [hi - int((hi - lo + 0.999) * ((i * turn) % 1.0)) for i in range(count)]


def _lengths(c):
    return _spread(c["len"], c["len_to"], c["batch"], 0.6180339887)


def _new(c):
    if (c["new"], c["new_to"]) == (c["len"], c["len_to"]):
        return _lengths(c)
    return [min(n, m) for n, m in zip(_spread(c["new"], c["new_to"], c["batch"], 0.7548776662), _lengths(c))]


def _pairs(c):
    """Visible (query, key) pairs of one head, and the cached positions that some query of a sequence sees."""
    pairs = seen = 0
    for n, m in zip(_new(c), _lengths(c)):
        if not c["causal"]:
            pairs, seen = pairs + n * m, seen + m
            continue
        first, w = m - n, c["window"] or m  # queries stand at first .. m - 1 and see min(p + 1, w) keys
        full = max(0, min(n, m - max(w, first + 1) + 1)) if w < m else 0  # queries that see w keys
        part = n - full
        pairs += full * w + part * (first + 1) + part * (part - 1) // 2
        seen += min(m, n + w - 1)
    return pairs, seen


def work(c):
    rows, row = sum(_new(c)), c["kv"] * c["dim"]
    held = 2 * c["kv"] * (c["dim"] // 2 + 4)  # a position's keys and values in the cache
    wide = {"bf16": 2, "fp32": 4}
    if c["op"] == "write":  # into the cache, and back out of it
        return {"bytes": rows * (2 * row * (wide[c["dtype"]] + wide[c["out"]]) + 2 * held), "flops": 6.0 * rows * row}
    if c["op"] == "read":
        return {"bytes": rows * (held + 2 * row * wide[c["out"]]), "flops": 2.0 * rows * row}
    pairs, seen = _pairs(c)
    out = rows * c["heads"] * (2 * c["dim"] * wide[c["dtype"]] + (4 if c["lse"] else 0))
    return {"bytes": seen * held + out, "flops": 4.0 * pairs * c["heads"] * c["dim"]}


def _keys(shape, g, dtype):
    """Rows as post-RoPE keys are: heavy tails (Student-t with 3 degrees) and some channels that are larger than the others."""
    x = torch.empty(shape, device="cuda").normal_(generator=g)
    s = sum(torch.empty(shape[:-1] + (1,), device="cuda").normal_(generator=g).square() for _ in range(3))
    x *= (3.0 / s.clamp_min(0.05)).sqrt()
    x[..., :: 16] *= 3.0
    return x.to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    lens, new = _lengths(c), _new(c)
    page, kv, dim = c["page"], c["kv"], c["dim"]
    need = [-(-m // page) for m in lens]
    pages, width = sum(need) + 3, max(need)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.zeros(c["batch"] + 1, dtype=torch.int64)
    at[1:] = torch.cumsum(torch.tensor(need), 0)
    col = torch.arange(width, device="cuda")
    first, count = at[:-1].cuda()[:, None], torch.tensor(need, device="cuda")[:, None]
    table = torch.where(col < count, order[(first + col).clamp(max=pages - 1)], -1)
    starts = torch.zeros(c["batch"] + 1, dtype=torch.int32)
    starts[1:] = torch.cumsum(torch.tensor(new), 0)
    s = {"case": c, "rows": sum(new), "max_new": max(new), "longest": max(lens), "table": table.contiguous(),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "starts": starts.cuda()}
    cache = {}
    for side in ("k", "v"):
        if c["op"] == "write":  # a cache that holds nothing yet at these rows
            cache[side + "_codes"] = torch.zeros((pages, kv, page, dim // 2), dtype=torch.uint8, device="cuda")
            cache[side + "_step"] = torch.zeros((pages, kv, page), device="cuda")
            cache[side + "_bos"] = torch.zeros((pages, kv, dim), dtype=torch.int8, device="cuda")
            s[side] = _keys((s["rows"], kv, dim), g, DTYPES[c["dtype"]])
        else:
            x = _keys((pages, kv, page, dim), g, torch.float32)
            cache[side + "_codes"], cache[side + "_step"], eight = _held(x, 4)
            cache[side + "_bos"] = eight[:, :, 0].contiguous()
            # the first page of a sequence begins with its 8-bit row
            begin = table[:, 0].long()
            cache[side + "_step"][begin, :, 0] = ((x[begin, :, 0].abs().amax(-1).double() + EPS) / Q8).float()
            del x, eight
    s["cache"] = cache
    if c["op"] == "attend":
        s["q"] = torch.empty((s["rows"], c["heads"], dim), device="cuda").normal_(generator=g).to(DTYPES[c["dtype"]])
    return s


# ------------------------------------------------------------------ the plain forms
def _held(x, bits):
    """Rows x as the cache holds them: packed codes, steps, and the codes that they have at 8 bits."""
    x = x.double()  # a code next to a border is decided exactly
    biggest = x.abs().amax(-1, keepdim=True)
    stat, q, low, high = (x.abs().mean(-1, keepdim=True), Q4, -8, 7) if bits == 4 else (biggest, Q3, -4, 3)
    code = (x * (q / (stat + EPS))).round().clamp(low, high).to(torch.int16)
    packed = ((code[..., 0::2] & 15) | ((code[..., 1::2] & 15) << 4)).to(torch.uint8)
    bos = (x * (Q8 / (biggest + EPS))).round().clamp(-128, 127).to(torch.int8)
    return packed, ((stat + EPS) / q).float()[..., 0], bos


def _tokens(s):
    """Of every row of the batch: its sequence and its position there."""
    row = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["starts"][1:].long(), row, right=True)
    return b, s["lens"].long()[b] - s["starts"].long()[b + 1] + row


def _values(s, side, b, pos):
    """Cached rows as fp32 values, [..., kv, dim], at positions `pos` of sequences `b`."""
    c, page = s["cache"], s["case"]["page"]
    at, off = s["table"][b, pos // page].long().clamp(min=0), pos % page
    held = c[side + "_codes"][at, :, off].to(torch.int32)
    code = torch.stack((((held & 15) ^ 8) - 8, ((held >> 4) ^ 8) - 8), -1).flatten(-2)
    code = torch.where((pos == 0)[..., None, None], c[side + "_bos"][at].to(torch.int32), code)
    return code.float() * c[side + "_step"][at, :, off][..., None]


def _write_plain(s):
    c, cache = s["case"], s["cache"]
    b, pos = _tokens(s)
    at, off = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    zero = pos == 0
    for side in ("k", "v"):
        packed, step, bos = _held(s[side], c["bits"])
        whole = ((s[side].double().abs().amax(-1) + EPS) / Q8).float()
        cache[side + "_codes"][at, :, off] = packed
        cache[side + "_step"][at, :, off] = torch.where(zero[:, None], whole, step)
        first, row = s["table"][:, 0].long(), s["starts"][:-1].long()
        fresh = (pos[row] == 0)[:, None, None]  # the sequences that begin in this batch
        cache[side + "_bos"][first] = torch.where(fresh, bos[row], cache[side + "_bos"][first])
    return _read_plain(s)


def _read_plain(s):
    b, pos = _tokens(s)
    return tuple(_values(s, side, b, pos).to(DTYPES[s["case"]["out"]]) for side in ("k", "v"))


def _attend_plain(s):
    c, q = s["case"], s["q"]
    kv, dim, group = c["kv"], c["dim"], c["heads"] // c["kv"]
    batch, wide = c["batch"], s["longest"]
    col = torch.arange(wide, device="cuda")
    every = torch.arange(batch, device="cuda")[:, None].expand(batch, wide)
    keys, values = (_values(s, side, every, col.expand(batch, wide)).permute(0, 2, 1, 3) for side in ("k", "v"))
    b, pos = _tokens(s)
    row = torch.arange(s["rows"], device="cuda") - s["starts"].long()[b]
    padded = torch.zeros((batch, s["max_new"], c["heads"], dim), device="cuda")
    padded[b, row] = q.float()
    padded = padded.view(batch, -1, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv, -1, dim)
    score = (padded @ keys.transpose(-1, -2)) * dim ** -0.5
    score = score.view(batch, kv, group, -1, wide)
    begin = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1]).long()
    p = begin[:, None] + torch.arange(s["max_new"], device="cuda")
    seen = (col < s["lens"].long()[:, None])[:, None, :].expand(batch, s["max_new"], wide)
    if c["causal"]:
        seen = seen & (col <= p[..., None])
    if c["window"]:
        seen = seen & (col > p[..., None] - c["window"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = score.view(batch, kv, -1, wide) @ values
    out = out.view(batch, kv, group, -1, dim) / torch.where(total == 0, torch.ones_like(total), total)
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, -1, c["heads"], dim)[b, row].to(q.dtype)
    if not c["lse"]:
        return (out,)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(batch, -1, c["heads"])[b, row]
    return out, lse


# ------------------------------------------------------------------ a pass
def run(state):
    s, c = state, state["case"]
    if not own:
        return {"write": _write_plain, "read": _read_plain, "attend": _attend_plain}[c["op"]](s)
    import ternary_weight_bit_b200 as tb

    if "handle" not in s:  # a program keeps the object that holds its cache
        s["handle"] = tb.KV4Cache(**s["cache"])
    batch = (s["table"], s["lens"], s["starts"])
    if c["op"] == "attend":
        out = tb.bitnet_kv4_attention(s["q"], s["handle"], *batch, causal=c["causal"], window=c["window"],
                                      max_q=s["max_new"], return_lse=c["lse"])
        return out if c["lse"] else (out,)
    if c["op"] == "write":
        tb.bitnet_kv4_write(s["k"], s["v"], s["handle"], *batch, bits=c["bits"], eps=EPS)
    return tb.bitnet_kv4_read(s["handle"], *batch, s["rows"], dtype=DTYPES[c["out"]])


# ------------------------------------------------------------------ the definition, in 64 bits
def _sequence(s, b):
    """(first row, rows, length, pages) of sequence b."""
    start, end, m = int(s["starts"][b]), int(s["starts"][b + 1]), int(s["lens"][b])
    return start, end - start, m, s["table"][b, : -(-m // s["case"]["page"])].long()


def _wide(s, side, b):
    """Everything that the cache holds of sequence b, [kv, length, dim] in 64 bits."""
    c = s["cache"]
    _, _, m, at = _sequence(s, b)
    kv, dim = s["case"]["kv"], s["case"]["dim"]
    nibble = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1], dtype=torch.float64, device="cuda")
    held = c[side + "_codes"][at].transpose(0, 1).reshape(kv, -1, dim // 2).long()
    x = torch.empty((kv, held.shape[1], dim), dtype=torch.float64, device="cuda")
    x[..., 0::2], x[..., 1::2] = nibble[held % 16], nibble[held // 16]
    x[:, 0] = c[side + "_bos"][at[0]].double()
    return (x * c[side + "_step"][at].transpose(0, 1).reshape(kv, -1, 1).double())[:, :m]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "read":
        got = ([], [])
        for b in range(c["batch"]):
            _, n, m, _ = _sequence(s, b)
            for side, into in zip(("k", "v"), got):
                into.append(_wide(s, side, b)[:, m - n:].transpose(0, 1))
        return tuple(torch.cat(x) for x in got)
    if c["op"] == "write":
        got = []
        for side in ("k", "v"):
            x = s[side].double()
            size = x.abs()
            scale = (size.sum(-1) / c["dim"] if c["bits"] == 4 else size.max(-1).values) + EPS
            levels, low, high = (math.sqrt(7.0), -8.0, 7.0) if c["bits"] == 4 else (3.0, -4.0, 3.0)
            step = (scale / levels)[..., None]
            y = torch.clamp(torch.round(x / step), low, high) * step
            for b in range(c["batch"]):
                start, n, m, _ = _sequence(s, b)
                if n and m == n:
                    step = (size[start].max(-1).values + EPS)[..., None] / 127.0
                    y[start] = torch.clamp(torch.round(x[start] / step), -128.0, 127.0) * step
            got.append(y)
        return tuple(got)
    if _pairs(c)[0] * c["heads"] * c["dim"] > 2e12:
        return None
    outs, sums = [], []
    for b in range(c["batch"]):
        start, n, m, _ = _sequence(s, b)
        k, v = _wide(s, "k", b), _wide(s, "v", b)
        q = s["q"][start:start + n].double().view(n, c["kv"], -1, c["dim"])
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:-1], dtype=torch.float64, device="cuda")
        t = torch.arange(m, device="cuda")
        for i in range(0, n, 512):
            p = m - n + torch.arange(i, min(n, i + 512), device="cuda")[:, None]
            hide = (t > p) if c["causal"] else torch.zeros((p.shape[0], m), dtype=torch.bool, device="cuda")
            if c["window"]:
                hide = hide | (t <= p - c["window"])
            z = torch.einsum("nhgd,htd->hgnt", q[i:i + 512], k) / math.sqrt(c["dim"])
            z = z.masked_fill(hide, -math.inf)
            lse[i:i + 512] = torch.logsumexp(z, -1).permute(2, 0, 1)
            out[i:i + 512] = torch.einsum("hgnt,htd->nhgd", torch.softmax(z, -1), v)
        outs.append(out.reshape(n, c["heads"], c["dim"]))
        sums.append(lse.reshape(n, c["heads"]))
    return (torch.cat(outs), torch.cat(sums)) if c["lse"] else (torch.cat(outs),)
