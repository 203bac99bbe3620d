"""The 8-bit cache of keys and values and the attention over it, as cases to be timed and compared.

* ``cache``   new tokens' keys and values quantised into the blocks of a cache
  (``cache_write_q8``), and the blocks that they touched read back
  (``cache_read_q8``);
* ``attend``  attention of queries over such a cache (``attention_q8``).

``own`` chooses who computes them: false, elementary torch operations; true, the
framework.

The cache: blocks of ``block`` tokens; a sequence's block j is row table[s, j] of
the cache, its length counts the new tokens too, and its new tokens, rows
starts[s] .. starts[s + 1] of the inputs, are its last.  Each block has one scale
for each head's keys and one for its values; a code q stands for q * scale.

Formulas:

* writing, for the new tokens of one block and head: need = max|x| / 127; where
  the block holds older tokens, their scale stays if need is not above it, and
  else becomes max(need, 1.25 scale), the older codes being rounded again:
  q scale / new scale; where it holds none, the scale is need.  q = x / scale,
  to nearest, ties to even;
* attention, for query i at position p_i and head h, whose keys are those of head
  h // (heads / kv_heads): o = sum_j softmax_j(q_i . k_j / sqrt(dim)) v_j over
  p_i - window < j <= p_i (without a window: 0 <= j); zeros where there is none.

Order of the codes: units of 32 tokens x 32 dimensions, 1 KiB (dimensions padded
with zeros to 64, 96, 128, 192 or 256), along the dimensions, then along the
tokens.  Byte by byte, slowest first: keys [(d % 32) / 8][t % 16][t / 16][d % 8],
values [(t % 16) / 4][d % 16][(d % 32) / 16][t / 16][t % 4].
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GROW = 1.25


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one request's newest token goes into its cache
        {"name": "append_token", "op": "cache", "seqs": 1, "new": 1, "ragged": False, "len": 1000, "kv_heads": 8,
         "dim": 128, "block": 64, "type": "bf16"},
        # the newest tokens of 64 requests of every length
        {"name": "append_batch", "op": "cache", "seqs": 64, "new": 1, "ragged": True, "len": 8192, "kv_heads": 8,
         "dim": 128, "block": 64, "type": "bf16"},
        # odd heads, odd numbers of tokens, some of them after half a block
        {"name": "write_odd", "op": "cache", "seqs": 5, "new": 301, "ragged": True, "len": 555, "kv_heads": 3, "dim": 80,
         "block": 32, "type": "fp16"},
        # eight prompts of 2048 tokens: the tokens of the int8 activation workload
        {"name": "write_prompts", "op": "cache", "seqs": 8, "new": 2048, "ragged": False, "len": 2048, "kv_heads": 8,
         "dim": 128, "block": 64, "type": "bf16"},
        # a decode step of one request: latency
        {"name": "attend_token", "op": "attend", "seqs": 1, "new": 1, "ragged": False, "len": 1000, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 64, "type": "bf16", "window": 0},
        # a decode step of 64 requests of every length
        {"name": "attend_batch", "op": "attend", "seqs": 64, "new": 1, "ragged": True, "len": 8192, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 64, "type": "bf16", "window": 0},
        # one token after a very long text
        {"name": "attend_long", "op": "attend", "seqs": 1, "new": 1, "ragged": False, "len": 262144, "heads": 64,
         "kv_heads": 8, "dim": 128, "block": 64, "type": "bf16", "window": 0},
        # odd heads and dimensions, a few new tokens or none, a request that has no tokens yet, a sliding window
        {"name": "attend_odd", "op": "attend", "seqs": 7, "new": 9, "ragged": True, "len": 2999, "heads": 15,
         "kv_heads": 3, "dim": 80, "block": 32, "type": "fp16", "window": 1000},
        # drafted tokens looked over at once, one key head for each query head, handed on in 32 bits
        {"name": "attend_draft", "op": "attend", "seqs": 16, "new": 5, "ragged": False, "len": 4097, "heads": 16,
         "kv_heads": 16, "dim": 64, "block": 128, "type": "fp32", "window": 0},
        # wide heads that share one or two key heads and see a window
        {"name": "attend_wide", "op": "attend", "seqs": 8, "new": 1, "ragged": True, "len": 16384, "heads": 16,
         "kv_heads": 2, "dim": 256, "block": 32, "type": "bf16", "window": 4096},
        # two prompts from their beginning
        {"name": "attend_prompts", "op": "attend", "seqs": 2, "new": 4096, "ragged": True, "len": 4096, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 64, "type": "bf16", "window": 0},
        # a chunk of a long prompt
        {"name": "attend_chunk", "op": "attend", "seqs": 1, "new": 512, "ragged": False, "len": 32768, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 64, "type": "bf16", "window": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("cache", "attend", "attend"))
    c = {"op": op, "block": rng.choice((32, 64, 128, 256)), "kv_heads": rng.choice((1, 2, 4, 8, 8, _log(rng, 1, 32))),
         "dim": rng.choice((64, 128, 128, 256, rng.randint(16, 256))), "type": rng.choice(("bf16", "bf16", "fp16", "fp32")),
         "ragged": rng.random() < 0.7}
    row = c["kv_heads"] * max(c["dim"], 64)
    if op == "cache":
        c["seqs"] = _log(rng, 1, 64)
        c["new"] = rng.choice((1, _log(rng, 1, max(1, min(4096, (1 << 24) // (row * c["seqs"]))))))
        c["len"] = max(c["new"], _log(rng, 1, max(1, min(16384, (1 << 27) // (row * c["seqs"])))))
        return c
    group = rng.choice((1, 4, 8, rng.randint(1, 16)))
    c["heads"] = group * c["kv_heads"]
    c["seqs"] = rng.choice((1, _log(rng, 1, 64)))
    c["len"] = _log(rng, 16, max(16, min(262144, (1 << 28) // (row * c["seqs"]))))
    pairs = (1 << 36) // (c["heads"] * max(c["dim"], 64) * c["seqs"] * c["len"])
    c["new"] = rng.choice((1, min(c["len"], _log(rng, 1, 16)), min(c["len"], _log(rng, 1, max(1, min(4096, pairs // 4))))))
    c["new"] = max(1, min(c["new"], pairs))
    c["window"] = rng.choice((0, 0, _log(rng, 1, c["len"])))
    return c


def _sizes(c):
    """Each sequence's new tokens and its length with them.  Ragged: both spread over
    their range, with a sequence that has none and one of a single token where there are more than four."""
    n, length = [c["new"]] * c["seqs"], [c["len"]] * c["seqs"]
    if c["ragged"]:
        step = 0.6180339887498949
        for s in range(1, c["seqs"]):
            f = (s * step) % 1.0
            length[s] = max(1, int(c["len"] * f))
            if c["new"] > 1:
                n[s] = min(length[s], int(c["new"] * ((s * step * step) % 1.0)))
        if c["seqs"] > 4:
            length[3] = 1
            n[3] = min(n[3], 1)
            if c["op"] == "attend" and c["new"] > 1:
                length[2] = n[2] = 0
    return n, length


def _bytes(t):
    return {"bf16": 2, "fp16": 2, "fp32": 4}[t]


def work(case):
    c, b = case, _bytes(case["type"])
    n, length = _sizes(c)
    if c["op"] == "cache":
        new = sum(n)
        back = sum(x - (x - m) // c["block"] * c["block"] if m else 0 for m, x in zip(n, length))
        touched = sum(-(-x // c["block"]) - (x - m) // c["block"] if m else 0 for m, x in zip(n, length))
        row = 2 * c["kv_heads"] * c["dim"]
        return {"bytes": row * (new * (b + 1) + back * (1 + b)) + touched * c["kv_heads"] * 16, "flops": row * (3 * new + back)}
    w = c["window"] or 1 << 40
    pairs = read = 0
    for m, x in zip(n, length):
        if not m:
            continue
        read += x - max(0, x - m - w + 1)
        # of the queries at x - m .. x - 1, each sees min(position + 1, window) keys
        a, e = x - m + 1, x
        full = max(0, e - max(a, w) + 1) if e >= w else 0
        rest = m - full
        pairs += full * w + rest * a + rest * (rest - 1) // 2 if full else (a + e) * m // 2
    return {"bytes": 2 * read * c["kv_heads"] * c["dim"] + 2 * sum(n) * c["heads"] * c["dim"] * b,
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# ---------------------------------------------------------------- inputs

def _padded(dim):
    return next(p for p in (64, 96, 128, 192, 256) if p >= dim)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    t, h, d, block, seqs = TYPES[c["type"]], c["kv_heads"], c["dim"], c["block"], c["seqs"]
    n, length = _sizes(c)
    pages = [-(-x // block) for x in length]
    width, count = max(1, max(pages)), max(1, sum(pages))
    units, tiles = _padded(d) // 32, block // 32

    def codes(keys):
        # what quantised keys and values look like: about normal, a few dimensions far larger than the others
        x = torch.randn(count, h, tiles, units, 1024, device=DEV, generator=g)
        if keys:
            x.mul_(torch.where(torch.rand(1, h, 1, units, 4, 1, 1, 8, device=DEV, generator=g) < 0.02, 3.0, 1.0)
                   .expand(1, h, 1, units, 4, 16, 2, 8).reshape(1, h, 1, units, 1024))
        x = x.mul_(30).round_().clamp_(-127, 127).to(torch.int8).view(count, h, tiles, units, 1024)
        if d % 32 or units * 32 > d:   # the padding's codes are zeros
            dims = torch.arange(units * 32, device=DEV).view(units, 32)
            if keys:
                dims = dims.view(units, 4, 1, 1, 8).expand(units, 4, 16, 2, 8)
            else:
                dims = dims.view(units, 1, 2, 16, 1, 1).permute(0, 1, 3, 2, 4, 5).expand(units, 4, 16, 2, 2, 4)
            x = x.masked_fill_(dims.reshape(units, 1024) >= d, 0)
        return x

    def steps():
        return (1 + 0.6 * torch.rand(count, h, device=DEV, generator=g)) / 36

    # blocks stand anywhere in the cache; entries past a sequence's blocks are of no meaning
    order = torch.randperm(count, device=DEV, generator=g).to(torch.int32)
    table = torch.full((seqs, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, p in enumerate(pages):
        table[s, :p] = order[at : at + p]
        at += p
    starts = [sum(n[:s]) for s in range(seqs + 1)]
    state = {"case": c, "k": codes(True), "v": codes(False), "k_scale": steps(), "v_scale": steps(), "table": table,
             "lengths": torch.tensor(length, dtype=torch.int32, device=DEV),
             "starts": torch.tensor(starts, dtype=torch.int32, device=DEV), "tokens": starts[-1], "single": c["new"] == 1}
    if c["op"] == "cache":
        def fresh():
            # tokens of different size: some of them past what a block has held so far
            x = torch.randn(starts[-1], h, d, device=DEV, generator=g)
            return x.mul_(torch.exp(0.3 * torch.randn(starts[-1], 1, 1, device=DEV, generator=g))).to(t)

        first = [(x - m) // block for m, x in zip(n, length)]
        last = [-(-x // block) if m else f for m, x, f in zip(n, length, first)]
        back = [0]
        for m, x, f in zip(n, length, first):
            back.append(back[-1] + (x - f * block if m else 0))
        spans = [(s, j) for s in range(seqs) for j in range(first[s], last[s])]
        state.update(new_k=fresh(), new_v=fresh(), back=torch.tensor(back, dtype=torch.int32, device=DEV),
                     back_tokens=back[-1], spans=torch.tensor(spans, dtype=torch.int64, device=DEV).view(-1, 2),
                     held=torch.tensor([j * block + i - f * block + b for (s, j), f, b in
                                        ((p, first[p[0]], back[p[0]]) for p in spans) for i in range(block)],
                                       dtype=torch.int64, device=DEV).view(-1, block))
    else:
        state.update(q=(2 * torch.randn(starts[-1], c["heads"], d, device=DEV, generator=g)).to(t),
                     most=max(n), longest=max(length))
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return _cache(c, state) if c["op"] == "cache" else _attend(c, state)


def _own(c, s):
    import lossless_entropy_coding_byte_amd as lecb

    cache = s.get("handle")
    if cache is None:   # a program makes it once, for all its steps
        cache = s["handle"] = lecb.CacheQ8(s["k"], s["v"], s["k_scale"], s["v_scale"], c["dim"], c["block"])
    starts = None if s["single"] else s["starts"]
    if c["op"] == "cache":
        lecb.cache_write_q8(cache, s["new_k"], s["new_v"], s["table"], s["lengths"], starts)
        k, v = lecb.cache_read_q8(cache, s["table"], s["lengths"], s["back"], s["back_tokens"], TYPES[c["type"]])
        return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return lecb.attention_q8(s["q"], cache, s["table"], s["lengths"], starts, window=c["window"] or None)


def _rows_of_keys(codes):
    """[blocks, heads, tiles, units, 1024] -> [blocks, heads, tokens, dims]"""
    b, h, tiles, units = codes.shape[:4]
    return codes.view(b, h, tiles, units, 4, 16, 2, 8).permute(0, 1, 2, 6, 5, 3, 4, 7).reshape(b, h, tiles * 32, units * 32)


def _rows_of_values(codes):
    b, h, tiles, units = codes.shape[:4]
    return (codes.view(b, h, tiles, units, 4, 16, 2, 2, 4).permute(0, 1, 2, 7, 4, 8, 3, 6, 5)
            .reshape(b, h, tiles * 32, units * 32))


def _keys_of_rows(rows):
    b, h, block, dims = rows.shape
    return (rows.view(b, h, block // 32, 2, 16, dims // 32, 4, 8).permute(0, 1, 2, 5, 6, 4, 3, 7)
            .reshape(b, h, block // 32, dims // 32, 1024))


def _values_of_rows(rows):
    b, h, block, dims = rows.shape
    return (rows.view(b, h, block // 32, 2, 4, 4, dims // 32, 2, 16).permute(0, 1, 2, 6, 4, 8, 7, 3, 5)
            .reshape(b, h, block // 32, dims // 32, 1024))


def _cache(c, s):
    block, d = c["block"], c["dim"]
    seq, j = s["spans"][:, 0], s["spans"][:, 1]
    page = s["table"][seq, j].long()
    length, begin = s["lengths"].long()[seq], s["starts"].long()
    old = length - (begin[seq + 1] - begin[seq])               # tokens held before
    pos = j[:, None] * block + torch.arange(block, device=page.device)
    fresh = (pos >= old[:, None]) & (pos < length[:, None])
    token = (begin[seq][:, None] + pos - old[:, None]).clamp(0, s["tokens"] - 1)
    kept = (j * block < old)[:, None]

    def write(x, codes, scale, rows_of, of_rows):
        rows = rows_of(codes[page])[..., :d]                                  # [spans, heads, block, d]
        x = x[token].permute(0, 2, 1, 3)                                      # the same, of the new tokens
        need = torch.where(fresh[:, None, :, None], x, 0).abs().amax((2, 3)).double().div(127).float()
        was = torch.where(kept, scale[page], 0)
        step = torch.where(need > was, torch.maximum(need, GROW * was), was)
        # the quotients in 64 bits: what lies half a step between two codes goes to the even one, all else to its nearest
        q = torch.where(fresh[:, None, :, None], x.double(), rows * was.double()[:, :, None, None])
        q = torch.where(step[:, :, None, None] > 0, q / step.double()[:, :, None, None], 0)
        rows = torch.nn.functional.pad(q.round().clamp(-127, 127).to(torch.int8), (0, codes.shape[3] * 32 - d))
        codes[page] = of_rows(rows)
        scale[page] = step
        values = rows_of(codes[page])[..., :d].float() * scale[page][:, :, None, None]
        values = values.permute(0, 2, 1, 3).reshape(-1, c["kv_heads"], d).to(TYPES[c["type"]])
        held = (pos < length[:, None]).view(-1)
        out = torch.empty(s["back_tokens"] + 1, c["kv_heads"], d, dtype=values.dtype, device=values.device)
        out[torch.where(held, s["held"].view(-1), s["back_tokens"])] = values   # what is past the end goes to the last row
        return out[:-1]

    return {"k": write(s["new_k"], s["k"], s["k_scale"], _rows_of_keys, _keys_of_rows),
            "v": write(s["new_v"], s["v"], s["v_scale"], _rows_of_values, _values_of_rows),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _attend(c, s):
    d, h, seqs, most = c["dim"], c["kv_heads"], c["seqs"], s["most"]
    group, pages = c["heads"] // h, -(-max(1, s["longest"]) // c["block"])
    page = s["table"][:, :pages].clamp_min(0).long().view(-1)
    length, begin = s["lengths"].long(), s["starts"].long()
    new = begin[1:] - begin[:-1]

    def values(codes, scale, rows_of):
        x = rows_of(codes[page])[..., :d].float() * scale[page][:, :, None, None]
        return x.view(seqs, pages, h, c["block"], d).permute(0, 2, 1, 3, 4).reshape(seqs, h, pages * c["block"], d)

    # queries, as many for each sequence as the most that one has
    i = torch.arange(most, device=page.device)
    row = (begin[:-1, None] + i).clamp_max(s["tokens"] - 1)
    q = s["q"][row].float().view(seqs, most, h, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, h, most * group, d)
    at = (length - new)[:, None] + i                                          # their positions
    key = torch.arange(pages * c["block"], device=page.device)
    seen = (key <= at[:, :, None]) & (i < new[:, None])[:, :, None]
    if c["window"]:
        seen = seen & (key > at[:, :, None] - c["window"])
    seen = seen[:, None, :, None, :].expand(-1, -1, -1, group, -1).reshape(seqs, 1, most * group, -1)
    score = q @ values(s["k"], s["k_scale"], _rows_of_keys).transpose(2, 3).contiguous()
    score = score.mul_(1 / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    score = (score - score.amax(3, keepdim=True).clamp_min(torch.finfo(torch.float32).min)).exp_()
    total = score.sum(3, keepdim=True)
    out = score @ values(s["v"], s["v_scale"], _rows_of_values)
    out = torch.where(total > 0, out / total, 0).view(seqs, h, most, group, d).permute(0, 2, 1, 3, 4)
    token = torch.arange(s["tokens"], device=page.device)
    seq = torch.searchsorted(begin, token, right=True) - 1
    return out[seq, token - begin[seq]].reshape(s["tokens"], c["heads"], d).to(s["q"].dtype)


# ---------------------------------------------------------------- in 64 bits

def _taken(codes, dims, tokens, keys):
    """Codes of the given tokens (places in a block) by their byte addresses, [blocks, heads, tokens, dims] in 64 bits."""
    units = codes.shape[3]
    t, e = tokens[:, None], dims[None, :]
    if keys:
        byte = ((e % 32 // 8 * 16 + t % 16) * 2 + t % 32 // 16) * 8 + e % 8
    else:
        byte = (((t % 16 // 4 * 16 + e % 16) * 2 + e % 32 // 16) * 2 + t % 32 // 16) * 4 + t % 4
    at = ((t // 32 * units + e // 32) * 1024 + byte).view(-1)
    return codes.flatten(2)[:, :, at].unflatten(2, (len(tokens), len(dims))).to(torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    c, f64 = s["case"], torch.float64
    n, length = _sizes(c)
    block, d = c["block"], c["dim"]
    dims, places = torch.arange(d, device=DEV), torch.arange(block, device=DEV)
    table, first = s["table"].tolist(), s["starts"].tolist()
    if c["op"] == "cache":
        out = {}
        for name in ("k", "v"):
            scale, parts = s[name + "_scale"].clone(), []
            for q in range(c["seqs"]):
                old = length[q] - n[q]
                for j in range(old // block, -(-length[q] // block) if n[q] else 0):
                    page, lo, hi = table[q][j], max(0, old - j * block), min(block, length[q] - j * block)
                    x = s["new_" + name][first[q] + j * block + lo - old :][: hi - lo].to(f64).transpose(0, 1)
                    step = (torch.linalg.vector_norm(x, ord=math.inf, dim=(1, 2)) / 127).float()
                    held = torch.empty(c["kv_heads"], 0, d, device=DEV, dtype=f64)
                    if lo:
                        was = scale[page]
                        step = torch.where(step <= was, was, torch.maximum(step, was * GROW))
                        held = _taken(s[name][page : page + 1], dims, places[:lo], name == "k")[0] * was.to(f64)[:, None, None]
                    scale[page] = step
                    step = step.to(f64)[:, None, None]
                    parts.append((torch.round(torch.cat((held, x), 1) / step.clamp_min(1e-300)) * step).transpose(0, 1))
            out[name] = torch.cat(parts)
            out[name + "_scale"] = scale.to(f64)
        return {k: out[k] for k in ("k", "v", "k_scale", "v_scale")}
    out = torch.zeros(s["tokens"], c["heads"], d, device=DEV, dtype=f64)
    group = c["heads"] // c["kv_heads"]
    for q in range(c["seqs"]):
        if not n[q]:
            continue
        begin = max(0, length[q] - n[q] - c["window"] + 1) // block * block if c["window"] else 0
        pages = s["table"][q, begin // block : -(-length[q] // block)].long()
        pos = torch.arange(length[q] - n[q], length[q], device=DEV)[:, None]
        key = torch.arange(begin, begin + len(pages) * block, device=DEV)[None]
        away = (key > pos) if not c["window"] else (key > pos) | (key + c["window"] <= pos)
        for h in range(c["kv_heads"]):
            k = _taken(s["k"][pages, h : h + 1], dims, places, True)[:, 0] * s["k_scale"][pages, h].to(f64)[:, None, None]
            v = _taken(s["v"][pages, h : h + 1], dims, places, False)[:, 0] * s["v_scale"][pages, h].to(f64)[:, None, None]
            k, v = k.reshape(-1, d).t().contiguous(), v.reshape(-1, d)
            for e in range(h * group, (h + 1) * group):
                x = torch.mm(s["q"][first[q] : first[q + 1], e].to(f64), k).div_(math.sqrt(d))
                p = torch.softmax(x.masked_fill_(away, -math.inf), 1)
                out[first[q] : first[q + 1], e] = torch.mm(p, v)
    return out
