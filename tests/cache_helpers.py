"""Plain forms, in 64 bits and token by token, of the 8-bit cache and the attention over it."""

import math

import torch

import lossless_entropy_coding_byte_amd as lecb

F32, BF16, F16, I8 = torch.float32, torch.bfloat16, torch.float16, torch.int8
HALF_STEP = {F32: 2.0**-24, BF16: 2.0**-8, F16: 2.0**-11}      # of a rounding, relative
SMALLEST = {F32: 2.0**-149, BF16: 2.0**-133, F16: 2.0**-24}    # a step at the bottom of the range


def padded(dim):
    return next(p for p in (64, 96, 128, 192, 256) if p >= dim)


def places(block, dim, keys):
    """Byte offset of (token, dimension) within a block's codes of one head, as lecb.h states it."""
    t, d = torch.arange(block)[:, None], torch.arange(dim)[None]
    unit = (t // 32) * (padded(dim) // 32) + d // 32
    t, d = t % 32, d % 32
    if keys:
        byte = (((d // 8) * 16 + t % 16) * 2 + t // 16) * 8 + d % 8
    else:
        byte = ((((t % 16) // 4 * 16 + d % 16) * 2 + d // 16) * 2 + t // 16) * 4 + t % 4
    return unit * 1024 + byte


def rows_of(codes, block, dim, keys):
    """int8 [blocks, heads, bytes] -> [blocks, heads, block, dim]"""
    at = places(block, dim, keys).to(codes.device)
    return codes[:, :, at.view(-1)].view(*codes.shape[:2], block, dim)


def random_cache(g, blocks, heads, dim, block, device, spread=0.5):
    """A cache of random codes (on `device`) whose blocks have scales of different size; g: a CPU generator."""
    cache = lecb.new_cache_q8(blocks, heads, dim, block, device="cpu")
    for codes, keys in ((cache.k, True), (cache.v, False)):
        x = (30 * torch.randn(blocks, heads, block, dim, generator=g)).round().clamp(-127, 127).to(I8)
        codes[:, :, places(block, dim, keys).view(-1)] = x.view(blocks, heads, -1)
    for s in (cache.k_scale, cache.v_scale):
        s.copy_(torch.exp(spread * torch.randn(blocks, heads, generator=g)) / 30)
    return lecb.CacheQ8(*(t.to(device) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)), dim, block)


def host(cache):
    return lecb.CacheQ8(*(t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)), cache.dim, cache.block)


def values(cache):
    """The numbers that a cache's codes stand for: keys and values, float64 [blocks, heads, block, dim]."""
    c = host(cache)
    return tuple(rows_of(q, c.block, c.dim, keys).double() * s.double()[:, :, None, None]
                 for q, s, keys in ((c.k, c.k_scale, True), (c.v, c.v_scale, False)))


def tables(g, lengths, block, blocks, device, width=None):
    """A table that gives each sequence blocks of its own, anywhere; entries past them are -1."""
    need = [-(-n // block) for n in lengths]
    order = torch.randperm(blocks, generator=g).tolist()
    assert sum(need) <= blocks
    table = torch.full((len(lengths), width or max(1, *need)), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        table[s, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    return table.to(device), torch.tensor(lengths, dtype=torch.int32, device=device)


def starts_of(news, device, first=0):
    at = [first]
    for n in news:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=device)


def attention(q, cache, table, lengths, starts=None, scale=None, causal=True, window=None):
    """(out, tolerance), float64 [tokens, heads, dim], of the formula on the numbers that the cache holds.

    The tolerance adds up, for each element, with A = sum p |v| and n tokens seen:
    * scores: a product of dim terms in 32 bits, (dim + 8) 2^-24 of sum |q k| scale with its factors' roundings and
      the exponent's; the same again for the row's maximum; 2^-22 of the exponential;  p changes by that times p, the quotient
      by twice its most;
    * a weight's rounding for the second product: 2^-11 where results are bfloat16, else 2^-22;
    * sums: parts of 32, one after another: (48 + n / 32) 2^-24 of A, twice with the denominator;
    * halves, whose smallest step is 2^-24, hold the largest weight times its scale as 2^11 or more: half a step, 2^-36 of it,
      times codes to 127, for each token;
    * the last rounding, half a step."""
    k, v = values(cache)
    q64, dim, block = q.cpu().double(), cache.dim, cache.block
    table, lengths = table.cpu().long(), lengths.cpu().tolist()
    starts = list(range(len(lengths) + 1)) if starts is None else starts.cpu().tolist()
    scale = 1 / math.sqrt(dim) if scale is None else scale
    group = q.shape[1] // cache.k_scale.shape[1]
    out, tol = torch.zeros_like(q64), torch.zeros_like(q64)
    weight = 2.0**-11 if q.dtype == BF16 else 2.0**-22
    for s, n in enumerate(lengths):
        rows = range(starts[s], starts[s + 1])
        if n == 0 or not len(rows):
            continue
        pages = table[s, : -(-n // block)]
        steps = cache.v_scale.cpu().double()[pages].t().repeat_interleave(block, 1)[:, :n]   # [heads, n]
        ks, vs = (x[pages].transpose(0, 1).flatten(1, 2)[:, :n] for x in (k, v))   # [heads, n, dim]
        for i, row in enumerate(rows):
            pos = n - len(rows) + i
            hi = pos + 1 if causal else n
            lo = max(0, pos - window + 1) if window else 0
            if hi <= lo:
                continue
            x = q64[row].view(-1, group, dim)
            kk, vv = ks[:, lo:hi], vs[:, lo:hi]
            score = (x @ kk.transpose(1, 2)) * scale
            size = ((x.abs() @ kk.abs().transpose(1, 2)) * abs(scale)).amax(2, keepdim=True)
            p = torch.softmax(score, 2)
            out[row] = (p @ vv).reshape(-1, dim)
            a = (p @ vv.abs())
            e = 2 * ((dim + 8) * 2.0**-24 * size + 2.0**-22) + weight + 2 * (48 + (hi - lo) / 32) * 2.0**-24
            low = 127 * (hi - lo) * 2.0**-36 * (p * steps[:, None, lo:hi]).amax(2, keepdim=True)
            tol[row] = (2 * e * a + low).reshape(-1, dim)
    return out, tol + HALF_STEP[q.dtype] * (out.abs() + tol) + SMALLEST[q.dtype]


def write(cache, k, v, table, lengths, starts=None):
    """The rows' codes and scales as the formula has them: changes a copy of the cache on the host, token order; returns
    (keys' codes, values' codes, k_scale, v_scale) with codes int8 [blocks, heads, block, dim]."""
    c = host(cache)
    table, lengths = table.cpu().tolist(), lengths.cpu().tolist()
    starts = list(range(len(lengths) + 1)) if starts is None else starts.cpu().tolist()
    block, result = c.block, []
    for x, codes, scale, keys in ((k, c.k, c.k_scale, True), (v, c.v, c.v_scale, False)):
        x, codes = x.cpu().double(), rows_of(codes, block, c.dim, keys).clone()
        for s, n in enumerate(lengths):
            new = starts[s + 1] - starts[s]
            if n > len(table[s]) * block:
                continue
            old = n - new
            for j in range(max(0, old) // block, -(-n // block) if new else 0):
                lo, hi = max(0, old - j * block), min(block, n - j * block)
                page = table[s][j]
                if hi <= lo or not 0 <= page < codes.shape[0]:
                    continue
                first = starts[s] + j * block + lo - old
                part = x[first : first + hi - lo].transpose(0, 1)          # [heads, tokens, dim]
                for h in range(codes.shape[1]):
                    most = part[h].abs().max()
                    need = (most / 127).float() if torch.isfinite(part[h]).all() else torch.tensor(math.nan)
                    step = need
                    if lo:
                        was = scale[page, h].clone()
                        if torch.isnan(was) or need <= was:
                            step = was
                        else:
                            step = torch.maximum(need, 1.25 * was) if not torch.isnan(need) else need
                            codes[page, h, :lo] = _codes(codes[page, h, :lo].double() * was.double(), step)
                    scale[page, h] = step
                    codes[page, h, lo:hi] = _codes(part[h], step)
        result.append((codes, scale))
    return result[0][0], result[1][0], result[0][1], result[1][1]


def _codes(x, step):
    """x / step to nearest, ties to even: the quotient in 64 bits never lies nearer to half a step than it is exact."""
    step = step.double()
    if not step > 0:
        return torch.zeros(x.shape, dtype=I8)
    return (x / step).round().clamp(-127, 127).to(I8)
