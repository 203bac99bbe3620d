"""Attention over the 8-bit cache at the ends of its scales' range, for many rows as for few; cache_helpers.attention derives
the tolerance."""

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from cache_helpers import BF16, F16, F32, attention, places, random_cache, starts_of, tables
from test_gpu_attention import near, queries
from test_gpu_layers import DEV, gen

pytestmark = pytest.mark.gpu
TYPES = [BF16, F16, F32]
SMALL = [2.0**-60, 2.0**-99, 2.0**-100, 2.0**-108, 2.0**-109, 2.0**-110, 2.0**-126, 2.0**-127, 2.0**-149]


def lost(tokens):
    """What scales of values below 2^-60 may lose besides: halves hold weights times max(scale, 2^-60) to 2^-36 of the
    largest, which is 2^-60 at most where all scales are below that; times codes to 127, for each token."""
    return 127 * tokens * 2.0**-96


FAR = [(2.0**-59, 2.0**119), (2.0**-149, 2.0**119), (2.0**-30, 2.0**90), (2.0**40, 2.0**101)]


def check_far_apart(low, high, dtype, length, rows):
    """Blocks whose scales are far apart, in either order, with equal weights and with any: the sum of weights counts all."""
    g = gen(11)
    n = -(-length // 32)
    for first, second in ((low, high), (high, low)):
        cache = random_cache(g, n, 1, 64, 32, DEV)
        table, lens = tables(g, [length], 32, n, DEV)
        starts = starts_of([rows], DEV)
        cache.v_scale[table[0, : n // 2].long()] = first
        cache.v_scale[table[0, n // 2 :].long()] = second
        for q in (torch.zeros(rows, 2, 64, dtype=dtype, device=DEV), queries(g, rows, 2, 64, dtype)):
            want, tol = attention(q, cache, table, lens, starts)
            near(lecb.attention_q8(q, cache, table, lens, starts), want, tol + lost(length))


@pytest.mark.parametrize("low,high", FAR)
@pytest.mark.parametrize("dtype,length,rows", [(BF16, 300, 3), (F32, 300, 3), (F32, 300, 200), (BF16, 5000, 1), (F32, 5000, 1),
                                               (F32, 5000, 40)])
def test_scales_far_apart(dtype, length, rows, low, high):
    check_far_apart(low, high, dtype, length, rows)


@pytest.mark.parametrize("low,high", FAR)
@pytest.mark.parametrize("length,rows", [(300, 200), (5000, 300)])
def test_scales_far_apart_for_many_rows(length, rows, low, high):
    check_far_apart(low, high, BF16, length, rows)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_a_block_of_tiny_values_among_others(dim, dtype):
    """Many rows: those that see the block get what the others give, those before it and past its window do not change."""
    g = gen(dim)
    cache = random_cache(g, 22, 1, dim, 32, DEV)
    table, lens = tables(g, [320, 200], 32, 22, DEV)
    news = [300, 120]
    starts = starts_of(news, DEV)
    q = queries(g, sum(news), 2, dim, dtype)
    block, ordinary = table[0, 5].item(), cache.v_scale.clone()      # tokens 160 .. 191: rows 140 .. 171
    for window in (None, 64):
        away = torch.ones(sum(news), dtype=torch.bool, device=DEV)
        away[140 : 300 if window is None else 172 + 63] = False
        plain = lecb.attention_q8(q, cache, table, lens, starts, window=window)
        for scale in SMALL:
            for sign in (1, -1):
                cache.v_scale[block] = sign * scale
                got = lecb.attention_q8(q, cache, table, lens, starts, window=window)
                assert torch.equal(got[away], plain[away])
            want, tol = attention(q, cache, table, lens, starts, window=window)
            near(got, want, tol + lost(320))
        cache.v_scale.copy_(ordinary)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("field", ["k_scale", "v_scale"])
def test_a_block_kept_for_tokens_to_come(field, dtype):
    """The block behind a sequence's last, an odd one, whose scales nobody has written: the same bits whatever they hold."""
    g = gen(7)
    cache = random_cache(g, 12, 2, 128, 32, DEV)
    table, lens = tables(g, [288], 32, 12, DEV, width=10)
    table[0, 9] = next(b for b in range(12) if b not in table[0].tolist())
    starts = starts_of([288], DEV)
    q = queries(g, 288, 4, 128, dtype)
    want = lecb.attention_q8(q, cache, table, lens, starts)
    for scale in SMALL + [0.0, 3e38, float("inf"), float("nan")]:
        getattr(cache, field)[table[0, 9].item()] = scale
        assert torch.equal(lecb.attention_q8(q, cache, table, lens, starts), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", SMALL)
def test_both_forms_on_the_same_rows(scale, dtype):
    """Rows of a prompt, and each of them alone, over blocks of tiny values and of ordinary ones."""
    g = gen(9)
    cache = random_cache(g, 10, 1, 64, 32, DEV)
    table, lens = tables(g, [300], 32, 10, DEV)
    cache.v_scale[table[0, ::3].long()] = scale
    q = queries(g, 300, 1, 64, dtype)
    want, tol = attention(q, cache, table, lens, starts_of([300], DEV))
    near(lecb.attention_q8(q, cache, table, lens, starts_of([300], DEV)), want, tol + lost(300))
    rows = torch.arange(0, 300, 7)
    each = (rows + 1).to(torch.int32).to(DEV)
    got = lecb.attention_q8(q[rows.to(DEV)], cache, table.repeat(len(rows), 1), each)
    near(got, want[rows], tol[rows] + lost(300))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news", [7, 200])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_block_whose_keys_are_no_numbers(bad, news, dtype):
    """Rows that see it are NaN, whatever the sign of their products with its codes; others are what they are."""
    g = gen(13)
    cache = random_cache(g, 10, 1, 64, 32, DEV)
    table, lens = tables(g, [300], 32, 10, DEV)
    keys = cache.k.cpu()
    keys[table[0, 9].item()] = keys[table[0, 9].item()].abs()      # tokens 288 .. 299, the last twelve rows
    cache.k.copy_(keys)
    starts = starts_of([news], DEV)
    for sign in (1, -1):
        q = sign * queries(g, news, 2, 64, dtype).abs()
        cache.k_scale[table[0, 9].item()] = 0.03
        want, tol = attention(q, cache, table, lens, starts)
        cache.k_scale[table[0, 9].item()] = bad
        got = lecb.attention_q8(q, cache, table, lens, starts)
        sees = min(news, 12)
        assert bool(got[news - sees :].isnan().all())
        near(got[: news - sees], want[: news - sees], tol[: news - sees])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("news", [3, 200])
@pytest.mark.parametrize("size", [2.0**-133, 2.0**-126, 2.0**-120, 2.0**-112, 2.0**-60, 2.0**100, 2.0**120])
def test_queries_and_keys_of_opposite_size(size, news, dtype):
    """Scores of ordinary size out of queries near either end of the range and keys near the other."""
    g = gen(17)
    cache = random_cache(g, 10, 1, 64, 32, DEV)
    cache.k_scale.mul_(min(2.0**120, 0.25 / size))
    table, lens = tables(g, [300], 32, 10, DEV)
    starts = starts_of([news], DEV)
    q = (size * torch.randn(news, 2, 64, generator=g).double()).to(dtype).to(DEV)
    for scale in (None, 2.0**-40):
        if scale is not None:
            cache.k_scale.mul_(2.0**30 if size > 1 else 1.0)
        want, tol = attention(q, cache, table, lens, starts, scale=scale)
        near(lecb.attention_q8(q, cache, table, lens, starts, scale=scale), want, tol)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news", [12, 300])
def test_rows_of_one_call_that_see_different_blocks(news, dtype):
    """A block that some rows of a call see and others do not, bad in each way: the others' results are the formula's, those
    of rows before it the same bits.  Codes behind the end are left over from other tokens."""
    g = gen(19)
    cache = random_cache(g, 14, 2, 80, 32, DEV)
    for first in (384, (390 - news // 2) // 32 * 32):      # the last block, and one in the middle of the rows
        table, lens = tables(g, [390], 32, 14, DEV)
        at, starts = first // 32, starts_of([news], DEV)
        q = queries(g, news, 4, 80, dtype)
        page, kept = table[0, at].item(), [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale, table)]
        want, tol = attention(q, cache, table, lens, starts, window=40)
        plain = lecb.attention_q8(q, cache, table, lens, starts, window=40)
        pos = torch.arange(390 - news, 390)
        before, past = pos < first, pos - 39 > first + 31
        for change in (lambda: cache.k_scale[page].fill_(float("inf")), lambda: cache.k_scale[page].fill_(float("nan")),
                       lambda: cache.v_scale[page].fill_(-float("inf")), lambda: cache.v_scale[page].fill_(float("nan")),
                       lambda: cache.v_scale[page].fill_(3e38), lambda: cache.v_scale[page].fill_(2.0**-149),
                       lambda: cache.k[page].fill_(-128), lambda: cache.v[page].fill_(-128),
                       lambda: table[0, at].fill_(-1), lambda: table[0, at].fill_(14), lambda: table[0, at].fill_(1 << 30)):
            change()
            got = lecb.attention_q8(q, cache, table, lens, starts, window=40)
            assert torch.equal(got[before.to(DEV)], plain[before.to(DEV)])
            near(got[past.to(DEV)], want[past], tol[past])
            for t, was in zip((cache.k, cache.v, cache.k_scale, cache.v_scale, table), kept):
                t.copy_(was)
        # codes behind the sequence's end
        for c, keys in ((cache.k, True), (cache.v, False)):
            c[table[0, 12].item()][:, places(32, 80, keys)[390 - 384 :].reshape(-1)] = -128
        assert torch.equal(lecb.attention_q8(q, cache, table, lens, starts, window=40), plain)
        for t, was in zip((cache.k, cache.v), kept):
            t.copy_(was)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_results_of_16_bits_are_those_of_32_rounded(dim, dtype):
    """Few rows: errors before the last rounding are those that 32 bits' results may have, so a result lies between the
    roundings of the ends of that interval.  Few tokens, of like weights: what a weight is off by shows."""
    g = gen(dim + 1)
    lengths = [2 + s % 8 for s in range(60)]
    cache = random_cache(g, 60, 2, dim, 32, DEV)
    table, lens = tables(g, lengths, 32, 60, DEV)
    q = queries(g, 60, 8, dim, dtype, size=0.1)
    want, tol = attention(q.float(), cache, table, lens)
    got = lecb.attention_q8(q, cache, table, lens).cpu()
    low, high = ((want + s * tol).to(dtype) for s in (-1, 1))
    assert bool(((low <= got) & (got <= high)).all())
