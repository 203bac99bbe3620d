"""Attention over the 8-bit cache against the formula in 64 bits; cache_helpers.attention derives the tolerance."""

import math

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from cache_helpers import BF16, F16, F32, attention, random_cache, starts_of, tables
from test_gpu_layers import DEV, gen, same

pytestmark = pytest.mark.gpu
TYPES = [BF16, F16, F32]


def near(got, want, tol):
    got = got.cpu().double()
    off = (got - want).abs()
    assert bool((off <= tol).all()), (off - tol).max().item()


def queries(g, tokens, heads, dim, dtype, size=2.0):
    return (size * torch.randn(tokens, heads, dim, generator=g)).to(dtype).to(DEV)


def check(g, lengths, news, heads, kv_heads, dim, block, dtype, size=2.0, **more):
    blocks = sum(-(-n // block) for n in lengths) + 2
    cache = random_cache(g, blocks, kv_heads, dim, block, DEV)
    table, lens = tables(g, lengths, block, blocks, DEV)
    starts = None if news is None else starts_of(news, DEV)
    q = queries(g, len(lengths) if news is None else sum(news), heads, dim, dtype, size)
    got = lecb.attention_q8(q, cache, table, lens, starts, **more)
    want, tol = attention(q, cache, table, lens, starts, **more)
    near(got, want, tol)
    again = lecb.attention_q8(q, cache, table, lens, starts, **more)
    assert torch.equal(got, again)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [1, 16, 33, 64, 65, 80, 96, 97, 128, 131, 192, 200, 256])
def test_dimensions(dim, dtype):
    check(gen(dim), [1, 31, 32, 33, 200, 0, 64], None, 6, 2, dim, 32, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 5), (3, 1), (8, 1), (16, 1), (17, 1), (40, 2), (64, 8), (100, 1)])
def test_heads(heads, kv_heads, dtype):
    check(gen(heads), [70, 1, 129], [3, 1, 2], heads, kv_heads, 64, 64, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [32, 64, 128, 256])
@pytest.mark.parametrize("window", [None, 1, 31, 33, 100, 5000])
def test_windows(block, window, dtype):
    check(gen(block), [1, 40, 300, 257, 64], [1, 7, 20, 1, 64], 4, 2, 96, block, dtype, window=window)


@pytest.mark.parametrize("dtype", TYPES)
def test_all_tokens(dtype):
    check(gen(2), [1, 40, 300, 257], [1, 7, 20, 1], 4, 2, 64, 64, dtype, causal=False)


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (80, F16), (256, BF16), (96, F32), (192, F16)])
@pytest.mark.parametrize("lengths,news", [([5000], [1]), ([5000, 3, 700, 0, 1200], [1, 3, 2, 0, 9]), ([3000, 3000], [30, 3])])
def test_long_sequences_are_split(lengths, news, dim, dtype):
    check(gen(dim), lengths, news, 4, 1, dim, 64, dtype)


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, BF16), (128, F16), (128, F32), (80, BF16), (256, BF16), (192, F16), (96, F32)])
@pytest.mark.parametrize("window", [None, 77])
def test_prompts(dim, dtype, window):
    """Many rows: from the first token on, after others, beside sequences of one row."""
    check(gen(dim), [150, 333, 64, 1, 500], [150, 90, 1, 1, 200], 4, 2, dim, 32, dtype, window=window)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_of_one_sequence(dtype):
    check(gen(1), [700], [700], 3, 1, 128, 64, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 72, 128, 160, 256])
def test_prompts_that_see_all_tokens(dim, dtype):
    """Many rows without a causal mask, and with windows of one token and of more than there are."""
    check(gen(dim), [150, 333, 2], [150, 90, 2], 4, 2, dim, 64, dtype, causal=False)
    check(gen(dim), [150, 333, 2], [150, 90, 2], 4, 2, dim, 64, dtype, window=1)
    check(gen(dim), [150, 333, 2], [150, 90, 2], 4, 2, dim, 64, dtype, window=(1 << 31) - 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news", [[3, 1], [120, 60]])
def test_scales_of_either_sign_and_zeros(news, dtype):
    """A code stands for code * scale, whatever the scale's sign; blocks of zeros stand beside blocks of small numbers."""
    g = gen(32)
    cache = random_cache(g, 12, 2, 64, 32, DEV)
    for s in (cache.k_scale, cache.v_scale):
        s.mul_(torch.where(torch.rand(12, 2, generator=g) < 0.4, -1.0, 1.0).to(DEV))
    table, lens = tables(g, [150, 200], 32, 12, DEV)
    starts = starts_of(news, DEV)
    q = queries(g, sum(news), 4, 64, dtype)
    for scale in (None, -0.1):
        want, tol = attention(q, cache, table, lens, starts, scale=scale)
        near(lecb.attention_q8(q, cache, table, lens, starts, scale=scale), want, tol)
    cache.v_scale.copy_(torch.where(torch.rand(12, 2, generator=g) < 0.4, 0.0, 2.0**-50))
    if dtype != F16:
        want, tol = attention(q, cache, table, lens, starts)
        near(lecb.attention_q8(q, cache, table, lens, starts), want, tol)


def test_many_sequences():
    check(gen(3), [(s * 41) % 130 for s in range(200)], None, 2, 1, 64, 32, BF16)


@pytest.mark.parametrize("dtype", TYPES)
def test_scale_and_sharp_rows(dtype):
    """A given scale, negative and 0 too; scores that leave one weight only; scores up to some thousands."""
    for scale in (0.0, -0.2, 1.0):
        check(gen(4), [100, 37], [2, 1], 4, 2, 64, 32, dtype, scale=scale)
    check(gen(5), [300, 37], [2, 1], 4, 2, 64, 32, dtype, size=300.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12, 1e30])
def test_queries_of_every_size(dtype, size):
    """Rows are lifted by a power of two: the scale takes it back."""
    check(gen(6), [100, 37], [2, 1], 4, 2, 64, 32, dtype, size=size, scale=1 / size)


@pytest.mark.parametrize("lengths,news,window", [([9] * 300, None, None), ([300], [300], 9)])
def test_weights_in_two_parts(lengths, news, window):
    """Results of 32 bits: the weights' two parts belong together, in each of some 170000 weights of about a ninth."""
    check(gen(34), lengths, news, 64, 1, 4, 32, F32, size=0.3, window=window)


def test_queries_with_small_and_large_elements():
    """A row's elements down to 2^-29 of its largest are exact, and what meets codes of 0 adds nothing."""
    g = gen(7)
    for dtype in (BF16, F32):
        cache = random_cache(g, 4, 1, 64, 32, DEV)
        rows = torch.zeros(4, 1, 32, 64, dtype=torch.int8)
        from cache_helpers import places
        at = places(32, 64, True)
        rows = cache.k.cpu().view(4, 1, -1)
        rows[:, :, at[:, 7]] = 0                       # the large elements' column
        cache.k.copy_(rows.view_as(cache.k))
        table, lens = tables(g, [100], 32, 4, DEV)
        q = queries(g, 1, 2, 64, dtype)
        q[:, :, 7] = 2.0**24
        want, tol = attention(q, cache, table, lens)
        plain = q.clone()
        plain[:, :, 7] = 0
        _, tol = attention(plain, cache, table, lens)   # held to what the other columns alone allow
        near(lecb.attention_q8(q, cache, table, lens), want, tol)


@pytest.mark.parametrize("dtype", TYPES)
def test_blocks_of_every_scale(dtype):
    """Values' scales 2^40 apart, and zeros: no weight is lost to the others' range."""
    g = gen(8)
    for spread in ((-20, 20), (0, 40), (-40, 0), (-20, 0)):
        cache = random_cache(g, 6, 2, 64, 32, DEV)
        cache.v_scale.copy_(2.0 ** torch.linspace(*spread, 12).view(6, 2))
        cache.v_scale[2] = 0
        cache.k_scale[3] = 0
        table = torch.arange(6, dtype=torch.int32, device=DEV)[None]
        lens = torch.tensor([180], dtype=torch.int32, device=DEV)
        for order in (table, table.flip(1)):
            q = queries(g, 1, 4, 64, dtype)
            if dtype == F16 and spread[1] > 0:
                continue                                # results past the type's range
            want, tol = attention(q, cache, order, lens)
            near(lecb.attention_q8(q, cache, order, lens), want, tol)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_large_scale_behind_small_weights(dtype):
    """The block of far larger values has weights that leave it behind the others: theirs keep their precision."""
    g = gen(10)
    cache = random_cache(g, 2, 1, 64, 32, DEV, spread=0.0)
    cache.v_scale.copy_(torch.tensor([[2.0**-10], [2.0**10]]))
    keys = cache.k.cpu()
    keys[0], keys[1] = 1, -1
    cache.k.copy_(keys)
    cache.k_scale.fill_(1.0)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([64], dtype=torch.int32, device=DEV)
    q = torch.full((1, 1, 64), 0.25, dtype=dtype, device=DEV)     # scores 16 and -16: weights e^32 = 2^46 apart
    want, tol = attention(q, cache, table, lens, scale=1.0)
    near(lecb.attention_q8(q, cache, table, lens, scale=1.0), want, tol)


def test_what_is_masked_never_matters():
    """Codes behind the end, blocks before the window or past the row with scales that are not numbers, entries
    of the table that are not blocks: the same bits as without them."""
    g = gen(12)
    for dtype in TYPES:
        cache = random_cache(g, 12, 2, 80, 32, DEV)
        table, lens = tables(g, [100, 150], 32, 12, DEV, width=6)
        starts = starts_of([5, 2], DEV)
        q = queries(g, 7, 4, 80, dtype)
        want = lecb.attention_q8(q, cache, table, lens, starts, window=20)
        codes, values = cache.k.clone(), cache.v.clone()
        poisoned = table.clone()
        for s, n in enumerate((100, 150)):
            first = (n - (5, 2)[s] - 19) // 32
            for j in range(first):
                for c in (cache.k_scale, cache.v_scale):
                    c[table[s, j].item()] = math.nan if j % 2 else math.inf
                poisoned[s, j] = -1 if j % 2 else 99
            poisoned[s, -(-n // 32):] = 1 << 30
        from cache_helpers import places
        for c, keys in ((cache.k, True), (cache.v, False)):
            last = table[0, 3].item()
            c[last][:, places(32, 80, keys)[100 - 96 :].reshape(-1)] = -128
        assert torch.equal(lecb.attention_q8(q, cache, table, lens, starts, window=20), want)
        assert torch.equal(lecb.attention_q8(q, cache, poisoned, lens, starts, window=20), want)
        # rows of one call that see different blocks: the first row of three ends where the third's block begins
        cache.k.copy_(codes), cache.v.copy_(values)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompts_past_blocks_without_a_number(dtype):
    """Many rows: those from the bad block on are NaN, for keys, values and the table; windows pass it by again."""
    g = gen(15)
    for bad, field in ((math.nan, "k_scale"), (math.nan, "v_scale"), (math.inf, "v_scale"), (None, "table")):
        cache = random_cache(g, 20, 1, 64, 32, DEV)
        table, lens = tables(g, [600], 32, 20, DEV)
        starts = starts_of([600], DEV)
        q = queries(g, 600, 2, 64, dtype)
        want, tol = attention(q, cache, table, lens, starts, window=64)
        if field == "table":
            table[0, 5] = -1
        else:
            getattr(cache, field)[table[0, 5].item()] = bad
        got = lecb.attention_q8(q, cache, table, lens, starts, window=64)
        away = torch.ones(600, dtype=torch.bool)
        away[160 : 192 + 63] = False
        near(got[away.to(DEV)], want[away], tol[away])
        assert bool(got[160 : 192 + 63].isnan().all())


def test_rows_that_see_no_number_are_nan_and_no_others():
    g = gen(14)
    for dtype in TYPES:
        for field in ("k_scale", "v_scale", "table"):
            cache = random_cache(g, 6, 1, 64, 32, DEV)
            table = torch.tensor([[4, 2, 0]], dtype=torch.int32, device=DEV)
            lens = torch.tensor([70], dtype=torch.int32, device=DEV)
            starts = starts_of([70], DEV)
            q = queries(g, 70, 2, 64, dtype)
            want, tol = attention(q, cache, table, lens, starts)
            if field == "table":
                table[0, 1] = 6
            else:
                getattr(cache, field)[2] = math.nan
            got = lecb.attention_q8(q, cache, table, lens, starts)
            near(got[:32], want[:32], tol[:32])
            assert bool(got[32:].isnan().all())
        # a query that is not finite: its row alone
        cache = random_cache(g, 6, 1, 64, 32, DEV)
        q = queries(g, 5, 2, 64, dtype)
        table[0, 1] = 2
        starts = starts_of([5], DEV)
        want, tol = attention(q, cache, table, lens, starts)
        for bad in (math.inf, -math.inf, math.nan):
            q[2, 1, 9] = bad
            got = lecb.attention_q8(q, cache, table, lens, starts)
            assert bool(got[2, 1].isnan().all())
            others = torch.ones(5, 2, dtype=torch.bool)
            others[2, 1] = False
            near(got[others.to(DEV)], want[others], tol[others])


def test_lengths_that_do_not_fit():
    """A sequence longer than its row of the table is NaN, the others are what they are; more rows than tokens: the first see
    nothing; a negative length is none."""
    g = gen(16)
    cache = random_cache(g, 8, 1, 64, 32, DEV)
    table, lens = tables(g, [60, 60, 10, 60], 32, 8, DEV)
    starts = starts_of([4, 4, 14, 4], DEV)
    q = queries(g, 26, 2, 64, BF16)
    want, tol = attention(q, cache, table, lens, starts)
    for bad in (65, (1 << 31) - 1):
        lens[1] = bad
        got = lecb.attention_q8(q, cache, table, lens, starts)
        assert bool(got[4:8].isnan().all()) and bool((got[8:12] == 0).all())
        near(got[:4], want[:4], tol[:4])
        near(got[12:], want[12:], tol[12:])
    for none in (0, -1, -(1 << 31)):
        lens[1] = none
        got = lecb.attention_q8(q, cache, table, lens, starts)
        assert bool((got[4:8] == 0).all())
        near(got[12:], want[12:], tol[12:])


def test_rows_of_no_sequence():
    g = gen(18)
    cache = random_cache(g, 80, 2, 64, 32, DEV)
    for lengths in ([60, 0, 40], [2000, 0, 40]):           # whole, and split
        table, lens = tables(g, lengths, 32, 80, DEV)
        starts = torch.tensor([3, 5, 5, 8], dtype=torch.int32, device=DEV)
        q = queries(g, 40, 4, 64, BF16)
        q[:3], q[8:] = math.nan, math.nan
        clean = torch.where(q.isnan(), 0, q)
        want, tol = attention(clean, cache, table, lens, starts)
        got = lecb.attention_q8(q, cache, table, lens, starts)
        near(got, want, tol)
        assert bool((got[:3] == 0).all()) and bool((got[8:] == 0).all())
        out = torch.full_like(q, 7.0)
        version = out._version
        assert lecb.attention_q8(q, cache, table, lens, starts, out=out) is out and out._version > version
        assert bool((out[:3] == 7).all()) and bool((out[8:] == 7).all()) and torch.equal(out[3:8], got[3:8])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 144, 256])
def test_one_sequence(dim, dtype):
    """One sequence goes by one of the forms: many heads to one, no starts; few rows of its own before many of none."""
    g = gen(36)
    check(g, [300], None, 100, 1, dim, 64, dtype)
    check(g, [3000], None, 100, 1, dim, 64, dtype)
    for length in (300, 3000):
        cache = random_cache(g, 50, 1, dim, 64, DEV)
        table, lens = tables(g, [length], 64, 50, DEV)
        starts = torch.tensor([2, 7], dtype=torch.int32, device=DEV)
        q = queries(g, 90, 2, dim, dtype)
        want, tol = attention(q, cache, table, lens, starts)
        near(lecb.attention_q8(q, cache, table, lens, starts), want, tol)


def test_strides():
    """Queries and results as columns of wider buffers, at odd addresses, heads before tokens."""
    g = gen(20)
    for dim, dtype in ((40, BF16), (128, BF16), (72, F32), (64, F16)):
        cache = random_cache(g, 9, 2, dim, 32, DEV)
        table, lens = tables(g, [70, 100, 33], 32, 9, DEV)
        starts = starts_of([30, 1, 2], DEV)
        base = queries(g, 1, 1, 33 * 9 * dim + 1, dtype).view(-1)
        wide = base[1:].view(33, 9, dim)
        q = wide[:, 1:5]
        want = lecb.attention_q8(q.contiguous(), cache, table, lens, starts)
        assert torch.equal(lecb.attention_q8(q, cache, table, lens, starts), want)
        assert torch.equal(lecb.attention_q8(q.transpose(0, 1).contiguous().transpose(0, 1), cache, table, lens, starts), want)
        rest = wide[:, 5:].clone()
        assert torch.equal(lecb.attention_q8(q, cache, table, lens, starts, out=wide[:, 5:9]), want)
        assert torch.equal(wide[:, 5:], want) and not torch.equal(rest, want)
        out = torch.empty(4, 33, dim, dtype=dtype, device=DEV).transpose(0, 1)
        assert torch.equal(lecb.attention_q8(q, cache, table, lens, starts, out=out), want)
        spaced = torch.cat((table, table), 1)[:, table.shape[1] :]
        assert torch.equal(lecb.attention_q8(q, cache, spaced, lens, starts), want)
        one = wide[:1, 1:2].expand(33, 4, dim)
        assert torch.equal(lecb.attention_q8(one, cache, table, lens, starts), lecb.attention_q8(one.contiguous(), cache, table, lens, starts))


def test_workspace_is_the_callers():
    g = gen(22)
    cache = random_cache(g, 200, 2, 64, 32, DEV)
    table, lens = tables(g, [6000], 32, 200, DEV)
    q = queries(g, 1, 4, 64, BF16)
    want = lecb.attention_q8(q, cache, table, lens)
    c = lecb.lecb_cache_q8(0, 0, 0, 0, 200, 2, 64, 32)
    need = lecb.lecb_attention_q8_workspace_bytes(c, 1, 1, table.shape[1], 4)
    assert need
    for fill in (0, 255):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(lecb.attention_q8(q, cache, table, lens, ws=ws[:need]), want)
        assert bool((ws[need:] == fill).all())
    with pytest.raises(lecb.LecbError):
        lecb.attention_q8(q, cache, table, lens, ws=ws[: need - 1])


def test_graph_follows_lengths():
    """One captured step for growing sequences: replays between eager work, each against the eager result."""
    g = gen(24)
    cache = random_cache(g, 300, 2, 128, 64, DEV)
    table, lens = tables(g, [9000, 64, 9000], 64, 300, DEV, width=200)   # blocks for what it grows to
    q = queries(g, 3, 8, 128, BF16)
    k, v = (queries(g, 3, 2, 128, BF16) for _ in range(2))
    lecb.attention_q8(q, cache, table, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lecb.cache_write_q8(cache, k, v, table, lens)
        out = lecb.attention_q8(q, cache, table, lens)
    for lengths in ([9000, 64, 3000], [9001, 60, 3001], [1, 2, 3], [9003, 1, 0], [40, 64, 8999]):
        lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        q.copy_(queries(g, 3, 8, 128, BF16))
        graph.replay()
        assert torch.equal(out, lecb.attention_q8(q, cache, table, lens))
        want, tol = attention(q, cache, table, lens)
        near(out, want, tol)
        torch.cuda.synchronize()


def test_side_stream_and_two_calls_at_once():
    g = gen(26)
    cache = random_cache(g, 300, 2, 128, 64, DEV)
    table, lens = tables(g, [9000, 7000], 64, 300, DEV)
    q = [queries(g, 2, 8, 128, BF16) for _ in range(2)]
    want = [lecb.attention_q8(x, cache, table, lens) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for x, s in zip(q, streams):
            with torch.cuda.stream(s):
                got.append(lecb.attention_q8(x, cache, table, lens))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_starts_that_do_not_rise():
    """Not stated what they give, but nothing beyond the results is written."""
    g = gen(28)
    cache = random_cache(g, 120, 2, 64, 32, DEV)
    table, lens = tables(g, [2000, 60, 900], 32, 120, DEV)
    q = queries(g, 50, 4, 64, BF16)
    buf = torch.full((70, 4, 64), 7.0, dtype=BF16, device=DEV)
    for starts in ([0, 50, 10, 50], [50, 0, 50, 0], [-5, 1 << 30, -(1 << 31), (1 << 31) - 1], [40, 30, 20, 10], [0, 50, 0, 50]):
        lecb.attention_q8(q, cache, table, lens, torch.tensor(starts, dtype=torch.int32, device=DEV), out=buf[10:60])
        assert bool((buf[:10] == 7).all()) and bool((buf[60:] == 7).all())


def test_backward_is_refused_by_name():
    cache = random_cache(gen(3), 4, 1, 64, 32, DEV)
    table, lens = tables(gen(3), [40], 32, 4, DEV)
    q = queries(gen(3), 1, 2, 64, F32).requires_grad_()
    out = lecb.attention_q8(q, cache, table, lens)
    assert out.requires_grad
    with pytest.raises(RuntimeError, match="attention_q8"):
        out.sum().backward()
    with torch.no_grad():
        assert same(lecb.attention_q8(q, cache, table, lens), out.detach())


def test_past_32_bits():
    """Blocks whose codes lie past 2^32 bytes."""
    blocks, heads, dim, block = 34000, 8, 128, 128
    cache = lecb.new_cache_q8(blocks, heads, dim, block, DEV)
    g = gen(30)
    part = random_cache(g, 4, heads, dim, block, DEV)
    pages = torch.tensor([blocks - 1, 0, 33000, blocks - 2], dtype=torch.int32, device=DEV)
    for a, b in ((cache.k, part.k), (cache.v, part.v), (cache.k_scale, part.k_scale), (cache.v_scale, part.v_scale)):
        a[pages.long()] = b
    lens = torch.tensor([500], dtype=torch.int32, device=DEV)
    for n in (1, 200):
        q = queries(g, n, 16, dim, BF16)
        starts = starts_of([n], DEV)
        few = torch.arange(4, dtype=torch.int32, device=DEV)[None]
        assert torch.equal(lecb.attention_q8(q, cache, pages[None], lens, starts), lecb.attention_q8(q, part, few, lens, starts))
