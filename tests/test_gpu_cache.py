"""The 8-bit cache on the GPU: codes and scales are defined exactly and compared so, values to the last bit."""

import math

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from cache_helpers import BF16, F16, F32, I8, host, random_cache, rows_of, starts_of, tables, values, write
from test_gpu_layers import DEV, gen, same

pytestmark = pytest.mark.gpu


def check_write(cache, k, v, table, lengths, starts=None):
    """A write against the formula; blocks that no row is in keep their bytes, codes behind a sequence's end may not."""
    before = host(cache)
    kc, vc, ks, vs = write(cache, k, v, table, lengths, starts)
    lecb.cache_write_q8(cache, k, v, table, lengths, starts)
    after = host(cache)
    at = list(range(len(lengths) + 1)) if starts is None else starts.cpu().tolist()
    assert same(after.k_scale, ks) and same(after.v_scale, vs)
    untouched = torch.ones(after.k.shape[0], dtype=torch.bool)
    held = torch.zeros(after.k.shape[0], dtype=torch.int64)
    for s, n in enumerate(lengths.tolist()):
        for j in range(max(0, n - (at[s + 1] - at[s])) // cache.block, -(-n // cache.block) if at[s + 1] > at[s] else 0):
            page = table[s, j].item() if j < table.shape[1] else -1
            if 0 <= page < len(held) and n <= table.shape[1] * cache.block:
                untouched[page] = False
                held[page] = min(cache.block, n - j * cache.block)
    for got, want, was, keys in ((after.k, kc, before.k, True), (after.v, vc, before.v, False)):
        assert torch.equal(got[untouched], was[untouched])
        rows = rows_of(got, cache.block, cache.dim, keys)
        seen = (torch.arange(cache.block) < held[:, None])[:, None, :, None]
        assert torch.equal(torch.where(seen, rows, 0), torch.where(seen, want, 0))
    return after


def randn(g, *size, dtype=BF16):
    return (torch.randn(*size, generator=g) * torch.exp(0.4 * torch.randn(*size[:-1], 1, generator=g))).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("dim,block,heads", [(1, 32, 1), (8, 64, 2), (63, 32, 3), (64, 64, 1), (80, 32, 2), (97, 128, 1), (128, 64, 3),
                                             (131, 256, 1), (192, 64, 2), (256, 256, 1), (250, 128, 2)])
def test_write_and_read(dtype, dim, block, heads):
    g = gen(dim)
    lengths = [1, block, block + 1, 3 * block - 1, 40, 2 * block, 5]
    news = [1, block, 1, 2 * block + 3, 0, block + 1, 5]
    cache = random_cache(g, 20, heads, dim, block, DEV)
    table, lens = tables(g, lengths, block, 20, DEV)
    starts = starts_of(news, DEV)
    k, v = (randn(g, sum(news), heads, dim, dtype=dtype) for _ in range(2))
    check_write(cache, k, v, table, lens, starts)
    # and back, all of the tokens in every type
    ks, vs = values(cache)
    everything = starts_of(lengths, DEV)
    for out in (F32, BF16, F16):
        back = lecb.cache_read_q8(cache, table, lens, everything, sum(lengths), out)
        for got, want in zip(back, (ks, vs)):
            rows = [want[table[s, p // block].item(), :, p % block] for s, n in enumerate(lengths) for p in range(n)]
            assert same(got, torch.stack(rows).float().to(out))   # codes by 24 bits: one rounding to 32 bits, one to the type


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_one_token_at_a_time(dtype):
    """A sequence grows token by token over blocks that are begun, filled, and grow their scales."""
    g = gen(5)
    cache = random_cache(g, 6, 2, 72, 32, DEV)
    table = torch.tensor([[3, 1, 4], [0, 5, 2]], dtype=torch.int32, device=DEV)
    for n in range(1, 80):
        k, v = (randn(g, 2, 2, 72, dtype=dtype) * (1 + n % 7) for _ in range(2))
        check_write(cache, k, v, table, torch.tensor([n, max(1, n - 30)], dtype=torch.int32, device=DEV))


def test_a_block_that_grows_keeps_its_tokens_near():
    """Each regrowth takes a quarter at least, so repeated roundings stay within half a step times 1 + 4/5 + (4/5)^2 .. = 2.5."""
    cache = lecb.new_cache_q8(1, 1, 64, 64, DEV)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    g = gen(9)
    x = torch.randn(64, 1, 64, generator=g) * 1.07 ** torch.arange(64)[:, None, None]
    for n in range(64):
        lecb.cache_write_q8(cache, x[n : n + 1].to(DEV), x[n : n + 1].to(DEV), table, torch.tensor([n + 1], dtype=torch.int32, device=DEV))
    for got, scale in zip(values(cache), (cache.k_scale, cache.v_scale)):
        assert (got[0, 0] - x[:, 0]).abs().max() <= 2.5 * scale.item() * (1 + 2**-20)


def test_ties_ends_and_what_is_not_finite():
    t = torch.tensor
    table, one = torch.zeros(1, 1, dtype=torch.int32, device=DEV), t([4], dtype=torch.int32, device=DEV)
    starts = t([0, 4], dtype=torch.int32, device=DEV)

    def rows(*values):
        x = torch.zeros(4, 1, 64, dtype=F32)
        x.view(-1)[: len(values)] = t(values)
        return x.to(DEV)

    top = torch.finfo(F32).max
    small = 2.0**-149
    cases = [rows(127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 3.4999998, 125.5, 126.5), rows(*[top, -top, top / 254, top / 2]),
             rows(127 * small, small, 63 * small, -5 * small), rows(3 * small, small), rows(100 * small, small, -50 * small), rows(),
             rows(2.0**-70, 2.0**-77, 1.5 * 2.0**-77), rows(1.0, math.inf, 2.0), rows(1.0, -math.inf), rows(1.0, math.nan, 3.0)]
    for x in cases:
        for y in (x, -x):
            check_write(random_cache(gen(1), 1, 1, 64, 32, DEV), x, y, table, one, starts)
    # beside older tokens: NaN stays, whether the scale or the token brings it
    for scale in (math.nan, 0.0, 2.0**-149, 1e30):
        for x in cases:
            cache = random_cache(gen(1), 1, 1, 64, 32, DEV)
            cache.k_scale.fill_(scale)
            check_write(cache, x, x, table, one + 9, starts)
            check_write(cache, x, x, table, one + 13, starts)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(dtype):
    """Keys and values as columns of one product's result, at odd addresses, heads before tokens."""
    g = gen(11)
    lengths, news = [70, 33, 5], [40, 33, 1]
    starts = starts_of(news, DEV)
    for dim in (40, 128):
        base = randn(g, 74 * (2 + 3 + 3) * dim + 1, 1, dtype=dtype).view(-1)
        wide = base[1:].view(74, 8, dim)
        for k, v in ((wide[:, 2:5], wide[:, 5:]), (wide[:, 2:5].transpose(0, 1).contiguous().transpose(0, 1), wide[:, 5:8]),
                     (wide[:1, 2:5].expand(74, 3, dim), wide[:, :1].expand(74, 3, dim))):
            cache = random_cache(g, 8, 3, dim, 32, DEV)
            table, lens = tables(g, lengths, 32, 8, DEV, width=5)
            check_write(cache, k, v, table, lens, starts)
            check_write(cache, k, v, torch.cat((table, table), 1)[:, 5:], lens, starts)


def test_blocks_that_are_not_there():
    """Entries out of range and lengths past the table: nothing is written, rows read as NaN."""
    g = gen(13)
    cache = random_cache(g, 8, 2, 64, 32, DEV)
    table = torch.tensor([[0, -1, 2], [3, 8, 4], [5, 6, 7], [2147483647, -2147483648, 1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([96, 96, 97, 96], dtype=torch.int32, device=DEV)
    starts = starts_of([96, 70, 97, 60], DEV)
    k, v = (randn(g, 323, 2, 64) for _ in range(2))
    check_write(cache, k, v, table, lens, starts)
    ks, vs = values(cache)
    for got, want in zip(lecb.cache_read_q8(cache, table, lens, starts, 323, F32), (ks, vs)):
        row = 0
        for s, n in enumerate((96, 70, 97, 60)):
            for i in range(n):
                pos = lens[s].item() - n + i
                page = table[s, pos // 32].item() if lens[s] <= 96 else -1
                w = want[page, :, pos % 32].float() if 0 <= page < 8 else torch.full((2, 64), math.nan)
                assert same(got[row], w)
                row += 1


def test_rows_of_no_sequence_and_without_tokens():
    g = gen(17)
    cache = random_cache(g, 8, 2, 64, 32, DEV)
    table, lens = tables(g, [40, 0, 10, 3], 32, 8, DEV)
    starts = torch.tensor([3, 8, 10, 30, 33], dtype=torch.int32, device=DEV)   # 3 rows before, 7 behind; 20 rows for 10 tokens
    got = lecb.cache_read_q8(cache, table, lens, starts, 40, BF16)
    for x, want in zip(got, values(cache)):
        full = torch.zeros(40, 2, 64, dtype=torch.float64)
        for i in range(5):
            full[3 + i] = want[table[0, (35 + i) // 32].item(), :, (35 + i) % 32]
        full[20:30] = want[table[2, 0].item(), :, :10].transpose(0, 1)
        full[30:33] = want[table[3, 0].item(), :, :3].transpose(0, 1)
        assert same(x, full.float().to(BF16))
    # explicit buffers: rows of no sequence stay as they are where that is asked for
    k, v = (torch.full((40, 2, 64), 7.0, dtype=BF16, device=DEV) for _ in range(2))
    c = lecb.lecb_cache_q8(cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), 8, 2, 64, 32)
    s = lecb.lecb_cache_seqs(table.data_ptr(), lens.data_ptr(), starts.data_ptr(), table.stride(0), table.shape[1], 4, 40)
    lecb.lecb_cache_read_q8(c, s, k, v, fill=False)
    for x, y in ((k, got[0]), (v, got[1])):
        assert bool((x[:3] == 7).all()) and bool((x[33:] == 7).all()) and torch.equal(x[3:33], y[3:33])
    # writing them changes nothing but the sequences' blocks; rows before a first token are left out
    x = randn(g, 40, 2, 64)
    x[:3], x[33:], x[10:20] = math.nan, math.nan, math.nan
    check_write(cache, x, x, table, lens, starts)
    assert torch.isfinite(cache.k_scale).all()


def test_many_sequences_and_none():
    g = gen(19)
    lengths = [1 + (s * 37) % 90 for s in range(300)]
    cache = random_cache(g, 900, 1, 24, 32, DEV)
    table, lens = tables(g, lengths, 32, 900, DEV)
    k, v = (randn(g, 300, 1, 24) for _ in range(2))
    check_write(cache, k, v, table, lens)
    news = [0 if s % 3 else 1 + s % 5 for s in range(300)]
    news = [min(n, x) for n, x in zip(news, lengths)]
    k, v = (randn(g, sum(news), 1, 24) for _ in range(2))
    check_write(cache, k, v, table, lens, starts_of(news, DEV))
    before = host(cache)
    lecb.cache_write_q8(cache, k[:0], v[:0], table, lens, starts_of([0] * 300, DEV))
    assert torch.equal(before.k, host(cache).k)
    assert [t.shape for t in lecb.cache_read_q8(cache, table, lens, starts_of([0] * 300, DEV), 0)] == [(0, 1, 24)] * 2


def test_starts_that_do_not_rise():
    """What they give is not stated; the blocks of sequences that are in order get what they should."""
    g = gen(23)
    cache = random_cache(g, 12, 1, 64, 32, DEV)
    table, lens = tables(g, [60, 60, 60], 32, 12, DEV)
    x = randn(g, 50, 1, 64)
    spare = torch.ones(12, dtype=torch.bool)
    spare[table.long().cpu().view(-1)] = False
    before = host(cache)
    for starts in ([0, 50, 10, 50], [50, 0, 50, 0], [-5, 1 << 30, -(1 << 31), (1 << 31) - 1], [40, 30, 20, 10]):
        at = torch.tensor(starts, dtype=torch.int32, device=DEV)
        lecb.cache_write_q8(cache, x, x, table, lens, at)
        lecb.cache_read_q8(cache, table, lens, at, 50)
    after = host(cache)
    assert torch.equal(after.k[spare], before.k[spare]) and torch.equal(after.v_scale[spare], before.v_scale[spare])


def test_graph_stream_and_version():
    g = gen(29)
    cache, eager = (random_cache(gen(29), 9, 2, 96, 64, DEV) for _ in range(2))
    table, lens = tables(g, [100, 1, 129], 64, 9, DEV, width=3)
    k, v = (randn(g, 3, 2, 96) for _ in range(2))
    version = cache.k._version, cache.v_scale._version
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lecb.cache_write_q8(cache, k, v, table, lens)
    torch.cuda.current_stream().wait_stream(side)
    assert cache.k._version > version[0] and cache.v_scale._version > version[1]
    lecb.cache_write_q8(eager, k, v, table, lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lecb.cache_write_q8(cache, k, v, table, lens)
        got = lecb.cache_read_q8(cache, table, lens, dtype=F32)
    for step in range(4):
        k.copy_(randn(g, 3, 2, 96))
        v.copy_(randn(g, 3, 2, 96))
        if step:
            lens.add_(torch.tensor([1, 1, 1], dtype=torch.int32, device=DEV))
        table[1, 0] = table[1, 0]
        graph.replay()
        check_write(eager, k, v, table, lens)
        for a, b in zip(got, lecb.cache_read_q8(eager, table, lens, dtype=F32)):
            assert torch.equal(a, b)
        assert torch.equal(cache.k, eager.k) and torch.equal(cache.v_scale, eager.v_scale)


def test_backward_is_refused_by_name():
    cache = random_cache(gen(3), 4, 1, 64, 32, DEV)
    table, lens = tables(gen(3), [40], 32, 4, DEV)
    x = torch.randn(1, 1, 64, device=DEV, requires_grad=True)
    lecb.cache_write_q8(cache, x, x, table, lens)      # codes are constants
    assert not cache.k_scale.requires_grad
    scales = cache.k_scale.clone().requires_grad_()
    k, v = lecb.cache_read_q8(lecb.CacheQ8(cache.k, cache.v, scales, cache.v_scale, 64, 32), table, lens)
    with pytest.raises(RuntimeError, match="cache_read_q8"):
        k.float().sum().backward()


def test_codec_takes_a_cache():
    """A cache's codes are bytes to the codec: through it and back they are the same."""
    g = gen(31)
    cache = random_cache(g, 16, 4, 128, 64, DEV)
    flat = cache.k.view(torch.uint8).view(-1)
    hist = torch.zeros(256, dtype=torch.int64, device=DEV)
    lecb.lecb_histogram(flat, hist)
    book = lecb.DeviceCodebook.upload(lecb.lecb_build_codebook(hist.cpu().numpy(), 16, 1), DEV)
    stream, res = lecb.encode(flat, book, 4096)
    size = int(lecb.results_to_numpy(res)[0]["bytes"])
    assert size < flat.numel()
    back, _ = lecb.decode(stream, size, book, 4096, flat.numel())
    assert torch.equal(back[: flat.numel()], flat)


def test_past_32_bits():
    """Blocks whose codes lie past 2^32 bytes, rows past 2^31 elements of their tensor."""
    blocks, heads, dim, block = 34000, 8, 128, 128
    cache = lecb.new_cache_q8(blocks, heads, dim, block, DEV)      # 4.46 GB each
    g = gen(37)
    table = torch.tensor([[blocks - 1, 0], [blocks - 2, 1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([200, 130], dtype=torch.int32, device=DEV)
    starts = starts_of([200, 130], DEV)
    wide = torch.empty(330, 1 << 23, dtype=BF16, device=DEV)       # rows 2^23 elements apart: the last ones past 2^31
    k, v = (x.view(330, heads, dim) for x in (wide[:, : heads * dim], wide[:, -heads * dim :]))
    k.copy_(randn(g, 330, heads, dim))
    v.copy_(randn(g, 330, heads, dim))
    lecb.cache_write_q8(cache, k, v, table, lens, starts)
    pages = table.view(-1).long()
    part = lecb.new_cache_q8(4, heads, dim, block, DEV)
    few = torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2)
    lecb.cache_write_q8(part, k.contiguous(), v.contiguous(), few, lens, starts)
    for a, b in ((cache.k, part.k), (cache.v, part.v), (cache.k_scale, part.k_scale), (cache.v_scale, part.v_scale)):
        assert torch.equal(a[pages], b)
    for a, b in zip(lecb.cache_read_q8(cache, table, lens, starts, 330), lecb.cache_read_q8(part, few, lens, starts, 330)):
        assert torch.equal(a, b)
    check_write(part, k.contiguous(), v.contiguous(), few, lens, starts)
