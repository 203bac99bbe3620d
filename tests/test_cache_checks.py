"""What the 8-bit cache and its attention refuse at the ends of their arguments' ranges, without a GPU."""

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from test_cache_host import INVALID, TOO_LARGE, call_attend, refused, structs, tensors


@pytest.mark.parametrize("scale", [2.36e38, 3.4e38, -2.36e38])
def test_a_scale_that_the_softmax_can_not_take(scale):
    """Finite, but not times log2(e), which is what scores are multiplied by."""
    assert call_attend(*structs(), scale=scale) == INVALID
    a = tensors()
    refused("scale", lambda: lecb.attention_q8(a["q"], a["cache"], a["table"], a["lengths"], a["starts"], scale=scale))
    refused("current GPU", lambda: lecb.attention_q8(a["q"], a["cache"], a["table"], a["lengths"], a["starts"], scale=2.35e38))


def test_a_cache_whose_parts_overlap_is_not_written():
    """Keys' and values' workgroups would race for the same bytes; reading is another matter."""
    ok = lecb.new_cache_q8(10, 4, 80, 64, device="cpu")
    wide = torch.zeros(2 * ok.k.numel() + 160, dtype=torch.int8)
    codes = lambda at: wide[at : at + ok.k.numel()].view(ok.k.shape)
    scales = wide[2 * ok.k.numel() :].view(torch.float32)
    for parts in ((ok.k, ok.k, ok.k_scale, ok.v_scale), (ok.k, ok.v, ok.k_scale, ok.k_scale), (codes(0), codes(64), ok.k_scale, ok.v_scale),
                  (codes(0), codes(ok.k.numel() + 16), scales.view(10, 4), ok.v_scale), (codes(128), ok.v, ok.k_scale, wide[:160].view(torch.float32).view(10, 4))):
        a = tensors(cache=lecb.CacheQ8(*parts, 80, 64))
        refused("parts overlap", lambda: lecb.cache_write_q8(a["cache"], a["k"], a["v"], a["table"], a["lengths"], a["starts"]))
        refused("current GPU", lambda: lecb.cache_read_q8(a["cache"], a["table"], a["lengths"], a["starts"], 7))
    a = tensors(cache=lecb.CacheQ8(codes(0), codes(ok.k.numel()), scales.view(10, 4), ok.v_scale, 80, 64))   # side by side
    refused("current GPU", lambda: lecb.cache_write_q8(a["cache"], a["k"], a["v"], a["table"], a["lengths"], a["starts"]))


def test_numbers_past_32_bits():
    """Not taken for what their low bits say."""
    wrap = 1 << 32
    for bad in ((10 + wrap, 4, 80, 64), (10, 4 + wrap, 80, 64), (10, 4, 80 + wrap, 64), (10, 4, 80, 64 + wrap), (10 + (1 << 64), 4, 80, 64)):
        assert lecb.lecb_cache_q8_bytes(*bad) == 0
        refused("new_cache_q8", lambda: lecb.new_cache_q8(*bad, device="cpu"))
    ok = lecb.new_cache_q8(10, 4, 80, 64, device="cpu")
    refused("CacheQ8", lambda: lecb.CacheQ8(ok.k, ok.v, ok.k_scale, ok.v_scale, 80, 64 + wrap))
    cache, seqs = structs()
    args = dict(seqs=3, tokens=7, width=1000, heads=8)
    assert lecb.lecb_attention_q8_workspace_bytes(cache, **args) > 0
    for name in args:
        assert lecb.lecb_attention_q8_workspace_bytes(cache, **{**args, name: args[name] + wrap}) == 0
    q = torch.zeros(7, 8, 80)
    for heads, window in ((8 + wrap, 0), (8, 5 + wrap), (8, -1)):
        refused("below 2.32", lambda: lecb.lecb_attention_q8(q, 640, 80, heads, cache, seqs, 0.1, True, window, q, 640, 80))


def test_lengths_without_a_dimension():
    a = tensors()
    refused("lengths", lambda: lecb.cache_read_q8(a["cache"], a["table"], torch.zeros((), dtype=torch.int32)))


def test_more_sequences_than_a_search_bears():
    """Each workgroup looks through all sequences: calls that would take minutes of that are refused."""
    many = dict(seqs=1 << 17, tokens=1 << 17)
    assert call_attend(*structs(**many)) == TOO_LARGE
    cache, _ = structs()
    size = lambda seqs, tokens: lecb.lecb_attention_q8_workspace_bytes(cache, seqs, tokens, 1000, 8)
    assert size(1 << 17, 1 << 17) == 0 and size(1 << 17, (1 << 24) - 1) == 0
    assert size(1 << 16, 1 << 16) > 0 and size(1 << 13, 1 << 23) > 0 and size(1 << 10, (1 << 24) - 1) > 0
    wide = lambda type: call_attend(*structs(seqs=1 << 14, tokens=(1 << 24) - 1, dim=256), ot=2048, oh=256, type=type, wsb=0)
    assert wide(0) == TOO_LARGE and wide(1) == lecb.LECB_ERR_WORKSPACE      # F32 goes by 16 rows there
    a = tensors(q=torch.zeros(1, 8, 80).expand(1 << 17, 8, 80), table=torch.zeros(1 << 17, 1, dtype=torch.int32),
                lengths=torch.zeros(1 << 17, dtype=torch.int32))
    refused("below 2.37", lambda: lecb.attention_q8(a["q"], a["cache"], a["table"], a["lengths"]))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_the_workspace_of_a_decoding_step(dim):
    """Calls that never go by the form for many rows have room for the other's sums alone: 2048 parts of 16 rows."""
    cache, _ = structs(heads=8, dim=dim, blocks=1 << 20)
    few = 2048 * 16 * (dim + 4) * 4
    for seqs, tokens, heads in ((64, 64, 32), (1, 1, 64), (1, 16, 32), (16, 64, 32)):
        assert 0 < lecb.lecb_attention_q8_workspace_bytes(cache, seqs, tokens, 4096, heads) <= few
    for seqs, tokens, heads in ((64, 65, 32), (1, 17, 32)):
        assert lecb.lecb_attention_q8_workspace_bytes(cache, seqs, tokens, 4096, heads) > few
