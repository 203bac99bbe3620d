"""Attention over the 8-bit cache at the ends of its scales' range, for many rows as for few; cache_helpers.attention derives
the tolerance."""

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from cache_helpers import BF16, F16, F32, attention, random_cache, starts_of, tables
from test_gpu_attention import near, queries
from test_gpu_layers import DEV, gen

pytestmark = pytest.mark.gpu
TYPES = [BF16, F16, F32]


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
