"""What the 8-bit cache and its attention refuse at the ends of their arguments' ranges, without a GPU."""

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from test_cache_host import INVALID, call_attend, refused, structs, tensors


@pytest.mark.parametrize("scale", [2.36e38, 3.4e38, -2.36e38])
def test_a_scale_that_the_softmax_can_not_take(scale):
    """Finite, but not times log2(e), which is what scores are multiplied by."""
    assert call_attend(*structs(), scale=scale) == INVALID
    a = tensors()
    refused("scale", lambda: lecb.attention_q8(a["q"], a["cache"], a["table"], a["lengths"], a["starts"], scale=scale))
    refused("current GPU", lambda: lecb.attention_q8(a["q"], a["cache"], a["table"], a["lengths"], a["starts"], scale=2.35e38))
