"""The example of attention over the 8-bit cache runs: prompts, captured steps, blocks through the codec."""

import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("argv", [[], ["--hidden", "1280", "--heads", "16", "--kv-heads", "2", "--prompt", "333", "--steps", "40"],
                                  ["--hidden", "512", "--heads", "4", "--kv-heads", "4", "--prompt", "64", "--steps", "3"]], ids=str)
def test_runs(argv):
    import cached_attention

    got = cached_attention.main(argv)
    # a step is a block's largest number's 127th, some 4.2 / 127 of a usual one's size, an error of that / sqrt(12) = 0.01
    # for the values, as much at most through the keys' scores, half as much again where scales have grown: doubled
    assert max(got["errors"]) < 0.05
    assert got["kept"] < got["size"]
