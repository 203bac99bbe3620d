"""The example of a quantised layer, run at small sizes."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("hidden,inner,tokens,prompt", [(256, 704, 1, 40), (1000, 1111, 3, 300)])
def test_quantised_layer(hidden, inner, tokens, prompt, capsys):
    import quantised_layer

    out = quantised_layer.main(["--hidden", str(hidden), "--inner", str(inner), "--tokens", str(tokens), "--prompt", str(prompt)])
    # weights rounded to a step of max / 7 of 128 normal ones (about 0.39 of their size): an error of 0.39 /
    # sqrt(12) = 0.11 of their norm a matrix, two matrices and a curve of slope about 1 between: 0.16, doubled
    assert all(0.02 < e < 0.32 for e in out["errors"]), out
    # codes of normal weights: about 3.1 bits of 4, scales besides
    assert out["kept"] < out["four"] < out["plain"]
    assert "us a replay" in capsys.readouterr().out
