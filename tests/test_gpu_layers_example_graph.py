"""The example of a quantised layer reads nothing of its graph before a replay has written it."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_graph_results_read_after_a_replay(monkeypatch):
    import quantised_layer

    captured = []
    plain_step = quantised_layer.step

    def step(*args):
        out = plain_step(*args)
        if torch.cuda.is_current_stream_capturing():
            captured.extend(out)
        return out

    class Graph(torch.cuda.graph):
        def __exit__(self, *exc):
            super().__exit__(*exc)
            # what the memory of a capture's results may hold until the first replay
            for t in captured:
                t.copy_(torch.full_like(t, float("nan")))

    monkeypatch.setattr(quantised_layer, "step", step)
    monkeypatch.setattr(torch.cuda, "graph", Graph)
    quantised_layer.main(["--hidden", "256", "--inner", "704", "--tokens", "1", "--prompt", "40"])
    assert len(captured) == 2
