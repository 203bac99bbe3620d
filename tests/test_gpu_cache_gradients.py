"""Writing the 8-bit cache from tensors that gradients are recorded for."""

import warnings

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from cache_helpers import host, random_cache, tables
from test_gpu_layers import DEV, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["k", "v"])
def test_a_write_that_ends_a_gradient_says_so(which):
    cache = random_cache(gen(3), 4, 1, 64, 32, DEV)
    table, lens = tables(gen(3), [40], 32, 4, DEV)
    rows = {n: torch.randn(1, 1, 64, device=DEV) for n in "kv"}
    rows[which].requires_grad_()
    with pytest.warns(UserWarning, match="cache_write_q8: no gradient"):
        lecb.cache_write_q8(cache, rows["k"], rows["v"], table, lens)
    written = host(cache)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with torch.no_grad():
            lecb.cache_write_q8(cache, rows["k"], rows["v"], table, lens)
        lecb.cache_write_q8(cache, rows["k"].detach(), rows["v"].detach(), table, lens)
        # where warnings are errors nothing is written
        with pytest.raises(UserWarning, match="no gradient"):
            lecb.cache_write_q8(cache, 2 * rows["k"], 2 * rows["v"], table, lens)
    assert torch.equal(host(cache).k, written.k) and torch.equal(host(cache).v, written.v)
    assert torch.equal(host(cache).k_scale, written.k_scale)
