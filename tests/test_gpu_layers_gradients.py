"""The operators of quantised layers have no derivatives: a backward pass through
them says so, and nothing else changes."""

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from test_gpu_layers import BF16, DEV, F32, I8, gen

pytestmark = pytest.mark.gpu


def _inputs():
    g = gen(1)
    w = torch.randn(48, 256, generator=g).to(BF16).to(DEV)
    x, r = (torch.randn(5, 256, generator=g).to(BF16).to(DEV) for _ in range(2))
    return w, x, r, torch.ones(256, dtype=BF16, device=DEV)


def _calls(w, x, r, weight):
    """(name, inputs, call on them, which of its results are numbers made from them)"""
    w4 = lecb.quantize_w4(w)
    q, scale, _ = lecb.rmsnorm_q8(x, weight, residual=r)
    yield "matvec_w4", (x,), lambda x: lecb.matvec_w4(x, w4), (0,)
    yield "matvec_w4", (scale,), lambda s: lecb.matvec_w4(q, w4, x_scale=s), (0,)
    yield "matvec_w4", (w4.scales,), lambda s: lecb.matvec_w4(x, lecb.W4Weights(w4.tiles, s, 48, 256)), (0,)
    yield "rmsnorm_q8", (x, weight, r), lambda x, v, r: lecb.rmsnorm_q8(x, v, residual=r), (1, 2)
    yield "rmsnorm_q8", (x, weight), lambda x, v: lecb.rmsnorm_q8(x, v), (1,)
    yield "dequantize_q8", (scale,), lambda s: lecb.dequantize_q8(q, s), (0,)
    yield "dequantize_w4", (w4.scales,), lambda s: lecb.dequantize_w4(lecb.W4Weights(w4.tiles, s, 48, 256)), (0,)


def test_backward_names_what_has_no_derivative():
    for name, inputs, call, numbers in _calls(*_inputs()):
        plain = call(*inputs)
        plain = plain if isinstance(plain, tuple) else (plain,)
        assert not any(p.requires_grad for p in plain)
        for which in range(len(inputs)):
            leaves = [t.detach().clone().requires_grad_(i == which) for i, t in enumerate(inputs)]
            got = call(*leaves)
            got = got if isinstance(got, tuple) else (got,)
            assert all(torch.equal(a, b) for a, b in zip(got, plain))
            for i in numbers:
                assert got[i].requires_grad and not got[i].is_leaf
                with pytest.raises(RuntimeError, match=name):
                    got[i].float().sum().backward()
            with torch.no_grad():
                got = call(*leaves)
                got = got if isinstance(got, tuple) else (got,)
            assert not any(t.requires_grad and t is not leaves[0] for t in got)
            assert all(leaf.grad is None for leaf in leaves)


def test_results_that_are_inputs_keep_their_gradients():
    """Without a residual h is x: its gradient is x's.  A fixed scale is returned as it was given."""
    _, x, _, weight = _inputs()
    x = x.requires_grad_()
    fixed = torch.tensor([0.05], device=DEV, requires_grad=True)
    q, scale, h = lecb.rmsnorm_q8(x, weight, scale=fixed)
    assert h is x and scale is fixed and q.dtype == I8
    (h * 2).sum().backward()
    assert bool((x.grad == 2).all())


def test_weights_are_constants():
    """Rounded weights carry no history: they can be kept, copied and used in serving as they are."""
    w, x, _, _ = _inputs()
    w4 = lecb.quantize_w4(torch.nn.Parameter(w))
    assert not w4.scales.requires_grad and not lecb.matvec_w4(x, w4, out_dtype=F32).requires_grad


def test_h_in_place_is_seen_by_autograd():
    """What a recorded product has kept is changed by a later call: its backward pass must not go on with it."""
    _, x, r, weight = _inputs()
    for kept in (x, r, torch.empty_like(x)):
        kept.zero_()
        before = kept._version
        leaf = torch.ones_like(x).requires_grad_()
        z = (leaf * kept).float().sum()
        lecb.rmsnorm_q8(x, weight, residual=r, out_h=kept)
        assert kept._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            z.backward()
    with torch.inference_mode():
        out = torch.empty_like(x)
        assert lecb.rmsnorm_q8(x, weight, residual=r, out_h=out)[2] is out
    assert lecb.rmsnorm_q8(x, weight, residual=r, out_h=out)[2] is out
