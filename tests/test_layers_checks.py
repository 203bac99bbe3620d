"""Checks of the tensor functions of quantised layers, without a GPU: each refusal
names what is wrong, before the device is looked at and before any launch."""

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb

I8, U8, BF16 = torch.int8, torch.uint8, torch.bfloat16


def w4(n=16, k=128, group=128, scale_dtype=torch.float32):
    return lecb.W4Weights(torch.zeros(1024, dtype=U8), torch.zeros(16 * (128 // group), dtype=scale_dtype), n, k, group)


@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=U8).expand(1 << 20), torch.zeros(2048, dtype=U8)[::2],
                                torch.zeros(64, 64, dtype=U8).t(), torch.zeros(1 << 20, dtype=I8),
                                torch.zeros(1 << 20), torch.zeros(4, dtype=torch.bool)],
                         ids=["expanded", "strided", "transposed", "int8", "float32", "bool"])
def test_workspace_of_another_kind(ws):
    """A workspace is written as that many bytes from its address on, so it has to be just that."""
    x = torch.zeros(9, 128, dtype=BF16)
    with pytest.raises(ValueError, match="ws"):
        lecb.matvec_w4(x, w4(), ws=ws)
    if not ws.is_contiguous():
        with pytest.raises(ValueError, match="ws"):
            lecb.lecb_matvec_w4(x, 128, None, 0, 9, w4().tiles, w4().scales, 128, 16, 128, torch.zeros(9, 16), 16, ws=ws)


@pytest.mark.parametrize("field,value", [("n", 17), ("n", 0), ("n", 1 << 31), ("k", 129), ("k", -1), ("group", 64),
                                         ("group", 16), ("tiles", torch.zeros(1024)),
                                         ("tiles", torch.zeros(1023, dtype=U8)),
                                         ("tiles", torch.zeros(1, dtype=U8).expand(1024)),
                                         ("scales", torch.zeros(1).expand(16)), ("scales", torch.zeros(15)),
                                         ("scales", torch.zeros(16, dtype=torch.float16))], ids=str)
def test_weights_changed_after_they_were_made(field, value):
    """Kernels go by n, k and group: fields that no longer fit one another are refused at each call."""
    bad = w4()
    setattr(bad, field, value)
    with pytest.raises(ValueError, match="weights"):
        lecb.dequantize_w4(bad)
    x = torch.zeros(1, bad.k if 0 < bad.k else 1, dtype=BF16)
    with pytest.raises(ValueError, match="weights"):
        lecb.matvec_w4(x, bad)


def _windows():
    """(x, residual, out_h) in buffers of their own or in one."""
    buf, other = torch.zeros(4096, dtype=BF16), torch.zeros(4096, dtype=BF16)

    def at(b, start, stride, rows=8, cols=32):
        return b.as_strided((rows, cols), (stride, 1), start)

    for start, stride in ((32, 32), (1, 32), (0, 64), (7 * 32, 32), (31, 64), (32, 64), (33, 64), (7 * 64 + 31, 64), (64, 40)):
        yield at(buf, 0, 32 if stride == 32 else 64), at(other, 0, 32), at(buf, start, stride)
    x = at(buf, 1024, 64)
    for start, stride in ((1024, 64), (1024 + 32, 64), (1024 - 32, 64), (1024 + 96, 64), (1024 + 65, 64), (1024 - 33, 64),
                          (1024 - 7 * 64 - 31, 64), (1024 - 7 * 64 - 32, 64), (1024 - 8 * 64, 64), (1024 + 8 * 64, 64),
                          (0, 128), (1024 + 32, 128), (1024 - 32, 128), (1024 + 33, 128), (1024 + 7 * 64 + 32, 32),
                          (1024 + 7 * 64 + 31, 32), (800, 96), (832, 96)):
        yield x, at(other, 0, 32), at(buf, start, stride)
        yield at(other, 0, 32), x, at(buf, start, stride)


@pytest.mark.parametrize("x,residual,out", list(_windows()), ids=lambda t: f"{t.storage_offset()}/{t.stride(0)}")
def test_result_over_other_rows(x, residual, out):
    """h may stand where x or the residual stand, row for row; over other rows of theirs it would
    be written while they are read.  Rows beside them in one buffer are not over them."""

    def places(t):
        return {t.untyped_storage().data_ptr() + 2 * (t.storage_offset() + r * t.stride(0) + c)
                for r in range(8) for c in range(32)}

    def same(t):
        return t.data_ptr() == out.data_ptr() and t.stride() == out.stride()

    meets = any(not same(t) and bool(places(t) & places(out)) for t in (x, residual))
    with pytest.raises(ValueError, match="out_h overlaps" if meets else "current GPU"):
        lecb.rmsnorm_q8(x, torch.ones(32, dtype=BF16), residual=residual, out_h=out)


def test_result_over_the_weight_or_the_scale():
    buf = torch.zeros(1024, dtype=BF16)
    x, r, out = torch.zeros(8, 32, dtype=BF16), torch.zeros(8, 32, dtype=BF16), buf[64:320].view(8, 32)
    for start in (33, 64, 200, 319):
        with pytest.raises(ValueError, match="out_h overlaps"):
            lecb.rmsnorm_q8(x, buf[start : start + 32], residual=r, out_h=out)
    for start in (32, 320):
        with pytest.raises(ValueError, match="current GPU"):
            lecb.rmsnorm_q8(x, buf[start : start + 32], residual=r, out_h=out)
    with pytest.raises(ValueError, match="out_h overlaps"):
        lecb.rmsnorm_q8(x, torch.ones(32), residual=r, out_h=out, scale=buf[100:102].view(torch.float32))
    wide = buf[:512].view(8, 64)[:, :32]     # rows 64 apart, the weight between two of them
    with pytest.raises(ValueError, match="current GPU"):
        lecb.rmsnorm_q8(x, buf[96:128], residual=r, out_h=wide)
    with pytest.raises(ValueError, match="out_h overlaps"):
        lecb.rmsnorm_q8(x, buf[95:127], residual=r, out_h=wide)


def test_tangents_are_refused():
    """Forward-mode derivatives would be lost without a word."""
    from torch.autograd import forward_ad as fw

    def dual(t):
        return fw.make_dual(t, torch.ones_like(t))

    x, weight, r = torch.zeros(3, 128, dtype=BF16), torch.ones(128, dtype=BF16), torch.zeros(3, 128, dtype=BF16)
    q, one = torch.zeros(3, 128, dtype=I8), torch.ones(1)
    with fw.dual_level():
        for call in (lambda: lecb.matvec_w4(dual(x), w4()), lambda: lecb.matvec_w4(q, w4(), x_scale=dual(one)),
                     lambda: lecb.rmsnorm_q8(dual(x), weight), lambda: lecb.rmsnorm_q8(x, dual(weight)),
                     lambda: lecb.rmsnorm_q8(x, weight, residual=dual(r)), lambda: lecb.dequantize_q8(q, dual(one)),
                     lambda: lecb.quantize_w4(dual(x)),
                     lambda: lecb.dequantize_w4(lecb.W4Weights(w4().tiles, dual(w4().scales), 16, 128))):
            with pytest.raises(ValueError, match="forward-mode"):
                call()


def test_result_in_place_while_gradients_are_recorded():
    """As torch's own out= arguments: with no derivative of what is written there."""
    x, weight, r = torch.zeros(3, 128, dtype=BF16), torch.ones(128, dtype=BF16), torch.zeros(3, 128, dtype=BF16)
    for which in range(3):
        args = [t.clone().requires_grad_(i == which) for i, t in enumerate((x, weight, r))]
        for out in (args[0], torch.empty_like(x)):
            with pytest.raises(ValueError, match="gradients"):
                lecb.rmsnorm_q8(args[0], args[1], residual=args[2], out_h=out)
            with torch.no_grad(), pytest.raises(ValueError, match="current GPU"):
                lecb.rmsnorm_q8(args[0], args[1], residual=args[2], out_h=out)


def test_workspace_of_many_tokens_and_rows():
    """Tokens and rows past what one pass of launches takes share its workspace."""
    ask = lecb.lecb_matvec_w4_workspace_bytes
    most = 65535 * 64
    assert ask(most, 64, 128) == most * 128 * 2
    for m in (most + 1, 2 * most, (1 << 31) - 1):
        assert ask(m, 64, 128) == ask(most, 64, 128)
    assert ask(100, (1 << 31) - 1, 128) == ask(100, 1 << 26, 128) >= 128 * 128 * 2
    # a workspace for the most tokens serves fewer
    for n, k in ((16, 28672), (1000, 8192), (8192, 8192), (64, 128)):
        sizes = [ask(m, n, k) for m in (1, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 512, 10000)]
        assert sizes == sorted(sizes)
