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
