"""Operators of quantised layers, without a GPU: sizes, and every refusal of the
C ABI and of the tensor functions (all of them come before any launch)."""

import ctypes
import math

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb

P = 1 << 20          # an aligned address that is never touched: every call below is refused
INVALID, WORKSPACE, TOO_LARGE = lecb.LECB_ERR_INVALID_ARG, lecb.LECB_ERR_WORKSPACE, lecb.LECB_ERR_TOO_LARGE
F32, BF16, F16, I8 = 0, 1, 2, 3


def test_sizes():
    for n in (1, 15, 16, 17, 1003, 8192):
        for k in (1, 127, 128, 129, 4096):
            cells = -(-n // 16) * -(-k // 128)
            assert lecb.lecb_w4_tile_bytes(n, k) == cells * 1024
            for g in (32, 64, 128):
                assert lecb.lecb_w4_scale_count(n, k, g) == cells * (128 // g) * 16
            assert lecb.lecb_w4_scale_count(n, k, 48) == 0
    for n, k in ((0, 5), (5, 0), (1 << 31, 5), (5, 1 << 31)):
        assert lecb.lecb_w4_tile_bytes(n, k) == 0
        assert lecb.lecb_w4_scale_count(n, k, 128) == 0
        assert lecb.lecb_matvec_w4_workspace_bytes(1, n, k) == 0
    assert lecb.lecb_matvec_w4_workspace_bytes(1 << 31, 64, 64) == 0


def _call(name, good, **change):
    args = dict(good)
    assert set(change) <= set(args), change
    args.update(change)
    return getattr(lecb.load(), name)(*args.values())


QUANT = dict(w=P, type=BF16, stride=256, n=16, k=256, group=128, tiles=P, scales=P, scale_type=BF16, stream=0)
BAD_QUANT = [dict(w=0), dict(w=P + 1), dict(type=I8), dict(type=9), dict(type=-1), dict(stride=255), dict(n=0), dict(k=0),
             dict(n=1 << 31), dict(group=0), dict(group=16), dict(group=256), dict(tiles=0), dict(tiles=P + 8),
             dict(scales=0), dict(scales=P + 4), dict(scale_type=F16), dict(scale_type=I8)]


@pytest.mark.parametrize("change", BAD_QUANT, ids=str)
def test_quantize_refusals(change):
    assert _call("lecb_quantize_w4", QUANT, **change) == INVALID


DEQUANT = dict(tiles=P, scales=P, scale_type=BF16, group=128, n=16, k=256, out=P, type=F16, stride=256, stream=0)


@pytest.mark.parametrize("change", [dict(tiles=0), dict(tiles=P + 8), dict(scales=0), dict(scales=P + 2),
                                    dict(scale_type=F16), dict(group=48), dict(n=0), dict(k=1 << 31), dict(out=0),
                                    dict(out=P + 1), dict(type=I8), dict(stride=255)], ids=str)
def test_dequantize_refusals(change):
    assert _call("lecb_dequantize_w4", DEQUANT, **change) == INVALID


@pytest.mark.parametrize("name", ["lecb_tile_w4", "lecb_untile_w4"])
def test_tile_refusals(name):
    lib = getattr(lecb.load(), name)
    tiles_first = name == "lecb_untile_w4"
    for src, n, k, dst in ((0, 4, 4, P), (P, 0, 4, P), (P, 4, 0, P), (P, 1 << 31, 4, P), (P, 4, 4, 0)):
        assert lib(src, n, k, dst, 0) == INVALID
    assert lib(P + 8 if tiles_first else P, 4, 4, P if tiles_first else P + 8, 0) == INVALID


NORM = dict(x=P, xs=512, res=P, rs=512, w=P, wt=BF16, type=BF16, rows=4, cols=512, eps=1e-6, h=2 * P, hs=512, q=P,
            scale=P, static=0, stream=0)


@pytest.mark.parametrize("change", [dict(x=0), dict(x=P + 1), dict(xs=511), dict(rs=511), dict(res=P + 1), dict(w=0),
                                    dict(w=P + 1), dict(wt=I8), dict(type=I8), dict(type=7), dict(cols=0),
                                    dict(cols=32769, xs=40000, rs=40000, hs=40000), dict(eps=0.0), dict(eps=-1.0),
                                    dict(eps=math.inf), dict(eps=math.nan), dict(hs=511), dict(h=2 * P + 1), dict(q=0),
                                    dict(scale=0), dict(scale=P + 2), dict(static=2), dict(h=P, hs=600)], ids=str)
def test_norm_refusals(change):
    assert _call("lecb_rmsnorm_q8", NORM, **change) == INVALID


def test_norm_without_rows_and_with_too_many():
    assert _call("lecb_rmsnorm_q8", NORM, rows=0) == lecb.LECB_OK
    assert _call("lecb_rmsnorm_q8", NORM, rows=1 << 31) == TOO_LARGE


def test_dequantize_q8_refusals():
    good = dict(q=P, rows=3, cols=5, scale=P, ss=1, out=P, type=BF16, stream=0)
    for change in (dict(q=0), dict(q=P + 8), dict(scale=0), dict(scale=P + 1), dict(ss=2), dict(ss=-1), dict(out=0),
                   dict(out=P + 8), dict(type=I8)):
        assert _call("lecb_dequantize_q8", good, **change) == INVALID
    for change in (dict(rows=1 << 31), dict(cols=1 << 31), dict(rows=1 << 20, cols=1 << 16)):
        assert _call("lecb_dequantize_q8", good, **change) == TOO_LARGE
    assert _call("lecb_dequantize_q8", good, rows=0, q=0) == lecb.LECB_OK
    assert _call("lecb_dequantize_q8", good, cols=0, q=0) == lecb.LECB_OK


MATVEC = dict(x=P, xt=I8, xs=256, xscale=P, xss=1, m=3, tiles=P, scales=P, st=BF16, group=128, n=64, k=256, y=P, yt=BF16,
              ys=64, ws=0, wsb=0, stream=0)


@pytest.mark.parametrize("change", [dict(x=0), dict(xt=BF16, xscale=0, x=P + 1), dict(xt=F32, xscale=0), dict(xt=5),
                                    dict(xt=BF16), dict(xs=255), dict(xscale=P + 2), dict(xss=2), dict(tiles=0),
                                    dict(tiles=P + 8), dict(scales=0), dict(scales=P + 8), dict(st=F16),
                                    dict(group=96), dict(n=0), dict(k=0), dict(n=1 << 31), dict(y=0), dict(y=P + 1),
                                    dict(yt=I8), dict(ys=63)], ids=str)
def test_matvec_refusals(change):
    assert _call("lecb_matvec_w4", MATVEC, **change) == INVALID


def test_matvec_without_tokens_and_with_too_many():
    assert _call("lecb_matvec_w4", MATVEC, m=0) == lecb.LECB_OK
    assert _call("lecb_matvec_w4", MATVEC, m=1 << 31) == TOO_LARGE


# --------------------------------------------------------------------------- tensor functions (host tensors)

def _w4(n=16, k=128, group=128, **change):
    a = dict(tiles=torch.zeros(1024, dtype=torch.uint8), scales=torch.zeros(16 * (128 // group)), n=n, k=k, group=group)
    a.update(change)
    return lecb.W4Weights(**a)


@pytest.mark.parametrize("change", [dict(n=17), dict(k=129), dict(k=0), dict(n=0), dict(group=16),
                                    dict(tiles=torch.zeros(1024)), dict(tiles=torch.zeros(1023, dtype=torch.uint8)),
                                    dict(tiles=torch.zeros(2048, dtype=torch.uint8)[::2]), dict(scales=torch.zeros(15)),
                                    dict(scales=torch.zeros(16, dtype=torch.float16)), dict(scales=torch.zeros(32)[::2])],
                         ids=str)
def test_w4weights_refusals(change):
    _w4()
    with pytest.raises(ValueError):
        _w4(**change)


def test_tensor_functions_refuse():
    w = torch.zeros(16, 128)
    f = torch.zeros
    cases = [
        lambda: lecb.quantize_w4(w),                                    # not on a GPU
        lambda: lecb.quantize_w4(w.int()),
        lambda: lecb.quantize_w4(w[0]),
        lambda: lecb.quantize_w4(w[:0]),
        lambda: lecb.quantize_w4(w, group=16),
        lambda: lecb.quantize_w4(w, scale_dtype=torch.float16),
        lambda: lecb.quantize_w4(w.t()),
        lambda: lecb.dequantize_w4(_w4()),
        lambda: lecb.dequantize_w4(_w4(), torch.int8),
        lambda: lecb.tile_w4(f(16, 64, dtype=torch.uint8), 16, 128),
        lambda: lecb.tile_w4(f(16, 64, dtype=torch.uint8), 16, 127 + 2),
        lambda: lecb.tile_w4(f(16, 64), 16, 128),
        lambda: lecb.untile_w4(f(1024, dtype=torch.uint8), 16, 128),
        lambda: lecb.untile_w4(f(1024, dtype=torch.uint8), 17, 128),
        lambda: lecb.rmsnorm_q8(f(2, 8), f(8)),
        lambda: lecb.rmsnorm_q8(f(2, 8), f(9)),
        lambda: lecb.rmsnorm_q8(f(2, 8).int(), f(8)),
        lambda: lecb.rmsnorm_q8(f(2, 0), f(0)),
        lambda: lecb.rmsnorm_q8(f(2, 40000), f(40000)),
        lambda: lecb.rmsnorm_q8(f(()), f(1)),
        lambda: lecb.dequantize_q8(f(2, 8, dtype=torch.int8), f(2)),
        lambda: lecb.dequantize_q8(f(2, 8, dtype=torch.int8), f(3)),
        lambda: lecb.dequantize_q8(f(2, 8), f(2)),
        lambda: lecb.dequantize_q8(f(2, 8, dtype=torch.int8), f(2, dtype=torch.float64)),
        lambda: lecb.matvec_w4(f(1, 128, dtype=torch.int8), _w4()),
        lambda: lecb.matvec_w4(f(1, 127, dtype=torch.int8), _w4()),
        lambda: lecb.matvec_w4(f(1, 128), _w4()),
        lambda: lecb.matvec_w4(f(1, 128, dtype=torch.bfloat16), _w4(), x_scale=f(1)),
        lambda: lecb.matvec_w4(f(3, 128, dtype=torch.int8), _w4(), x_scale=f(2)),
        lambda: lecb.matvec_w4(f(1, 128, dtype=torch.int8), _w4(), out_dtype=torch.int8),
    ]
    for i, case in enumerate(cases):
        with pytest.raises(ValueError):
            case()
            pytest.fail(f"case {i} was taken")


def test_codec_import_needs_no_torch():
    """The package's host functions alone do not pull the tensor functions in."""
    import subprocess
    import sys

    code = "import lossless_entropy_coding_byte_amd as l, sys; assert 'torch' not in sys.modules; l.quantize_w4"
    assert subprocess.run([sys.executable, "-c", code], cwd=str(pytest.importorskip("pathlib").Path(__file__).parents[1])).returncode == 0
    with pytest.raises(AttributeError):
        lecb.no_such_name
    assert ctypes.sizeof(ctypes.c_void_p) == 8
