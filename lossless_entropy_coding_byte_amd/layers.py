"""Operators of quantised layers on torch tensors: what makes the 4-bit weights
and 8-bit activations that the codec stores, and what a layer computes with them.

``lecb_*`` functions mirror the C ABI of ``include/lecb.h`` (explicit buffers,
optional stream); the functions below them check shapes, types and devices
(``ValueError``), allocate their results with torch and run on the current
stream of the current device.  Every step runs in the HIP library; the functions
that a layer calls step by step are native (``csrc/tensors.cpp``).

>>> w4 = quantize_w4(weight)                             # [n, k] float -> 4-bit tiles + scales
>>> q, scale, h = rmsnorm_q8(x, norm_weight, residual=r) # h = x + r; q int8, scale per row
>>> y = matvec_w4(q, w4, x_scale=scale)                  # [rows, n] bf16
"""

from __future__ import annotations

import torch

from . import _check, _ptr, _stream, load

load()   # raises if nothing is built
from . import _tensors  # noqa: E402  (checks, results and calls of the tensor functions: csrc/tensors.cpp)

LECB_F32, LECB_BF16, LECB_F16, LECB_I8 = 0, 1, 2, 3
NORM_MAX_COLS = 32768

_TYPES = {torch.float32: LECB_F32, torch.bfloat16: LECB_BF16, torch.float16: LECB_F16, torch.int8: LECB_I8}
_SCALES = (torch.float32, torch.bfloat16)


def _type(dtype, allowed, what):
    if dtype not in allowed:
        raise ValueError(f"{what}: {dtype} is not one of {', '.join(str(d) for d in allowed)}")
    return _TYPES[dtype]


# --------------------------------------------------------------------------- the C ABI, one to one

def lecb_w4_tile_bytes(n: int, k: int) -> int:
    return load().lecb_w4_tile_bytes(n, k)


def lecb_w4_scale_count(n: int, k: int, group: int) -> int:
    return load().lecb_w4_scale_count(n, k, group)


def lecb_matvec_w4_workspace_bytes(m: int, n: int, k: int) -> int:
    return load().lecb_matvec_w4_workspace_bytes(m, n, k)


def lecb_quantize_w4(w, w_stride, n, k, group, tiles, scales, stream=None) -> None:
    _check(load().lecb_quantize_w4(_ptr(w), _TYPES[w.dtype], w_stride, n, k, group, _ptr(tiles), _ptr(scales),
                                   _TYPES[scales.dtype], _stream(stream)), "lecb_quantize_w4")


def lecb_dequantize_w4(tiles, scales, group, n, k, out, out_stride, stream=None) -> None:
    _check(load().lecb_dequantize_w4(_ptr(tiles), _ptr(scales), _TYPES[scales.dtype], group, n, k, _ptr(out),
                                     _TYPES[out.dtype], out_stride, _stream(stream)), "lecb_dequantize_w4")


def lecb_tile_w4(rows, n, k, tiles, stream=None) -> None:
    _check(load().lecb_tile_w4(_ptr(rows), n, k, _ptr(tiles), _stream(stream)), "lecb_tile_w4")


def lecb_untile_w4(tiles, n, k, rows, stream=None) -> None:
    _check(load().lecb_untile_w4(_ptr(tiles), n, k, _ptr(rows), _stream(stream)), "lecb_untile_w4")


def lecb_rmsnorm_q8(x, x_stride, res, res_stride, weight, rows, cols, eps, h, h_stride, q, scale,
                    static_scale: bool = False, stream=None) -> None:
    _check(load().lecb_rmsnorm_q8(_ptr(x), x_stride, _ptr(res), res_stride, _ptr(weight), _TYPES[weight.dtype],
                                  _TYPES[x.dtype], rows, cols, eps, _ptr(h), h_stride, _ptr(q), _ptr(scale),
                                  int(static_scale), _stream(stream)), "lecb_rmsnorm_q8")


def lecb_dequantize_q8(q, rows, cols, scale, scale_stride, out, stream=None) -> None:
    _check(load().lecb_dequantize_q8(_ptr(q), rows, cols, _ptr(scale), scale_stride, _ptr(out),
                                     _TYPES[out.dtype], _stream(stream)), "lecb_dequantize_q8")


def lecb_matvec_w4(x, x_stride, x_scale, x_scale_stride, m, tiles, scales, group, n, k, y, y_stride, ws=None,
                   stream=None) -> None:
    if ws is not None and not ws.is_contiguous():
        raise ValueError("lecb_matvec_w4: ws is contiguous")
    _check(load().lecb_matvec_w4(_ptr(x), _TYPES[x.dtype], x_stride, _ptr(x_scale), x_scale_stride, m, _ptr(tiles),
                                 _ptr(scales), _TYPES[scales.dtype], group, n, k, _ptr(y), _TYPES[y.dtype], y_stride,
                                 _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0,
                                 _stream(stream)), "lecb_matvec_w4")


# --------------------------------------------------------------------------- tensors

def _here(x, *tensors):
    """Checks that every tensor is on the current device."""
    here = torch.cuda.current_device() if x.is_cuda else None
    for t in (x, *tensors):
        if t is not None and t.get_device() != here:   # -1: host memory
            raise ValueError(f"tensor on {t.device}: the current GPU's memory is needed")


class W4Weights:
    """4-bit weights [n, k] in the tile order of ``include/lecb.h``: ``tiles``
    (uint8, lecb_w4_tile_bytes) and ``scales`` (float32 or bfloat16,
    lecb_w4_scale_count; shape [ceil(n/16), groups, 16])."""

    __slots__ = ("tiles", "scales", "n", "k", "group")

    def __init__(self, tiles, scales, n: int, k: int, group: int = 128):
        if n < 1 or k < 1 or group not in (32, 64, 128):
            raise ValueError("W4Weights: n and k are at least 1, group is 32, 64 or 128")
        cells = -(-n // 16) * -(-k // 128)
        if tiles.dtype != torch.uint8 or tiles.numel() != cells * 1024 or not tiles.is_contiguous():
            raise ValueError(f"W4Weights: tiles are {cells * 1024} contiguous uint8")
        _type(scales.dtype, _SCALES, "scales")
        if scales.numel() != cells * (2048 // group) or not scales.is_contiguous():
            raise ValueError(f"W4Weights: scales are {cells * (2048 // group)} contiguous numbers")
        self.tiles, self.scales, self.n, self.k, self.group = tiles, scales, n, k, group


def quantize_w4(w, group: int = 128, scale_dtype=torch.bfloat16) -> W4Weights:
    """Round a float matrix [n, k] to 4-bit codes with one scale per row and ``group`` columns.
    No gradient goes back to w."""
    tiles, scales = _tensors.quantize_w4(w, group, scale_dtype)
    return W4Weights(tiles, scales, *w.shape, group)


def dequantize_w4(w4: W4Weights, dtype=torch.bfloat16):
    """The weights [n, k] that the codes stand for."""
    return _tensors.dequantize_w4(w4.tiles, w4.scales, w4.group, w4.n, w4.k, dtype)


def tile_w4(rows, n: int, k: int):
    """Row-major codes (uint8 [n, ceil(k/2)], column 2j in the low half of byte j) as tiles."""
    if rows.dtype != torch.uint8 or n < 1 or k < 1 or rows.numel() != n * ((k + 1) // 2) or not rows.is_contiguous():
        raise ValueError("tile_w4: n * ceil(k / 2) contiguous uint8 are needed")
    _here(rows)
    tiles = rows.new_empty((-(-n // 16), -(-k // 128), 1024))
    lecb_tile_w4(rows, n, k, tiles)
    return tiles


def untile_w4(tiles, n: int, k: int):
    """Tiles back to row-major codes, uint8 [n, ceil(k/2)]."""
    if (tiles.dtype != torch.uint8 or n < 1 or k < 1 or not tiles.is_contiguous()
            or tiles.numel() != -(-n // 16) * -(-k // 128) * 1024):
        raise ValueError("untile_w4: the contiguous uint8 tiles of [n, k] are needed")
    _here(tiles)
    rows = tiles.new_empty((n, (k + 1) // 2))
    lecb_untile_w4(tiles, n, k, rows)
    return rows


def rmsnorm_q8(x, weight, residual=None, eps: float = 1e-6, scale=None, out_h=None):
    """h = x + residual, its root-mean-square norm times weight, in 8 bits.

    x, residual [..., cols] of one float type; weight [cols].  Returns (q int8
    [..., cols], scale float32 [...], h in x's type).  Without a residual h is
    x itself.  scale: a float32 tensor of one number fixes the scale for every
    row (values past it saturate) and is returned as given.  out_h: where h
    goes; x or residual themselves will do, other rows of theirs will not, nor
    inputs that gradients are recorded for."""
    return _tensors.rmsnorm_q8(x, weight, residual, eps, scale, out_h)


def dequantize_q8(q, scale, dtype=torch.bfloat16):
    """The values q * scale of int8 codes [..., cols]; scale: one float32 per row, or one.
    q is contiguous and 16-byte aligned (as rmsnorm_q8 returns it; rows of it may not be)."""
    return _tensors.dequantize_q8(q, scale, dtype)


def matvec_w4(x, w4: W4Weights, x_scale=None, out_dtype=None, ws=None):
    """y = x W^T for tokens x [..., k] of int8 (x_scale: float32, one per row or one), bfloat16 or float16.

    Returns y [..., n] of out_dtype (x's type; bfloat16 for int8 x).  An infinity
    or NaN in a token changes that token's results alone.  ws: a uint8 workspace
    of lecb_matvec_w4_workspace_bytes that the caller keeps; calls that overlap in
    time must not share one."""
    return _tensors.matvec_w4(x, w4.tiles, w4.scales, w4.n, w4.k, w4.group, x_scale, out_dtype, ws)
