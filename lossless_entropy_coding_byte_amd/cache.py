"""The 8-bit cache of keys and values on torch tensors, and the attention that
reads it: what lies between a layer's products.

``lecb_*`` functions mirror the C ABI of ``include/lecb.h`` (explicit buffers,
optional stream); the functions below them check shapes, types and devices
(``ValueError``), allocate their results with torch and run on the current stream
of the current device.  They are native (``csrc/tensors.cpp``) and run forwards only.

>>> cache = new_cache_q8(blocks, kv_heads, head_dim, block=64)
>>> cache_write_q8(cache, k, v, table, lengths, starts)     # the new tokens' keys and values
>>> out = attention_q8(q, cache, table, lengths, starts)    # of their queries over all tokens so far

Sequences: ``table`` int32 [seqs, blocks], row s the cache's blocks of sequence s in
order; ``lengths`` int32 [seqs], its tokens with this call's; ``starts`` int32
[seqs + 1], rising: rows starts[s] .. starts[s + 1] - 1 of the call are its last
tokens.  Without starts row s is sequence s's newest token.  All three stay on the
GPU: a captured step follows what is written into them between replays.
"""

from __future__ import annotations

import ctypes

import torch

from . import _check, _ptr, _stream, load
from .layers import _TYPES, _tensors


# --------------------------------------------------------------------------- the C ABI, one to one

class lecb_cache_q8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("blocks", ctypes.c_uint64), ("heads", ctypes.c_uint32),
                ("dim", ctypes.c_uint32), ("block", ctypes.c_uint32)]


class lecb_cache_seqs(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("starts", ctypes.c_void_p),
                ("table_stride", ctypes.c_uint64), ("width", ctypes.c_uint32), ("seqs", ctypes.c_uint32),
                ("tokens", ctypes.c_uint32)]


def _fits(*numbers: int) -> bool:
    # ctypes keeps the low bits of what does not
    return min(numbers) >= 0 and max(numbers) < 1 << 32


def lecb_cache_q8_bytes(blocks: int, heads: int, dim: int, block: int) -> int:
    if not _fits(blocks, heads, dim, block):
        return 0
    return load().lecb_cache_q8_bytes(blocks, heads, dim, block)


def lecb_cache_write_q8(cache: lecb_cache_q8, seqs: lecb_cache_seqs, k, k_token, k_head, v, v_token, v_head,
                        stream=None) -> None:
    _check(load().lecb_cache_write_q8(ctypes.byref(cache), ctypes.byref(seqs), _ptr(k), _ptr(v), _TYPES[k.dtype],
                                      k_token, k_head, v_token, v_head, _stream(stream)), "lecb_cache_write_q8")


def lecb_cache_read_q8(cache: lecb_cache_q8, seqs: lecb_cache_seqs, k, v, fill: bool = True, stream=None) -> None:
    _check(load().lecb_cache_read_q8(ctypes.byref(cache), ctypes.byref(seqs), _ptr(k), _ptr(v), _TYPES[k.dtype],
                                     int(fill), _stream(stream)), "lecb_cache_read_q8")


def lecb_attention_q8_workspace_bytes(cache: lecb_cache_q8, seqs: int, tokens: int, width: int, heads: int) -> int:
    if not _fits(seqs, tokens, width, heads):
        return 0
    return load().lecb_attention_q8_workspace_bytes(ctypes.byref(cache), seqs, tokens, width, heads)


def lecb_attention_q8(q, q_token, q_head, heads, cache: lecb_cache_q8, seqs: lecb_cache_seqs, scale, causal, window,
                      out, out_token, out_head, fill: bool = True, ws=None, stream=None) -> None:
    if ws is not None and not ws.is_contiguous():
        raise ValueError("lecb_attention_q8: ws is contiguous")
    if not _fits(heads, window):
        raise ValueError("lecb_attention_q8: heads and window are below 2^32")
    _check(load().lecb_attention_q8(_ptr(q), q_token, q_head, _TYPES[q.dtype], heads, ctypes.byref(cache),
                                    ctypes.byref(seqs), scale, int(causal), window, _ptr(out), out_token, out_head,
                                    int(fill), _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0,
                                    _stream(stream)), "lecb_attention_q8")


# --------------------------------------------------------------------------- tensors

class CacheQ8:
    """Keys and values of ``blocks`` blocks of ``block`` tokens (32, 64, 128 or 256) in the order of
    ``include/lecb.h``: ``k`` and ``v`` (int8, lecb_cache_q8_bytes each), ``k_scale`` and ``v_scale`` (float32
    [blocks, heads]).  The codes are bytes to the codec; a block's are adjacent."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "dim", "block")

    def __init__(self, k, v, k_scale, v_scale, dim: int, block: int = 64):
        if k_scale.dim() != 2:
            raise ValueError("CacheQ8: scales are [blocks, heads]")
        size = lecb_cache_q8_bytes(*k_scale.shape, dim, block) if 0 < dim <= 256 and block > 0 else 0
        if not size:
            raise ValueError("CacheQ8: 1 to 2^31 - 1 blocks of 32, 64, 128 or 256 tokens, 1 to 65535 heads of 1 to 256 "
                             "dimensions are needed")
        for t in (k, v):
            if t.dtype != torch.int8 or t.numel() != size or not t.is_contiguous():
                raise ValueError(f"CacheQ8: k and v are {size} contiguous int8")
        for t in (k_scale, v_scale):
            if t.dtype != torch.float32 or t.shape != k_scale.shape or not t.is_contiguous():
                raise ValueError("CacheQ8: scales are contiguous float32 [blocks, heads]")
        self.k, self.v, self.k_scale, self.v_scale, self.dim, self.block = k, v, k_scale, v_scale, dim, block


def new_cache_q8(blocks: int, heads: int, dim: int, block: int = 64, device=None) -> CacheQ8:
    """A cache of zeros on ``device`` (the current GPU)."""
    size = lecb_cache_q8_bytes(blocks, heads, dim, block) if min(blocks, heads, dim, block) > 0 else 0
    if not size:
        raise ValueError("new_cache_q8: 1 to 2^31 - 1 blocks of 32, 64, 128 or 256 tokens, 1 to 65535 heads of 1 to 256 "
                         "dimensions are needed")
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    shape = (blocks, heads, size // (blocks * heads))
    codes = [torch.zeros(shape, dtype=torch.int8, device=device) for _ in range(2)]
    scales = [torch.zeros(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
    return CacheQ8(*codes, *scales, dim, block)


def cache_write_q8(cache: CacheQ8, k, v, table, lengths, starts=None) -> None:
    """Quantise the new tokens' keys and values [tokens, heads, dim] (float32, bfloat16 or float16; tokens and heads
    at any stride) into the cache.

    Each block has one scale for each head's keys and one for its values.  A block that holds older tokens of the
    sequence keeps its scale while that is enough; else it grows, by a quarter at least, and the older
    codes are rounded again.  The blocks that a call writes must belong to one sequence each and stand in its
    row of the table once.  Tokens whose
    block is not one of the cache's, or whose sequence is longer than its row of the table, are left out.  An
    infinity or NaN makes the block's scale for this head NaN.  No gradient goes back to k and v; where one is recorded
    for them, a warning says so."""
    _tensors.cache_write_q8(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.dim, cache.block, k, v, table, lengths,
                            starts)


def cache_read_q8(cache: CacheQ8, table, lengths, starts=None, tokens: int | None = None, dtype=torch.bfloat16):
    """The keys and values of the sequences' last tokens as the cache holds them: (k, v), [tokens, heads, dim] each.

    Sequence s gives its last starts[s + 1] - starts[s] tokens, to these rows; ``tokens`` is the number of rows,
    starts[-1] (without starts: one to each sequence).  Rows whose block is not one of the cache's, or whose
    sequence is longer than its row of the table, are NaN; rows without a token are 0."""
    if tokens is None:
        if starts is not None:
            raise ValueError("cache_read_q8: with starts the number of rows, tokens, is needed")
        tokens = lengths.numel()
    return _tensors.cache_read_q8(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.dim, cache.block, table, lengths,
                                  starts, tokens, dtype)


def attention_q8(q, cache: CacheQ8, table, lengths, starts=None, scale: float | None = None, causal: bool = True,
                 window: int | None = None, out=None, ws=None):
    """Softmax attention of q [tokens, heads, dim] (float32, bfloat16 or float16) over the cache.

    heads is a multiple of the cache's: query head h reads head h // (heads / cache heads).  A row sees its
    sequence's tokens up to its own (causal: all of them where false), the last ``window`` of these if given.
    scale: 1 / sqrt(dim).  Returns [tokens, heads, dim] in q's type.  A row that sees nothing is 0; so is a row of
    no sequence, which a given ``out`` keeps as it was.  A row that sees a block with a scale that is not finite, one
    that is not the cache's, or that belongs to a sequence longer than its row of the table, is NaN; what
    is masked never matters.  The order of sums follows from the lengths of all sequences.  Products and sums have 32
    bits, the softmax's weights 22 in the second product; 11 for bfloat16 where a sequence has more than 64 rows by
    heads of one cache head.  out: must not overlap what is read.  ws: a uint8 workspace of
    lecb_attention_q8_workspace_bytes that the caller keeps; calls that overlap in time must not share one."""
    return _tensors.attention_q8(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.dim, cache.block, q, table, lengths,
                                 starts, scale, causal, window, out, ws)
