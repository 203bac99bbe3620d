"""The 8-bit cache and its attention, without a GPU: sizes, and every refusal of the C ABI and of the tensor
functions (all of them come before any launch)."""

import ctypes
import math

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from cache_helpers import padded, places

P = 1 << 20          # an aligned address that is never touched: every call below is refused
INVALID, WORKSPACE, TOO_LARGE = lecb.LECB_ERR_INVALID_ARG, lecb.LECB_ERR_WORKSPACE, lecb.LECB_ERR_TOO_LARGE
F32, BF16, F16, I8 = 0, 1, 2, 3
CACHE = dict(k=P, v=P, k_scale=P, v_scale=P, blocks=10, heads=4, dim=80, block=64)
SEQS = dict(table=P, lengths=P, starts=P, table_stride=5, width=5, seqs=3, tokens=7)
WRITE = dict(k=P, v=P, type=BF16, kt=320, kh=80, vt=320, vh=80, stream=0)
READ = dict(k=P, v=P, type=BF16, fill=1, stream=0)
ATTEND = dict(scale=0.1, causal=1, window=0, out=P, ot=640, oh=80, fill=1, ws=P, wsb=1 << 40, stream=0)

BAD_CACHE = [dict(k=0), dict(v=0), dict(k=P + 8), dict(v=P + 8), dict(k_scale=0), dict(v_scale=0), dict(k_scale=P + 2),
             dict(v_scale=P + 2), dict(blocks=0), dict(blocks=1 << 31), dict(heads=0), dict(heads=65536), dict(dim=0),
             dict(dim=257), dict(block=0), dict(block=16), dict(block=48), dict(block=512)]
BAD_SEQS = [dict(table=0), dict(table=P + 2), dict(lengths=0), dict(lengths=P + 1), dict(starts=P + 2), dict(starts=0),
            dict(width=0), dict(table_stride=4)]
LARGE_SEQS = [dict(width=(1 << 31) // 64, table_stride=1 << 30), dict(seqs=1 << 20), dict(tokens=1 << 27)]


def structs(**change):
    cache, seqs = dict(CACHE), dict(SEQS)
    for name, value in change.items():
        (cache if name in cache else seqs)[name] = value
    return lecb.lecb_cache_q8(**cache), lecb.lecb_cache_seqs(**seqs)


def call_write(cache, seqs, **change):
    a = {**WRITE, **change}
    return lecb.load().lecb_cache_write_q8(ctypes.byref(cache), ctypes.byref(seqs), *a.values())


def call_read(cache, seqs, **change):
    a = {**READ, **change}
    return lecb.load().lecb_cache_read_q8(ctypes.byref(cache), ctypes.byref(seqs), *a.values())


def call_attend(cache, seqs, q=P, qt=640, qh=80, type=BF16, heads=8, **change):
    a = {**ATTEND, **change}
    assert set(a) == set(ATTEND)
    return lecb.load().lecb_attention_q8(q, qt, qh, type, heads, ctypes.byref(cache), ctypes.byref(seqs), *a.values())


def test_sizes():
    for dim in (1, 64, 65, 96, 97, 128, 129, 192, 193, 256):
        for block in (32, 64, 128, 256):
            assert lecb.lecb_cache_q8_bytes(7, 3, dim, block) == 7 * 3 * block * padded(dim)
    for bad in ((0, 3, 64, 32), (1 << 31, 3, 64, 32), (7, 0, 64, 32), (7, 65536, 64, 32), (7, 3, 0, 32), (7, 3, 257, 32),
                (7, 3, 64, 16), (7, 3, 64, 96)):
        assert lecb.lecb_cache_q8_bytes(*bad) == 0


@pytest.mark.parametrize("keys", [True, False])
def test_the_stated_order_is_one_to_one(keys):
    at = places(64, 96, keys)
    assert sorted(at.view(-1).tolist()) == list(range(64 * 96))


@pytest.mark.parametrize("call", [call_write, call_read, call_attend], ids=lambda f: f.__name__)
@pytest.mark.parametrize("change", BAD_CACHE + BAD_SEQS, ids=str)
def test_refused_structs(call, change):
    assert call(*structs(**change)) == INVALID


@pytest.mark.parametrize("call", [call_write, call_read, call_attend], ids=lambda f: f.__name__)
@pytest.mark.parametrize("change", LARGE_SEQS, ids=str)
def test_too_large(call, change):
    assert call(*structs(**change)) == TOO_LARGE


@pytest.mark.parametrize("call", [call_write, call_read, call_attend], ids=lambda f: f.__name__)
def test_nothing_to_do(call):
    assert call(*structs(tokens=0)) == lecb.LECB_OK
    assert call(*structs(tokens=0, seqs=0, table=0, lengths=0, starts=0, width=0)) == lecb.LECB_OK


@pytest.mark.parametrize("change", [dict(k=0), dict(v=0), dict(k=P + 1), dict(v=P + 1), dict(type=I8), dict(type=7)], ids=str)
def test_write_refusals(change):
    assert call_write(*structs(), **change) == INVALID


@pytest.mark.parametrize("change", [dict(k=0), dict(v=0), dict(k=P + 1), dict(v=P + 1), dict(type=I8), dict(fill=2)], ids=str)
def test_read_refusals(change):
    assert call_read(*structs(), **change) == INVALID


@pytest.mark.parametrize("change", [dict(q=0), dict(q=P + 1), dict(type=I8), dict(heads=0), dict(heads=6), dict(scale=math.inf),
                                    dict(scale=math.nan), dict(causal=2), dict(window=5, causal=0), dict(window=1 << 31),
                                    dict(out=0), dict(out=P + 1), dict(ot=79), dict(oh=79), dict(fill=2)], ids=str)
def test_attention_refusals(change):
    assert call_attend(*structs(), **change) == INVALID


def test_attention_workspace_and_rows():
    # a long table: the keys of few rows are shared out over workgroups, whose sums go through the workspace
    cache, seqs = structs(width=1000, table_stride=1000)
    need = lecb.lecb_attention_q8_workspace_bytes(cache, 3, 7, 1000, 8)
    assert need > 0 and need % 16 == 0
    assert call_attend(cache, seqs, ws=0) == INVALID
    assert call_attend(cache, seqs, ws=P + 8) == INVALID
    assert call_attend(cache, seqs, wsb=need - 1) == WORKSPACE
    assert lecb.lecb_attention_q8_workspace_bytes(cache, 3, 7, 1, 8) == 0      # one block: nothing to share out
    for bad in ((0, 7, 1000, 8), (3, 0, 1000, 8), (1 << 20, 7, 1000, 8), (3, 1 << 27, 1000, 8), (3, 7, 1 << 26, 8),
                (3, 7, 1000, 6), (3, 7, 1000, 0)):
        assert lecb.lecb_attention_q8_workspace_bytes(cache, *bad) == 0
    assert call_attend(*structs(tokens=1 << 24)) == TOO_LARGE                  # by 8 heads
    # a workspace for a table serves narrower ones and fewer rows
    sizes = [lecb.lecb_attention_q8_workspace_bytes(cache, 3, 7, w, 8) for w in (1, 10, 100, 1000, 10000)]
    assert sizes == sorted(sizes)


# --------------------------------------------------------------------------- tensor functions (host tensors)

def tensors(**change):
    a = dict(k=torch.zeros(7, 4, 80), v=torch.zeros(7, 4, 80), q=torch.zeros(7, 8, 80),
             table=torch.zeros(3, 5, dtype=torch.int32), lengths=torch.zeros(3, dtype=torch.int32),
             starts=torch.zeros(4, dtype=torch.int32), cache=lecb.new_cache_q8(10, 4, 80, 64, device="cpu"))
    a.update(change)
    return a


def refused(match, call):
    with pytest.raises(ValueError, match=match):
        call()


def everything(match, **change):
    a = tensors(**change)
    refused(match, lambda: lecb.cache_write_q8(a["cache"], a["k"], a["v"], a["table"], a["lengths"], a["starts"]))
    refused(match, lambda: lecb.cache_read_q8(a["cache"], a["table"], a["lengths"], a["starts"], 7))
    refused(match, lambda: lecb.attention_q8(a["q"], a["cache"], a["table"], a["lengths"], a["starts"]))


i32 = torch.int32


def test_host_memory_is_refused():
    everything("current GPU")


@pytest.mark.parametrize("change", [dict(table=torch.zeros(3, 5)), dict(table=torch.zeros(2, 5, dtype=i32)),
                                    dict(table=torch.zeros(3, dtype=i32)), dict(table=torch.zeros(3, 0, dtype=i32)),
                                    dict(table=torch.zeros(5, 3, dtype=i32).t()), dict(table=torch.zeros(1, 5, dtype=i32).expand(3, 5)),
                                    dict(table=torch.zeros(3, 5, dtype=torch.int64))], ids=lambda c: str(c["table"].shape))
def test_tables(change):
    everything("table", **change)


@pytest.mark.parametrize("change", [dict(lengths=torch.zeros(3)), dict(lengths=torch.zeros(3, 1, dtype=i32)),
                                    dict(lengths=torch.zeros(6, dtype=i32)[::2]), dict(lengths=torch.zeros(0, dtype=i32)),
                                    dict(lengths=torch.zeros(3, dtype=torch.int64))], ids=lambda c: str(c["lengths"].dtype))
def test_lengths(change):
    everything("lengths", **change)


def test_starts():
    for starts in (torch.zeros(3, dtype=i32), torch.zeros(4), torch.zeros(8, dtype=i32)[::2], torch.zeros(4, 1, dtype=i32)):
        everything("starts", starts=starts)
    everything("without starts", starts=None)
    refused("number of rows", lambda: lecb.cache_read_q8(tensors()["cache"], tensors()["table"], tensors()["lengths"], tensors()["starts"]))
    a = tensors()
    refused("negative", lambda: lecb.cache_read_q8(a["cache"], a["table"], a["lengths"], a["starts"], -1))


@pytest.mark.parametrize("field,value", [("dim", 0), ("dim", 257), ("dim", 97), ("block", 48), ("block", 32), ("k", torch.zeros(5, dtype=torch.int8)),
                                         ("v", torch.zeros(10 * 4 * 64 * 96)), ("k", torch.zeros(1, dtype=torch.int8).expand(10 * 4 * 64 * 96)),
                                         ("k_scale", torch.zeros(40)), ("v_scale", torch.zeros(10, 5)),
                                         ("v_scale", torch.zeros(10, 4, dtype=torch.float64)), ("k_scale", torch.zeros(4, 10).t())], ids=str)
def test_caches_changed_after_they_were_made(field, value):
    """Kernels go by the fields: those that no longer fit one another are refused at each call."""
    a = tensors()
    setattr(a["cache"], field, value)
    everything("cache", cache=a["cache"])


def test_cache_refusals():
    ok = lecb.new_cache_q8(2, 3, 40, 32, device="cpu")
    lecb.CacheQ8(ok.k, ok.v, ok.k_scale, ok.v_scale, 40, 32)
    for change in (dict(dim=65), dict(dim=0), dict(block=16), dict(block=-32), dict(k=ok.k[:1]), dict(v=ok.v.float()), dict(v=ok.v.transpose(0, 1)),
                   dict(k_scale=ok.k_scale[0]), dict(v_scale=ok.v_scale[:1]), dict(v_scale=ok.v_scale.half()),
                   dict(k_scale=torch.zeros(2, 1).expand(2, 3))):
        args = dict(k=ok.k, v=ok.v, k_scale=ok.k_scale, v_scale=ok.v_scale, dim=40, block=32)
        args.update(change)
        refused("CacheQ8", lambda: lecb.CacheQ8(**args))
    for bad in ((0, 1, 1, 32), (1, 0, 1, 32), (1, 1, 0, 32), (1, 1, 1, 33), (-1, 1, 1, 32), (1, 1, 300, 32)):
        refused("new_cache_q8", lambda: lecb.new_cache_q8(*bad, device="cpu"))


def test_rows_refused():
    for x, match in ((torch.zeros(7, 5, 80), "heads and dim"), (torch.zeros(7, 4, 81), "heads and dim"), (torch.zeros(7, 320), "tokens, heads"),
                     (torch.zeros(7, 4, 80, dtype=torch.int8), "types"), (torch.zeros(7, 80, 4).transpose(1, 2), "contiguous")):
        a = tensors(k=x, v=x)
        refused(match, lambda: lecb.cache_write_q8(a["cache"], a["k"], a["v"], a["table"], a["lengths"], a["starts"]))
    for v in (torch.zeros(6, 4, 80), torch.zeros(7, 4, 80, dtype=torch.bfloat16)):
        a = tensors(v=v)
        refused("shape and type", lambda: lecb.cache_write_q8(a["cache"], a["k"], a["v"], a["table"], a["lengths"], a["starts"]))
    a = tensors()
    refused("types", lambda: lecb.cache_read_q8(a["cache"], a["table"], a["lengths"], a["starts"], 7, torch.int8))


def test_attention_rows_refused():
    a = tensors()

    def attend(q=a["q"], **more):
        return lecb.attention_q8(q, a["cache"], a["table"], a["lengths"], a["starts"], **more)

    for q, match in ((torch.zeros(7, 6, 80), "multiple"), (torch.zeros(7, 8, 64), "dim"), (torch.zeros(7, 640), "tokens, heads"),
                     (torch.zeros(7, 8, 80, dtype=torch.int8), "types"), (torch.zeros(7, 80, 8).transpose(1, 2), "contiguous")):
        refused(match, lambda: attend(q))
    for more, match in ((dict(scale=math.inf), "scale"), (dict(scale=1e300), "scale"), (dict(window=0), "window"), (dict(window=-1), "window"),
                        (dict(window=1 << 31), "window"), (dict(window=4, causal=False), "window"),
                        (dict(ws=torch.zeros(64)), "ws"), (dict(ws=torch.zeros(1, dtype=torch.uint8).expand(99)), "ws"),
                        (dict(out=torch.zeros(7, 8, 81)), "out"), (dict(out=torch.zeros(7, 8, 80, dtype=torch.bfloat16)), "out"),
                        (dict(out=torch.zeros(1, 8, 80).expand(7, 8, 80)), "overlap"), (dict(out=torch.zeros(7, 1, 80).expand(7, 8, 80)), "overlap"),
                        (dict(out=torch.zeros(7 * 640).as_strided((7, 8, 80), (80, 80, 1))), "overlap"),
                        (dict(out=a["q"]), "overlaps"), (dict(out=torch.zeros(7, 80, 8).transpose(1, 2)), "contiguous")):
        refused(match, lambda: attend(**more))
    # results beside the queries in one buffer, heads or tokens outermost
    wide = torch.zeros(7, 20, 80)
    refused("current GPU", lambda: attend(wide[:, :8], out=wide[:, 8:16]))
    refused("overlaps", lambda: attend(wide[:, :8], out=wide[:, 7:15]))
    refused("current GPU", lambda: attend(out=torch.zeros(8, 7, 80).transpose(0, 1)))
    refused("overlaps", lambda: attend(ws=a["cache"].k.view(torch.uint8)))
    refused("overlaps", lambda: attend(out=a["cache"].k.view(torch.float32).view(-1)[: 7 * 640].view(7, 8, 80)))


def test_what_a_write_reads_is_not_the_cache():
    a = tensors()
    inside = a["cache"].k.view(torch.float32).view(-1)[: 7 * 320].view(7, 4, 80)
    refused("overlaps", lambda: lecb.cache_write_q8(a["cache"], inside, a["v"], a["table"], a["lengths"], a["starts"]))
    table = a["cache"].v_scale.view(torch.int32)[:3]
    refused("overlaps", lambda: lecb.cache_write_q8(a["cache"], a["k"], a["v"], table, a["lengths"], a["starts"]))


def test_gradients_and_tangents():
    from torch.autograd import forward_ad as fw

    a = tensors()
    with fw.dual_level():
        dual = {n: fw.make_dual(a[n], torch.ones_like(a[n])) for n in ("k", "q")}
        refused("forward-mode", lambda: lecb.cache_write_q8(a["cache"], dual["k"], a["v"], a["table"], a["lengths"], a["starts"]))
        refused("forward-mode", lambda: lecb.attention_q8(dual["q"], a["cache"], a["table"], a["lengths"], a["starts"]))
    a["cache"].k_scale.requires_grad_()
    refused("gradients", lambda: lecb.cache_write_q8(a["cache"], a["k"], a["v"], a["table"], a["lengths"], a["starts"]))
    q = a["q"].clone().requires_grad_()
    refused("gradients", lambda: lecb.attention_q8(q, a["cache"], a["table"], a["lengths"], a["starts"], out=torch.zeros(7, 8, 80)))
