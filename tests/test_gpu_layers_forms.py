"""The operators of quantised layers in each of their forms (which one takes a
call goes by its sizes): tokens in rows, 4 and 8; laid out, 16, 32 and 64 at a
time; the 32 x 32 products of many tokens.  Tolerances as in test_gpu_layers.py,
whose plain implementations these tests use."""

import math

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from test_gpu_layers import (BF16, DEV, F16, F32, F64, I8, check_matvec, gen, ref_quantize, ref_scales, ref_tiles, same,
                             tokens, weights)

pytestmark = pytest.mark.gpu

# tokens x rows that need many rounds of 64 x 32 outputs on the compute units: the form for many tokens, the
# last ones in workgroups of 512 rows; one, two and three tiles of columns, whole or not
MANY = [(300, 16400, 128), (300, 16400, 37), (257, 20001, 300), (512, 12300, 384), (64, 60000, 129), (33, 66000, 256),
        (65, 70001, 200)]


@pytest.mark.parametrize("m,n,k", MANY)
@pytest.mark.parametrize("dtype", [I8, BF16, F16], ids=str)
@pytest.mark.parametrize("group,sdt", [(32, F32), (32, BF16), (64, BF16), (64, F32), (128, BF16), (128, F32)], ids=str)
def test_many_tokens(m, n, k, dtype, group, sdt):
    """Every output's rows: the first and last 256 rows of W and the tiles between against 64 bits."""
    q, s, w4 = weights(n, k, group, sdt, m + n + k)
    x, xs = tokens(m, k, dtype, m * k)
    y = lecb.matvec_w4(x.to(DEV), w4, x_scale=None if xs is None else xs.to(DEV), out_dtype=F32)
    rows = torch.cat([torch.arange(256), torch.arange(300, n - 256, 61), torch.arange(n - 256, n)])
    check_matvec(y[:, rows.to(DEV)], x, xs, q[rows], s[rows], group)


@pytest.mark.parametrize("dtype", [I8, BF16, F16], ids=str)
def test_many_tokens_long_columns(dtype):
    """Sums over many tiles of columns, an odd number of them, the last one partial."""
    m, n, k = 70, 34000, 1111
    q, s, w4 = weights(n, k, 128, BF16, 5)
    x, xs = tokens(m, k, dtype, 6)
    xd = x.to(DEV)
    y = lecb.matvec_w4(xd, w4, x_scale=None if xs is None else xs.to(DEV), out_dtype=F32)
    rows = torch.arange(0, n, 37)
    check_matvec(y[:, rows.to(DEV)], x, xs, q[rows], s[rows], 128)
    for _ in range(3):
        assert torch.equal(y, lecb.matvec_w4(xd, w4, x_scale=None if xs is None else xs.to(DEV), out_dtype=F32))
    wide = torch.zeros(m, k + 5, dtype=dtype, device=DEV)
    wide[:, 5:] = xd
    assert torch.equal(y, lecb.matvec_w4(wide[:, 5:], w4, x_scale=None if xs is None else xs.to(DEV), out_dtype=F32))


@pytest.mark.parametrize("m", list(range(1, 18)) + [31, 32, 33, 47, 63, 64, 65, 95])
@pytest.mark.parametrize("dtype", [I8, BF16, F16], ids=str)
def test_every_number_of_tokens(m, dtype):
    """The border of each form; a token's row equals what a call of the same form gives with other tokens beside it."""
    n, k = 100, 1000
    q, s, w4 = weights(n, k, 64, BF16, m)
    x, xs = tokens(m, k, dtype, m + 1)
    xsd = None if xs is None else xs.to(DEV)
    y = lecb.matvec_w4(x.to(DEV), w4, x_scale=xsd, out_dtype=F32)
    check_matvec(y, x, xs, q, s, 64)
    other = x.clone()
    other[: m // 2] = 1
    z = lecb.matvec_w4(other.to(DEV), w4, x_scale=xsd, out_dtype=F32)
    assert torch.equal(y[m // 2 :], z[m // 2 :])


@pytest.mark.parametrize("m,n", [(3, 200), (12, 200), (60, 200), (300, 16400)])
def test_bad_tokens_stay_alone(m, n):
    q, s, w4 = weights(n, 384, 128, BF16, 2)
    for dtype in (BF16, F16):
        x = torch.randn(m, 384, generator=gen(m)).to(dtype).to(DEV)
        ref = lecb.matvec_w4(x, w4)
        x[1, 7], x[2, 300] = math.nan, math.inf
        y = lecb.matvec_w4(x, w4)
        keep = [0] + list(range(3, m))
        assert torch.equal(y[keep], ref[keep])
        assert not torch.isfinite(y[1:3].float()).any()


@pytest.mark.parametrize("m,n", [(1, 48), (7, 48), (20, 48), (70, 48), (300, 16400)])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_tokens_at_the_ends_of_their_type(m, n, dtype):
    """The largest numbers of the type (sums that fit 32 bits do not overflow on the way) and its smallest."""
    k, group = 256, 64
    q, s, w4 = weights(n, k, group, F32, 3)
    f = torch.finfo(dtype)
    base = torch.randn(m, k, generator=gen(m))
    for size in (f.max / 2 ** 13, f.smallest_normal * 2 ** 12, f.smallest_normal):
        # with |x| up to 5 size, 256 products of 8 s <= 0.1 stay below 2 ** 7 size
        x = (base.clamp(-5, 5).to(F64) * size).to(dtype)
        y = lecb.matvec_w4(x.to(DEV), w4, out_dtype=F32)
        if size * 2 ** -8 * f.eps > 2.0 ** -149:   # products are numbers of 32 bits to their last place
            check_matvec(y, x, None, q[:n], s[:n], group)
        assert bool(torch.isfinite(y).all())
    x = torch.full((m, k), f.max, dtype=dtype)
    q0 = torch.zeros(n, k, dtype=torch.int64)
    q0[:, 0] = 1
    w1 = lecb.W4Weights(ref_tiles(q0).to(DEV), ref_scales(torch.full((n, k // group), 2.0 ** -4), n, k, group).to(DEV), n, k, group)
    y = lecb.matvec_w4(x.to(DEV), w1, out_dtype=F32).cpu().to(F64)
    # one code that is not 0: 1/16 of the largest, next to a group's offsets of 24 (and as much again) that cancel
    want = torch.tensor(f.max, dtype=F64) / 16
    assert bool(((y - want).abs() <= 2 * 2.0 ** -24 * 2 * group * 56 * want).all())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("sdt", [BF16, F32], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_halves_of_steps(dtype, sdt, group):
    """16-bit weights that lie half a step between two codes, and the numbers next to them."""
    g = gen(group)
    step = (torch.rand(512, 1, generator=g) + 0.5).to(BF16).to(F32) * 2.0 ** torch.randint(-8, 9, (512, 1), generator=g)
    half = (torch.randint(-7, 7, (512, 255), generator=g) + 0.5) * step
    w = torch.cat([7 * step, half], 1).to(dtype)
    near = torch.randint(-1, 2, w.shape, generator=g)
    bits = w.view(torch.int16) + near.to(torch.int16)
    w = torch.cat([w, torch.where((w.abs() > 0.001) & (w.abs() < 100), bits.view(dtype), w)], 0)
    w[:, 0] = torch.cat([7 * step, 7 * step], 0)[:, 0].to(dtype)
    w[:, group::group] = w[:, :1]
    q, s, _ = ref_quantize(w, group, sdt)
    w4 = lecb.quantize_w4(w.to(DEV), group=group, scale_dtype=sdt)
    assert same(w4.scales, ref_scales(s, w.shape[0], 256, group))
    assert torch.equal(w4.tiles.cpu(), ref_tiles(q))


@pytest.mark.parametrize("m", [1, 4, 5, 8, 9, 13, 16])
@pytest.mark.parametrize("k", [1160, 1111, 8320])
@pytest.mark.parametrize("dtype", [I8, BF16, F16], ids=str)
def test_few_tokens_by_alignment(m, k, dtype):
    """Aligned rows are read as they lie, others laid out first: the same bits, whatever the address and stride."""
    n = 300
    q, s, w4 = weights(n, k, 64, BF16, m + k)
    x, _ = tokens(m, k, dtype, m * k)
    ref = None
    for pad, start in ((0, 0), (8, 0), (8, 8), (16, 16), (3, 0), (9, 1)):
        big = torch.zeros(m, (k + 15) // 16 * 16 + pad, dtype=dtype, device=DEV)
        big[:, start : start + k] = x.to(DEV)
        y = lecb.matvec_w4(big[:, start : start + k], w4, out_dtype=F32)
        if ref is None:
            ref = y
            check_matvec(y, x, None, q, s, 64)
        assert torch.equal(y, ref), (pad, start)


@pytest.mark.parametrize("m", [1, 4, 7, 12, 16, 20, 40, 70])
@pytest.mark.parametrize("n,k", [(7, 28672), (300, 9000), (40, 20001)])
@pytest.mark.parametrize("dtype", [I8, BF16], ids=str)
def test_few_rows_and_many_columns(m, n, k, dtype):
    """Columns shared out over workgroups, the last share shorter, its last tile partial; strided rows, same bits."""
    q, s, w4 = weights(n, k, 128, BF16, m + k)
    x, xs = tokens(m, k, dtype, m * k)
    xd, xsd = x.to(DEV), None if xs is None else xs.to(DEV)
    y = lecb.matvec_w4(xd, w4, x_scale=xsd, out_dtype=F32)
    check_matvec(y, x, xs, q, s, 128)
    big = torch.zeros(m, k + 3, dtype=dtype, device=DEV)
    big[:, 1 : k + 1] = xd
    for _ in range(2):
        assert torch.equal(y, lecb.matvec_w4(big[:, 1 : k + 1], w4, x_scale=xsd, out_dtype=F32))
    assert torch.equal(y.to(BF16), lecb.matvec_w4(xd, w4, x_scale=xsd, out_dtype=BF16))


def test_workspace_of_the_caller():
    """A workspace kept by the caller, its contents of no matter; calls with less are refused."""
    q, s, w4 = weights(80, 512, 64, BF16, 11)
    for m in (9, 33, 200):
        need = lecb.lecb_matvec_w4_workspace_bytes(m, 80, 512)
        x, xs = tokens(m, 512, BF16, m)
        xd = x.to(DEV)
        ref = lecb.matvec_w4(xd, w4)
        for fill in (0, 255):
            ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
            assert torch.equal(lecb.matvec_w4(xd, w4, ws=ws), ref)
        with pytest.raises(lecb.LecbError) as e:
            lecb.matvec_w4(xd, w4, ws=torch.empty(need - 16, dtype=torch.uint8, device=DEV))
        assert e.value.status == lecb.LECB_ERR_WORKSPACE
    assert lecb.lecb_matvec_w4_workspace_bytes(8, 80, 512) == 0
