"""Operators of quantised layers on more rows, tiles and tokens than one launch takes
(fewer than 2^32 lanes): the same bits as calls on parts."""

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from test_gpu_layers import BF16, DEV, F32, I8, U

pytestmark = pytest.mark.gpu


def need(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"{gib} GiB of GPU memory are needed")


def seeded(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# lanes a row: 64, 256
@pytest.mark.parametrize("rows,cols,part", [((1 << 26) + 1003, 8, 1 << 22), ((1 << 24) + 37, 513, 1 << 20)])
def test_norm_of_many_rows(rows, cols, part):
    need(96)
    g = seeded(cols)
    x = torch.randn(rows, cols, dtype=BF16, device=DEV, generator=g)
    r = torch.randn(rows, cols, dtype=BF16, device=DEV, generator=g)
    w = torch.rand(cols, device=DEV, generator=g) + 0.5
    fixed = torch.tensor([0.02], device=DEV)
    q, s, h = lecb.rmsnorm_q8(x, w, residual=r)
    qf, _, _ = lecb.rmsnorm_q8(x, w, scale=fixed)
    for at in range(0, rows, part):
        p = slice(at, at + part)
        for got, want in zip((q, s, h), lecb.rmsnorm_q8(x[p], w, residual=r[p])):
            assert torch.equal(got[p], want), at
        assert torch.equal(qf[p], lecb.rmsnorm_q8(x[p], w, scale=fixed)[0]), at
    got = lecb.rmsnorm_q8(x, w, residual=r, out_h=x)
    assert got[2] is x and torch.equal(x, h) and torch.equal(got[0], q) and torch.equal(got[1], s)


def test_weights_of_many_tiles():
    """2^26 tiles and some: rows of one column, so that only the tiles are long."""
    need(160)
    n, k, part = (1 << 30) + 21, 1, 1 << 24
    w = torch.randn(n, k, dtype=BF16, device=DEV, generator=seeded(1))
    w4 = lecb.quantize_w4(w)
    values = lecb.dequantize_w4(w4)
    codes = lecb.untile_w4(w4.tiles, n, k)
    tiles = lecb.tile_w4(codes, n, k)
    for at in range(0, n, part):
        rows, cells = slice(at, at + part), slice(at // 16, (at + part) // 16)
        want = lecb.quantize_w4(w[rows])
        assert torch.equal(w4.tiles[cells], want.tiles) and torch.equal(w4.scales[cells], want.scales), at
        assert torch.equal(values[rows], lecb.dequantize_w4(want)), at
        assert torch.equal(codes[rows], lecb.untile_w4(want.tiles, want.n, k)), at
        assert torch.equal(tiles[cells], want.tiles), at


def weights(n, k, group=128):
    cells, g = (-(-n // 16), -(-k // 128)), seeded(n + k)
    tiles = torch.empty(*cells, 1024, dtype=torch.uint8, device=DEV)
    for at in range(0, cells[0], 1 << 20):
        tiles[at : at + (1 << 20)].random_(0, 256, generator=g)
    scales = torch.rand(cells[0], cells[1] * 128 // group, 16, device=DEV, generator=g).to(BF16)
    return lecb.W4Weights(tiles, scales, n, k, group)


# more than 65535 workgroups of 64 tokens; of the form for few tokens, whatever their number
@pytest.mark.parametrize("m,n,k", [(65535 * 64 + 65, 64, 128), (65536 * 64 * 2 + 1, 16, 37)])
@pytest.mark.parametrize("dtype", [I8, BF16], ids=str)
def test_product_of_many_tokens(m, n, k, dtype):
    need(40)
    w4, g, part = weights(n, k), seeded(m), 1 << 20
    x = torch.randint(-99, 100, (m, k), device=DEV, generator=g, dtype=I8).to(dtype)
    xs = torch.rand(m, device=DEV, generator=g) if dtype == I8 else None
    y = lecb.matvec_w4(x, w4, x_scale=xs, out_dtype=F32)
    for at in range(0, m - part, part):
        end = at + part if at + 2 * part < m else m
        p = slice(at, end)
        assert torch.equal(y[p], lecb.matvec_w4(x[p], w4, x_scale=None if xs is None else xs[p], out_dtype=F32)), at
    w = lecb.dequantize_w4(w4, F32).double()
    for p in (slice(0, 100), slice(65535 * 64 - 50, 65535 * 64 + 50), slice(m - 100, m)):
        want = x[p].double() @ w.t()
        if xs is not None:
            want *= xs[p, None].double()
        # one group, products of whole numbers: the scale's, the factor's and the sums' roundings
        assert bool(((y[p].double() - want).abs() <= 8 * U * (x[p].double().abs() @ w.t().abs())).all())


def test_product_with_many_rows():
    """2^30 rows of W and some, of one tile of columns."""
    need(150)
    n, k, part = (1 << 30) + 21, 96, 1 << 26
    w4, g = weights(n, k), seeded(3)
    for m, dtype in ((1, I8), (3, BF16), (20, I8)):
        x = torch.randint(-99, 100, (m, k), device=DEV, generator=g, dtype=I8).to(dtype)
        out = F32 if m < 20 else BF16
        y = lecb.matvec_w4(x, w4, out_dtype=out)
        for at in range(0, n, part):
            rows, cells = slice(at, min(n, at + part)), slice(at // 16, (at + part) // 16)
            some = lecb.W4Weights(w4.tiles[cells], w4.scales[cells], rows.stop - at, k)
            assert torch.equal(y[:, rows], lecb.matvec_w4(x, some, out_dtype=out)), (m, at)
        del y


@pytest.mark.parametrize("dtype", [I8, BF16], ids=str)
def test_product_of_long_rows(dtype):
    """Tokens of 2^29 columns and some that are laid out first, nearly all of them 0, so that sums are exact."""
    need(120)
    m, n, k = 5, 3, (1 << 29) + 300
    w4, g = weights(n, k), seeded(4)
    w4.scales.fill_(0.5)
    big = torch.zeros(m, k + 9, dtype=dtype, device=DEV)
    x = big[:, 1 : k + 1]   # at odd addresses
    at = torch.cat([torch.randint(0, k, (2000,), device=DEV, generator=g), torch.tensor([0, k - 1, 1 << 28, (1 << 28) - 1], device=DEV)])
    x[:, at] = torch.randint(-99, 100, (m, at.numel()), device=DEV, generator=g, dtype=I8).to(dtype)
    y = lecb.matvec_w4(x, w4, out_dtype=F32)
    kt, at = -(-k // 128), at.unique()
    words = w4.tiles.view(-1, 1024).view(torch.int32).view(kt, 4, 16, 4)   # [c, r, d]
    col = at % 128
    codes = torch.stack([words[at // 128, col % 32 // 8, r, col // 32] << (28 - 4 * (col % 8)).int() >> 28 for r in range(n)])
    want = x[:, at].double() @ codes.t().double() * 0.5
    assert torch.equal(y.double(), want)
