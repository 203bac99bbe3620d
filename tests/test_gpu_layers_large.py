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
