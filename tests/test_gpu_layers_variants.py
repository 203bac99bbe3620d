"""matvec_w4 for few tokens against many rows of W, where a wave takes two or four
tiles of rows: every group, type of scales and of tokens, tokens in rows and laid
out, all outputs against 64 bits.

16 tokens a workgroup take two tiles from 8192 rows on and four from 16384, 32
alike, 64 two.  Tolerances: products are exact; int8 tokens' group sums are whole
numbers below 2^24, then comes one rounding a group, one for each of up to 16 waves'
sums, the factors and the result: (groups + 24) u of the sum of |x q s|.  16-bit
tokens' group sums have up to group additions of 2 u each besides."""

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from test_gpu_layers import BF16, DEV, F16, F32, F64, I8, U

pytestmark = pytest.mark.gpu

TOKENS = [1, 4, 6, 8, 12, 16, 20, 32, 40, 64]


def make(n, k, group, sdt):
    """(codes [n, k], scales [n, groups], the two as W4Weights), from the layout's definition."""
    g = torch.Generator(device=DEV)
    g.manual_seed(n + k + group)
    nt, kt, per = -(-n // 16), -(-k // 128), 128 // group
    q = torch.randint(-8, 8, (n, k), device=DEV, generator=g)
    s = (0.004 + 0.008 * torch.rand(n, -(-k // group), device=DEV, generator=g)).to(sdt)
    full = torch.nn.functional.pad(q, (0, kt * 128 - k, 0, nt * 16 - n)) & 15
    words = sum(full[:, i::8] << (4 * i) for i in range(8))            # [rows, kt * 16]: word 4 d + c
    words = words.view(nt, 16, kt, 4, 4).permute(0, 2, 4, 1, 3)        # [nt, kt, c, r, d]
    tiles = torch.stack([words >> (8 * i) & 255 for i in range(4)], -1).to(torch.uint8).reshape(nt, kt, 1024)
    scales = torch.zeros(nt * 16, kt * per, dtype=sdt, device=DEV)
    scales[:n, : s.shape[1]] = s
    scales = scales.view(nt, 16, kt * per).permute(0, 2, 1).contiguous()
    return q, s, lecb.W4Weights(tiles, scales, n, k, group)


@pytest.mark.parametrize("n", [8200, 16400, 20001])
@pytest.mark.parametrize("k", [129, 384, 1111, 2200])   # tokens of 2200 columns at odd addresses are laid out first
@pytest.mark.parametrize("group,sdt", [(32, F32), (32, BF16), (64, F32), (64, BF16), (128, F32), (128, BF16)], ids=str)
def test_many_rows_few_tokens(n, k, group, sdt):
    q, s, w4 = make(n, k, group, sdt)
    w = q.to(F64) * s.to(F64).repeat_interleave(group, 1)[:, :k]
    size, g = w.abs(), torch.Generator(device=DEV)
    g.manual_seed(k)
    groups = s.shape[1]
    for dtype in (I8, BF16, F16):
        big = torch.zeros(max(TOKENS), (k + 31) // 16 * 16, dtype=dtype, device=DEV)
        big.copy_(torch.randint(-127, 128, big.shape, device=DEV, generator=g) if dtype == I8
                  else torch.randn(big.shape, device=DEV, generator=g))
        xs = 0.01 + 0.02 * torch.rand(max(TOKENS), device=DEV, generator=g) if dtype == I8 else None
        for m in TOKENS:
            for start in (0, 1) if k == 2200 else (0,):
                x = big[:m, start : start + k]
                f = xs[:m, None].to(F64) if dtype == I8 else 1.0
                want, most = (x.to(F64) @ w.t()) * f, (x.to(F64).abs() @ size.t()) * f
                y = lecb.matvec_w4(x, w4, x_scale=None if xs is None else xs[:m], out_dtype=F32).to(F64)
                tol = (groups + 24 + (0 if dtype == I8 else 2 * group)) * U * most
                worst = ((y - want).abs() - tol).max().item()
                assert worst <= 0, (m, dtype, start, worst)
