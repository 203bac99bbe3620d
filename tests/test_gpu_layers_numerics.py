"""matvec_w4 with 16-bit tokens where sums lose most: tokens of one sign, columns
far larger than the rest whose codes are 0, infinities, the smallest numbers and
the largest scales.

Tolerances, for fp32 results, u = 2^-24.  A product x q has at most 15 bits and is
exact in 32; of a group's sum every addition is rounded (2 u: the matrix unit may
cut off) at no more than the group's sum of |x q|; then come one rounding a group
and those of the waves' sums.  So the error is at most (2 group + groups + 24) u of
the sum of |x q s|: a column whose code is 0 takes no part, whatever x is there.

By the norm: a group's own roundings are small against the whole (its sum is), which
leaves the groups that a wave adds up, u / sqrt(3) of the partial sum each, their sizes
growing to the whole's: about sqrt(groups / waves / 3) u and a few for the waves' sums;
64 groups over 4 waves and more: below 4 u.  8 u are allowed."""

import math

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb
from test_gpu_layers import BF16, DEV, F16, F32, F64, U, gen, ref_scales, ref_tiles

pytestmark = pytest.mark.gpu

# each form: tokens in rows, laid out for 16 (odd rows), 32 and 64, many
FORMS = [(1, 96, 4096), (6, 96, 4096), (12, 96, 4096), (20, 96, 4096), (40, 96, 4096), (300, 16400, 1024)]
KINDS = ["normal", "positive", "outlier", "huge", "alternating"]


def make(m, n, k, group, dtype, kind, seed):
    g = gen(seed)
    q = torch.randint(-8, 8, (n, k), generator=g)
    s = 0.004 + 0.008 * torch.rand(n, k // group, generator=g)
    x = torch.randn(m, k, generator=g)
    if kind == "positive":
        x = x.clamp_min(0)
    if kind == "alternating":   # one sign over each group, the signs in turn
        x = x.abs() * (1 - 2 * (torch.arange(k) // group % 2))
    if kind in ("outlier", "huge"):
        for c in (5, k // 2 + 77):
            x[:, c] = 1000.0 if kind == "outlier" else 3e4
            q[::2, c] = 0
    return x.to(dtype), q, s


def exact(x, q, s, group):
    """(x W^T, the sum of |x q s|) in 64 bits."""
    w = q.to(F64) * s.to(F64).repeat_interleave(group, 1)
    return x.to(F64) @ w.t(), x.to(F64).abs() @ w.abs().t()


@pytest.mark.parametrize("m,n,k", FORMS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_errors_follow_the_products(m, n, k, kind, dtype, group):
    x, q, s = make(m, n, k, group, dtype, kind, m + group)
    w4 = lecb.W4Weights(ref_tiles(q).to(DEV), ref_scales(s, n, k, group).to(DEV), n, k, group)
    rows = torch.arange(0, n, 2)[:200]   # those whose codes are 0 at the large columns
    rows = torch.cat([rows, torch.arange(1, min(n, 400), 2)])
    y = lecb.matvec_w4(x.to(DEV), w4, out_dtype=F32)[:, rows.to(DEV)].cpu().to(F64)
    want, size = exact(x, q[rows], s[rows], group)
    off = (y - want).abs()
    assert bool((off <= (2 * group + k // group + 24) * U * size).all()), (off / size).max().item() / U
    even = rows % 2 == 0
    rel = ((y - want)[:, even].norm() / want[:, even].norm()).item()
    assert rel <= 8 * U, rel / U


@pytest.mark.parametrize("m,n,k", [(3, 80, 400), (12, 80, 401), (40, 80, 400), (300, 16400, 400)])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_infinities_as_the_formula_has_them(m, n, k, dtype):
    """An infinity times a code that is not 0 keeps its sign, times 0 it is NaN; other tokens do not see it."""
    g = gen(7)
    q = torch.randint(-8, 8, (n, k), generator=g)
    s = 0.01 + torch.rand(n, -(-k // 64), generator=g)
    w4 = lecb.W4Weights(ref_tiles(q).to(DEV), ref_scales(s, n, k, 64).to(DEV), n, k, 64)
    x = torch.randn(m, k, generator=g).to(dtype)
    ref = lecb.matvec_w4(x.to(DEV), w4, out_dtype=F32)
    x[0, 9], x[2, k - 1] = math.inf, -math.inf
    x[1, 200] = math.nan
    y = lecb.matvec_w4(x.to(DEV), w4, out_dtype=F32)
    assert torch.equal(y[3:], ref[3:])
    assert bool(y[1].isnan().all())
    for token, column, sign in ((0, 9, 1.0), (2, k - 1, -1.0)):
        want = q[:, column].to(F32) * (sign * math.inf)
        got = y[token].cpu()
        assert bool(((got == want) | (got.isnan() & want.isnan())).all())


@pytest.mark.parametrize("m,n,k", [(3, 80, 384), (12, 80, 401), (40, 80, 384), (300, 16400, 384)])
@pytest.mark.parametrize("dtype,least", [(BF16, 2.0 ** -133), (F16, 2.0 ** -24)], ids=str)
@pytest.mark.parametrize("group", [32, 128])
def test_smallest_numbers(m, n, k, dtype, least, group):
    """Tokens of a few times the type's smallest number: every sum is a whole number of those, below 2^24, so exact."""
    g = gen(8)
    q = torch.randint(-8, 8, (n, k), generator=g)
    s = torch.full((n, -(-k // group)), 1.0)
    w4 = lecb.W4Weights(ref_tiles(q).to(DEV), ref_scales(s, n, k, group).to(DEV), n, k, group)
    whole = torch.randint(-127, 128, (m, k), generator=g)
    x = (whole.to(F64) * least).to(dtype)
    assert torch.equal(x.to(F64), whole.to(F64) * least)
    rows = torch.cat([torch.arange(40), torch.arange(n - 40, n)])
    y = lecb.matvec_w4(x.to(DEV), w4, out_dtype=F32)[:, rows.to(DEV)].cpu().to(F64)
    assert torch.equal(y, (whole.to(F64) @ q[rows].t().to(F64)) * least)


@pytest.mark.parametrize("m", [2, 12, 40])
@pytest.mark.parametrize("dtype,scale", [(BF16, 2.0 ** 117), (F16, 2.0 ** 125)], ids=str)
def test_largest_scales(m, dtype, scale):
    """Scales up to the stated limit: powers of two change nothing but the exponent."""
    n, k, group = 48, 256, 64
    g = gen(9)
    q = torch.randint(-8, 8, (n, k), generator=g)
    x = (torch.randint(-64, 65, (m, k), generator=g).to(F32) * 2.0 ** -20).to(dtype)
    w4 = lecb.W4Weights(ref_tiles(q).to(DEV), ref_scales(torch.full((n, k // group), scale), n, k, group).to(DEV), n, k, group)
    y = lecb.matvec_w4(x.to(DEV), w4, out_dtype=F32).cpu().to(F64)
    assert torch.equal(y, (x.to(F64) @ q.t().to(F64)) * scale)
