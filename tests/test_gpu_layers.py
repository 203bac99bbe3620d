"""Operators of quantised layers on the GPU against plain implementations in 64 bits.

u = 2^-24 is half a step of fp32 relative to the value; eps(T) / 2 that of T.
Codes, scales and values of 4-bit weights are defined exactly and compared so;
the tolerances of the other two stand beside their tests."""

import math

import pytest
import torch

import lossless_entropy_coding_byte_amd as lecb

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F64 = torch.float64
BF16, F16, F32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def same(a, b):
    """Equal bit for bit up to the NaN's own bits and the sign of zero."""
    a, b = a.cpu(), b.cpu()
    return a.shape == b.shape and a.dtype == b.dtype and bool(((a == b) | (a.isnan() & b.isnan())).all())


# ---------------------------------------------------------------------------- 4-bit weights

def ref_tiles(q):
    """Codes [n, k] (int64, CPU) in tile order, one word at a time from the layout's definition."""
    n, k = q.shape
    nt, kt = -(-n // 16), -(-k // 128)
    full = torch.zeros(nt * 16, kt * 128, dtype=torch.int64)
    full[:n, :k] = q & 15
    words = torch.zeros(nt * 16, kt * 16, dtype=torch.int64)
    for i in range(8):
        words |= full[:, i::8] << (4 * i)
    out = torch.zeros(nt, kt, 4, 16, 4, dtype=torch.int64)
    for c in range(4):
        for d in range(4):
            out[:, :, c, :, d] = words.view(nt, 16, kt, 16)[:, :, :, 4 * d + c].permute(0, 2, 1)
    b = torch.stack([(out >> (8 * j)) & 255 for j in range(4)], -1)
    return b.to(torch.uint8).view(nt, kt, 1024)


def ref_scales(s, n, k, group):
    """Scales [n, ceil(k / group)] in their stored order."""
    nt, per = -(-n // 16), -(-k // 128) * (128 // group)
    full = torch.zeros(nt * 16, per, dtype=s.dtype)
    full[:n, : s.shape[1]] = s
    return full.view(nt, 16, per).permute(0, 2, 1).contiguous()


def ref_quantize(w, group, scale_dtype):
    """(codes int64, scales [n, groups], values float64) of W on the CPU."""
    n, k = w.shape
    groups = -(-k // group)
    full = torch.zeros(n, groups * group, dtype=F64)
    full[:, :k] = w.to(F64)
    full = full.view(n, groups, group)
    amax = full.abs().amax(2)
    s32 = amax.to(F32) / torch.tensor(7.0, dtype=F32)
    s = s32.to(scale_dtype)
    bad = ~torch.isfinite(full).all(2) | ~torch.isfinite(s.to(F32))
    s = torch.where(bad, torch.tensor(math.nan, dtype=scale_dtype), s)
    d = s.to(F64)
    ok = (d > 0)[:, :, None]
    q = torch.where(ok, torch.nan_to_num(full / torch.where(d > 0, d, 1.0)[:, :, None]).round().clamp(-7, 7), 0.0)
    v = (q * d[:, :, None]).view(n, groups * group)[:, :k]
    return q.view(n, groups * group)[:, :k].to(torch.int64), s, v


SHAPES = [(1, 1), (1, 7), (3, 8), (16, 128), (17, 129), (15, 127), (5, 33), (33, 96), (100, 1000), (64, 4096), (2, 2049)]


@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("group,sdt", [(32, BF16), (64, F32), (128, BF16)], ids=str)
def test_quantize_w4(n, k, dtype, group, sdt):
    w = (torch.randn(n, k, generator=gen(n * 7 + k)) * 0.02).to(dtype)
    q, s, v = ref_quantize(w, group, sdt)
    w4 = lecb.quantize_w4(w.to(DEV), group=group, scale_dtype=sdt)
    assert torch.equal(w4.tiles.cpu(), ref_tiles(q))
    assert same(w4.scales, ref_scales(s, n, k, group))
    for out in (F32, BF16, F16):
        # q * s is one fp32 product, rounded once more to 16 bits
        assert same(lecb.dequantize_w4(w4, out), (q.to(F32) * s.to(F32).repeat_interleave(group, 1)[:, :k]).to(out))
    packed = lecb.untile_w4(w4.tiles, n, k)
    lo, hi = (q & 15), torch.zeros_like(q)
    hi[:, :-1] = q[:, 1:] & 15
    assert torch.equal(packed.cpu(), (lo[:, ::2] | (hi[:, ::2] << 4)).to(torch.uint8))
    assert torch.equal(lecb.tile_w4(packed, n, k), w4.tiles)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("sdt", [F32, BF16], ids=str)
def test_quantize_w4_extremes(dtype, sdt):
    """Zero rows, infinities and NaN, the type's smallest and largest values, half steps."""
    f = torch.finfo(dtype)
    g = gen(5)
    rows = [torch.zeros(128), torch.full((128,), f.max), torch.full((128,), f.tiny), torch.full((128,), f.smallest_normal / 8),
            torch.linspace(-f.max, f.max, 128, dtype=F64), torch.linspace(-1, 1, 128) * f.tiny * 7,
            torch.cat([torch.tensor([7.0]), torch.arange(127) % 14 / 2 - 3.25]), torch.cat([torch.tensor([7.0]), torch.arange(127) % 15 - 6.5])]
    for bad in (math.inf, -math.inf, math.nan):
        r = torch.randn(128, generator=g)
        r[77] = bad
        rows.append(r)
    rows += [torch.randn(128, generator=g) * 10.0 ** e for e in (-44, -40, -30, -20, -8, -5, 3, 4, 20, 37)]
    w = torch.stack([r.to(F64) for r in rows]).to(dtype)
    for group in (32, 64, 128):
        q, s, v = ref_quantize(w, group, sdt)
        w4 = lecb.quantize_w4(w.to(DEV), group=group, scale_dtype=sdt)
        assert torch.equal(w4.tiles.cpu(), ref_tiles(q))
        assert same(w4.scales, ref_scales(s, w.shape[0], 128, group))


def test_quantize_w4_ties_of_fp32():
    """fp32 weights next to half a step, where a quotient in 32 bits would land on the wrong side."""
    g = gen(9)
    s = torch.rand(4096, 1, generator=g) + 0.5
    half = (torch.randint(-7, 7, (4096, 127), generator=g) + 0.5) * s
    half = torch.nextafter(half, half + torch.randint(-1, 2, half.shape, generator=g))
    w = torch.cat([s * 7, half], 1).to(F32)
    q, sc, _ = ref_quantize(w, 128, F32)
    w4 = lecb.quantize_w4(w.to(DEV), group=128, scale_dtype=F32)
    assert torch.equal(w4.tiles.cpu(), ref_tiles(q)) and same(w4.scales, ref_scales(sc, 4096, 128, 128))


def test_w4_strides_and_alignment():
    base = torch.randn(40, 700, generator=gen(3)).to(BF16)
    dev = base.to(DEV)
    for c0, k in ((0, 256), (1, 256), (8, 264), (3, 129), (16, 600)):
        a = lecb.quantize_w4(dev[:, c0 : c0 + k])
        b = lecb.quantize_w4(dev[:, c0 : c0 + k].contiguous())
        assert torch.equal(a.tiles, b.tiles) and torch.equal(a.scales, b.scales)
        out = torch.full((40, 704), 7.0, dtype=BF16, device=DEV)
        lecb.lecb_dequantize_w4(a.tiles, a.scales, a.group, 40, k, out[:, c0:], 704)
        assert torch.equal(out[:, c0 : c0 + k], lecb.dequantize_w4(a))
        assert bool((out[:, :c0] == 7).all()) and bool((out[:, c0 + k :] == 7).all())
    # rows of packed codes at an odd address
    rows = torch.randint(0, 256, (33 * 64 + 1,), dtype=torch.uint8, generator=gen(4)).to(DEV)
    odd, even = rows[1:].view(33, 64), rows[1:].clone().view(33, 64)
    t = lecb.tile_w4(even, 33, 128)
    assert torch.equal(lecb.tile_w4(odd, 33, 128), t)
    back = torch.zeros(33 * 64 + 1, dtype=torch.uint8, device=DEV)
    lecb.lecb_untile_w4(t, 33, 128, back[1:])
    assert torch.equal(back[1:].view(33, 64), even)


# ---------------------------------------------------------------------------- 8-bit norm

def ref_norm(x, res, weight, eps):
    """(h fp32 as added, y float64) on the CPU."""
    h = x.to(F32) + res.to(F32) if res is not None else x.to(F32)
    hd = h.to(F64)
    return h, hd * weight.to(F64) / (hd.square().mean(-1, keepdim=True) + eps).sqrt()


def check_norm(q, scale, h, x, res, weight, eps, static=None):
    """scale: the sum of squares has relative error below 64 u -- at most 32
    terms a lane, one rounding each, then the lanes' and waves' sums -- which
    the root halves; product, root and quotient add 6 u.  Codes: h weight, the
    factor and their product are off by 8 u of at most 127 steps together (the
    factor of a fixed scale carries the root's 32 u too), so q lies
    within 1/2 + 127 * 8 u (40 u) of y / scale."""
    rh, y = ref_norm(x, res, weight, eps)
    assert same(h, rh.to(x.dtype))
    q, s = q.cpu().to(F64), scale.cpu().to(F64)
    rs = y.abs().amax(-1) / 127 if static is None else torch.full(x.shape[:-1], static, dtype=F64)
    assert bool(((s - rs).abs() <= 40 * U * rs).all())
    steps = torch.where(rs[..., None] > 0, y / torch.where(rs > 0, rs, 1.0)[..., None], 0.0).clamp(-127, 127)
    off = (q - steps).abs().max().item()
    assert off <= 0.5 + 127 * (8 if static is None else 40) * U, off
    assert q.abs().max() <= 127


NORM_SHAPES = [(1, 1), (1, 7), (3, 8), (5, 64), (2, 513), (4, 1367), (1, 4096), (33, 2048), (7, 2056), (3, 8192), (2, 8200),
               (2, 16384), (1, 32768), (2, 32767), (3000, 256)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("wdt", [F32, BF16, F16], ids=str)
def test_rmsnorm_q8(rows, cols, dtype, wdt):
    g = gen(rows * 3 + cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).to(dtype)
    weight = (1 + 0.3 * torch.randn(cols, generator=g)).to(wdt)
    for res in (None, torch.randn(rows, cols, generator=g).to(dtype)):
        q, s, h = lecb.rmsnorm_q8(x.to(DEV), weight.to(DEV), residual=None if res is None else res.to(DEV), eps=1e-5)
        check_norm(q, s, h, x, res, weight, 1e-5)
        for out in (F32, BF16, F16):
            v = lecb.dequantize_q8(q, s, out)
            assert same(v, (q.cpu().to(F32) * s.cpu()[:, None]).to(out))


@pytest.mark.parametrize("cols", [64, 1000, 1001])
def test_rmsnorm_q8_fixed_scale(cols):
    g = gen(cols)
    x, weight = torch.randn(9, cols, generator=g), 1 + 0.1 * torch.randn(cols, generator=g)
    x[3] = 0
    for value in (0.02, 0.01, 3.0):     # covers the row, saturates, coarse
        scale = torch.tensor([value], device=DEV)
        q, s, h = lecb.rmsnorm_q8(x.to(DEV), weight.to(DEV), scale=scale)
        assert s is scale
        check_norm(q, s.expand(9), h, x, None, weight, 1e-6, static=float(torch.tensor(value)))
        assert same(lecb.dequantize_q8(q, s, F32), q.cpu().to(F32) * torch.tensor(value))
    for value in (0.0, -1.0, math.nan):
        q, _, _ = lecb.rmsnorm_q8(x.to(DEV), weight.to(DEV), scale=torch.tensor([value], device=DEV))
        assert not q.any()


@pytest.mark.parametrize("cols", [96, 97, 3000])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_rmsnorm_q8_rows_without_a_norm(cols, dtype):
    """Zero rows, rows with an infinity or NaN, tiny and huge rows; the others are not touched by them."""
    g = gen(cols)
    x = torch.randn(10, cols, generator=g)
    x[1] = 0
    x[2, 5], x[3, cols - 1], x[4, 0] = math.inf, -math.inf, math.nan
    x[5] *= 1e-20
    x[6] *= 1e-38
    x[7] *= 1e15
    x = x.to(dtype)
    weight = 1 + 0.1 * torch.randn(cols, generator=g)
    q, s, h = lecb.rmsnorm_q8(x.to(DEV), weight.to(DEV), eps=1e-6)
    assert s[1].item() == 0 and not q[1].any()
    assert s[2:5].isnan().all() and not q[2:5].any()
    assert lecb.dequantize_q8(q, s)[2:5].isnan().all()
    keep = [0, 1, 5, 6, 7, 8, 9]
    check_norm(q[keep], s[keep], h[keep], x[keep], None, weight, 1e-6)
    bad = weight.clone()
    bad[2] = math.nan
    q, s, _ = lecb.rmsnorm_q8(x.to(DEV), bad.to(DEV))
    assert s.isnan().all() and not q.any()


def test_rmsnorm_q8_strides_and_in_place():
    g = gen(1)
    for c0, cols in ((0, 512), (8, 1024), (3, 513), (5, 8)):
        base, rbase = torch.randn(20, 1100, generator=g).to(BF16), torch.randn(20, 1048, generator=g).to(BF16)
        x, r, w = base.to(DEV)[:, c0 : c0 + cols], rbase.to(DEV)[:, :cols], (1 + torch.rand(cols, generator=g)).to(BF16).to(DEV)
        ref = lecb.rmsnorm_q8(x.contiguous(), w, residual=r.contiguous())
        for mine in (x, r):
            xx, rr = x.clone() if mine is x else x, r.clone() if mine is r else r
            out = xx if mine is x else rr
            got = lecb.rmsnorm_q8(xx, w, residual=rr, out_h=out)
            assert got[2] is out and all(torch.equal(a, b) for a, b in zip(got, ref))
        got = lecb.rmsnorm_q8(x.view(4, 5, cols), w, residual=r.view(4, 5, cols))
        assert got[0].shape == (4, 5, cols) and got[1].shape == (4, 5) and torch.equal(got[0].view(20, cols), ref[0])
    q, s, h = lecb.rmsnorm_q8(torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV))
    assert q.shape == (0, 64) and s.shape == (0,)


# ---------------------------------------------------------------------------- products

def weights(n, k, group, sdt, seed, low=-8):
    g = gen(seed)
    q = torch.randint(low, 8, (n, k), generator=g)
    s = (0.004 + 0.008 * torch.rand(n, -(-k // group), generator=g)).to(sdt)
    w4 = lecb.W4Weights(ref_tiles(q).to(DEV), ref_scales(s, n, k, group).to(DEV), n, k, group)
    return q, s, w4


def check_matvec(y, x, xs, q, s, group):
    """int8: group sums are whole numbers below 2^24, exact in fp32; then one
    rounding per group, wave sum and factor of at most the sum of magnitudes.
    16-bit x: each group also sums 2 * group products of at most |x| (24 + 32)
    in fp32, every addition rounded (2 u: the matrix unit may cut off)."""
    n, k = q.shape
    groups = s.shape[1]
    w = q.to(F64) * s.to(F64).repeat_interleave(group, 1)[:, :k]
    f = torch.ones(x.shape[0], 1, dtype=F64) if xs is None else xs.cpu().to(F64).reshape(-1, 1)
    xd = x.cpu().to(F64)
    ref = (xd @ w.t()) * f
    mag = (xd.abs() @ w.abs().t()) * f
    tol = (groups + 24) * U * mag
    if x.dtype != I8:
        ws = s.to(F64).repeat_interleave(group, 1)[:, :k]
        tol = tol + 2 * U * 2 * group * 56 * (xd.abs() @ ws.t())
    tol = tol + (torch.finfo(y.dtype).eps / 2) * (ref.abs() + tol)
    got = y.cpu().to(F64)
    assert got.shape == ref.shape and bool(torch.isfinite(got).all())
    worst = ((got - ref).abs() / tol.clamp_min(1e-300)).max().item()
    assert worst <= 1, worst
    if x.dtype != I8 and y.dtype == F32 and k >= 32:
        # and by the norm: 2 group / 32 roundings a group at up to 6 times the sums' size, eightfold
        rel = ((got - ref).norm() / ref.norm()).item()
        assert rel <= 8 * U * 6 * math.sqrt(2 * group / 32), rel


def tokens(m, k, dtype, seed):
    g = gen(seed)
    if dtype == I8:
        return torch.randint(-127, 128, (m, k), generator=g).to(I8), (0.01 + torch.rand(m, generator=g) * 0.02)
    return torch.randn(m, k, generator=g).to(dtype), None


MV_SHAPES = [(1, 1, 1), (1, 16, 128), (2, 15, 7), (3, 17, 129), (5, 1003, 1111), (15, 33, 31), (16, 64, 256), (17, 100, 33),
             (1, 4096, 4096), (1, 64, 28672), (32, 256, 1024), (33, 48, 640), (64, 130, 1000), (65, 144, 2048),
             (130, 272, 384), (257, 520, 1160), (512, 1024, 1024)]


@pytest.mark.parametrize("m,n,k", MV_SHAPES)
@pytest.mark.parametrize("dtype", [I8, BF16, F16], ids=str)
@pytest.mark.parametrize("group,sdt", [(32, F32), (64, BF16), (128, BF16), (128, F32)], ids=str)
def test_matvec_w4(m, n, k, dtype, group, sdt):
    q, s, w4 = weights(n, k, group, sdt, m + n + k)
    x, xs = tokens(m, k, dtype, m * k)
    xd, xsd = x.to(DEV), None if xs is None else xs.to(DEV)
    for out in (F32, BF16, F16):
        y = lecb.matvec_w4(xd, w4, x_scale=xsd, out_dtype=out)
        check_matvec(y, x, xs, q, s, group)
    assert lecb.matvec_w4(xd, w4, x_scale=xsd).dtype == (BF16 if dtype == I8 else dtype)


def test_matvec_w4_largest_whole_numbers():
    """The largest group sums of int8 x: +-127 against -8, every group."""
    for group in (32, 64, 128):
        q = torch.full((32, 4096), -8)
        s = torch.ones(32, 4096 // group)
        w4 = lecb.W4Weights(ref_tiles(q).to(DEV), ref_scales(s, 32, 4096, group).to(DEV), 32, 4096, group)
        for v in (127, -127, -128):
            x = torch.full((3, 4096), v, dtype=I8, device=DEV)
            y = lecb.matvec_w4(x, w4, out_dtype=F32)
            assert bool((y == -8.0 * v * 4096).all())


@pytest.mark.parametrize("dtype", [I8, BF16], ids=str)
@pytest.mark.parametrize("m", [1, 4, 40, 200])
def test_matvec_w4_strides_scales_rows(dtype, m):
    n, k, group = 80, 512, 64
    q, s, w4 = weights(n, k, group, BF16, 11)
    big, xs = tokens(m, k + 77, dtype, 12)
    bd = big.to(DEV)
    for c0 in (0, 1, 8, 16):
        x = bd[:, c0 : c0 + k]
        a = lecb.matvec_w4(x, w4, out_dtype=F32)
        check_matvec(a, big[:, c0 : c0 + k], None, q, s, group)
        # the tokens' address and stride choose loads, not values
        assert torch.equal(a, lecb.matvec_w4(x.contiguous(), w4, out_dtype=F32))
    if dtype == I8:
        one = torch.tensor([0.03], device=DEV)
        check_matvec(lecb.matvec_w4(bd[:, :k], w4, x_scale=one, out_dtype=F32), big[:, :k], one.cpu().expand(m), q, s, group)
    y = torch.full((m, n + 3), 5.0, device=DEV)
    x = bd[:, :k].contiguous()
    lecb.lecb_matvec_w4(x, k, None, 0, m, w4.tiles, w4.scales, group, n, k, y, n + 3,
                        ws=torch.empty(max(16, lecb.lecb_matvec_w4_workspace_bytes(m, n, k)), dtype=torch.uint8, device=DEV))
    assert torch.equal(y[:, :n], lecb.matvec_w4(x, w4, out_dtype=F32)) and bool((y[:, n:] == 5).all())
    assert lecb.matvec_w4(x.view(m, 1, k), w4).shape == (m, 1, n)
    assert lecb.matvec_w4(x[:0], w4).shape == (0, n)


def test_matvec_w4_a_bad_token_stays_alone():
    q, s, w4 = weights(48, 384, 128, BF16, 2)
    for m in (3, 20, 70):
        x = torch.randn(m, 384, generator=gen(m)).to(BF16).to(DEV)
        ref = lecb.matvec_w4(x, w4)
        x[1, 7], x[2, 300] = math.nan, math.inf
        y = lecb.matvec_w4(x, w4)
        keep = [0] + list(range(3, m))
        assert torch.equal(y[keep], ref[keep])
        assert not torch.isfinite(y[1:3].float()).any()


def test_matvec_w4_same_twice():
    for m, n, k in ((1, 64, 28672), (7, 512, 8192), (100, 512, 8192)):
        q, s, w4 = weights(n, k, 128, BF16, 3)
        x, xs = tokens(m, k, BF16, 4)
        a = lecb.matvec_w4(x.to(DEV), w4, out_dtype=F32)
        for _ in range(5):
            assert torch.equal(a, lecb.matvec_w4(x.to(DEV), w4, out_dtype=F32))


# ---------------------------------------------------------------------------- streams, graphs, long tensors

def _chain(x, res, weight, w4):
    q, s, h = lecb.rmsnorm_q8(x, weight, residual=res)
    return h, q, s, lecb.matvec_w4(q, w4, x_scale=s), lecb.matvec_w4(h, w4)


def test_other_stream_and_graph():
    """The chain on a stream of its own, and captured: every replay equals the eager result on the same inputs."""
    w = torch.randn(200, 512, generator=gen(1)).to(BF16).to(DEV)
    w4 = lecb.quantize_w4(w)
    weight = torch.ones(512, dtype=BF16, device=DEV)
    x, res = torch.empty(20, 512, dtype=BF16, device=DEV), torch.empty(20, 512, dtype=BF16, device=DEV)
    side = torch.cuda.Stream()

    def fill(seed):
        x.copy_(torch.randn(20, 512, generator=gen(seed)))
        res.copy_(torch.randn(20, 512, generator=gen(seed + 100)))

    fill(1)
    ref = _chain(x, res, weight, w4)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _chain(x, res, weight, w4)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _chain(x, res, weight, w4)
        again = lecb.quantize_w4(w)
        values = lecb.dequantize_w4(again)
    for seed in (2, 3, 4, 5):
        fill(seed)
        g.replay()
        torch.cuda.synchronize()
        ref = _chain(x, res, weight, w4)
        assert all(torch.equal(a, b) for a, b in zip(ref, out)), seed
        assert torch.equal(values, lecb.dequantize_w4(w4)), seed


def test_offsets_beyond_32_bits():
    """Tensors of more than 2^31 elements and tiles of more than 2^32 bytes: the ends are right."""
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("40 GiB of GPU memory are needed")
    rows, cols = 70001, 32768
    x = torch.zeros(rows, cols, dtype=BF16, device=DEV)
    tail = torch.randn(3, cols, generator=gen(8)).to(BF16)
    x[-3:] = tail.to(DEV)
    w = torch.ones(cols, device=DEV)
    q, s, h = lecb.rmsnorm_q8(x, w)
    check_norm(q[-3:], s[-3:], h[-3:], tail, None, w.cpu(), 1e-6)
    assert not s[:-3].any()
    v = lecb.dequantize_q8(q, s)
    assert same(v[-3:], (q[-3:].cpu().to(F32) * s[-3:].cpu()[:, None]).to(BF16))
    del q, v, h
    w4 = lecb.quantize_w4(x)
    qr, sr, _ = ref_quantize(tail, 128, BF16)
    back = lecb.dequantize_w4(w4)
    assert same(back[-3:], (qr.to(F32) * sr.to(F32).repeat_interleave(128, 1)).to(BF16))
    assert not back[:100].any()
    packed = lecb.untile_w4(w4.tiles, rows, cols)
    assert torch.equal(lecb.tile_w4(packed, rows, cols), w4.tiles)
    del back, packed, x, w4
    n, k = 270000, 32768
    tiles = torch.randint(0, 256, (-(-n // 16) * (k // 128) * 1024,), dtype=torch.uint8, device=DEV)
    assert tiles.numel() > 1 << 32
    scales = torch.ones(-(-n // 16) * (k // 128) * 16, dtype=BF16, device=DEV)
    for m, dt in ((1, I8), (3, BF16), (70, I8)):
        xx, _ = tokens(m, k, dt, m)
        y = lecb.matvec_w4(xx.to(DEV), lecb.W4Weights(tiles, scales, n, k), out_dtype=F32)
        end = lecb.W4Weights(tiles[-2 * (k // 128) * 1024 :].clone(), scales[-2 * (k // 128) * 16 :].clone(), 32, k)
        qe = lecb.dequantize_w4(end, F32).cpu().to(torch.int64)
        check_matvec(y[:, -32:], xx, None, qe, torch.ones(32, k // 128), 128)


def test_refusals_on_the_gpu():
    q, s, w4 = weights(16, 128, 128, BF16, 1)
    x = torch.zeros(4, 128, dtype=BF16, device=DEV)
    host = x.cpu()
    for bad in (lambda: lecb.matvec_w4(host, w4), lambda: lecb.matvec_w4(x.t(), w4), lambda: lecb.matvec_w4(x.float(), w4),
                lambda: lecb.matvec_w4(x.as_strided((4, 128), (64, 1)), w4),
                lambda: lecb.matvec_w4(x[:, ::2], w4), lambda: lecb.rmsnorm_q8(x, torch.ones(128)),
                lambda: lecb.rmsnorm_q8(x, x[0], residual=x[:2]), lambda: lecb.rmsnorm_q8(x, x[0], residual=x.float()),
                lambda: lecb.rmsnorm_q8(x, x[0], out_h=x), lambda: lecb.rmsnorm_q8(x, x[0], scale=torch.ones(4, device=DEV)),
                lambda: lecb.quantize_w4(x[:, ::2]), lambda: lecb.dequantize_q8(x.to(I8)[:, ::2], torch.ones(4, device=DEV))):
        with pytest.raises(ValueError):
            bad()
            pytest.fail("taken")
    with pytest.raises(lecb.LecbError) as e:
        lecb.rmsnorm_q8(x, x[0], eps=0.0)
    assert e.value.status == lecb.LECB_ERR_INVALID_ARG
    with pytest.raises(lecb.LecbError) as e:
        lecb.lecb_matvec_w4(x, 64, None, 0, 4, w4.tiles, w4.scales, 128, 16, 128, torch.empty(4, 16, device=DEV), 16)
    assert e.value.status == lecb.LECB_ERR_INVALID_ARG
