"""The operators of quantised layers, as cases to be timed and compared.

Three operators that stand next to the codec, on the tensors it stores:

* ``quantize_w4``  float weights to 4-bit codes with one scale per row and
  group of columns, in the tile order the products read, and back to values;
* ``rmsnorm_q8``   the residual's addition, the root-mean-square norm and the
  quantisation of its output to 8 bits with one scale per row, and the values
  those 8 bits stand for;
* ``matvec_w4``    products of one or many tokens with 4-bit weights.

``own`` chooses who computes them: false, elementary torch operations; true,
the framework.

Formulas (i row, j column, groups of ``group`` columns):

* ``quantize_w4``: s = max|w| / 7 over the row's group, rounded to the scales'
  type; q = w / s rounded to the nearest whole number (ties to even) and kept
  in -7..7, 0 where s = 0; the weight that q stands for is q * s;
* ``rmsnorm_q8``: h = x + residual; y_j = h_j * weight_j / sqrt(mean(h^2) + eps);
  scale = max|y| / 127; q = y / scale rounded to nearest; h is returned in x's
  type, q as the values q * scale;
* ``matvec_w4``: y[i, n] = sum_k x[i, k] q[n, k] s[n, k // group], times the
  row's scale where x is held in 8 bits.

Tile order of 4-bit weights [n, k], both padded with zeros (rows to 16, columns
to 128): eight codes of neighbouring columns make a 32-bit word, the first in
its lowest four bits; word (r, d, c) of a tile, for columns 32 d + 8 c and
following of row r, stands at place (c, r, d) of the tile's 4 x 16 x 4 words;
tiles follow one another along k, then along n.  Scales: [n / 16, groups, 16].
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8}
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a decode step enters a layer
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16", "residual": True},
        # a ragged little batch, rows that no vector width divides, no residual
        {"name": "norm_odd", "op": "norm", "rows": 37, "cols": 1367, "type": "fp16", "residual": False},
        # the activations [8, 2048, 2048] of the int8 workloads, before their quantisation
        {"name": "norm_acts", "op": "norm", "rows": 16384, "cols": 2048, "type": "bf16", "residual": True},
        # a residual stream kept in 32 bits
        {"name": "norm_wide", "op": "norm", "rows": 4096, "cols": 8192, "type": "fp32", "residual": True},
        # a small odd projection, quantised on its own
        {"name": "quant_odd", "op": "quant", "n": 333, "k": 1001, "type": "fp16", "group": 32, "scales": "fp32"},
        # the 64 Mi bf16 weights of the weight workload
        {"name": "quant_bf16", "op": "quant", "n": 8192, "k": 8192, "type": "bf16", "group": 128, "scales": "bf16"},
        # the 64 Mi fp32 weights, as a trainer holds them
        {"name": "quant_fp32", "op": "quant", "n": 8192, "k": 8192, "type": "fp32", "group": 64, "scales": "bf16"},
        # one token against a square projection: the latency of a decode step
        {"name": "mv_token_q8", "op": "mv", "m": 1, "n": 4096, "k": 4096, "type": "int8", "out": "bf16",
         "group": 128, "scales": "bf16"},
        # one token against the widest matrix of a large layer: the weights' bytes count
        {"name": "mv_token_wide", "op": "mv", "m": 1, "n": 28672, "k": 8192, "type": "bf16", "out": "bf16",
         "group": 128, "scales": "bf16"},
        # odd sizes, the smallest groups, scales and sums handed on in 32 bits
        {"name": "mv_odd", "op": "mv", "m": 5, "n": 1003, "k": 1111, "type": "fp16", "out": "fp32",
         "group": 32, "scales": "fp32"},
        # a decode step of 32 requests
        {"name": "mv_batch_q8", "op": "mv", "m": 32, "n": 8192, "k": 8192, "type": "int8", "out": "bf16",
         "group": 128, "scales": "bf16"},
        # a chunk of a prompt
        {"name": "mv_chunk", "op": "mv", "m": 512, "n": 8192, "k": 8192, "type": "bf16", "out": "bf16",
         "group": 64, "scales": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _size(rng, lo, hi):
    """A size of [lo, hi]: of three, one any number, one a multiple of 8, one of 128 where that fits."""
    v, step = _log(rng, lo, hi), rng.choice((1, 8, 128))
    return max(lo, v - v % step) if v >= step else v


def draw(rng):
    op = rng.choice(("norm", "quant", "mv", "mv"))
    if op == "norm":
        cols = _size(rng, 64, 16384)
        return {"op": op, "rows": _log(rng, 1, min(16384, (1 << 25) // cols)), "cols": cols,
                "type": rng.choice(("bf16", "fp16", "fp32")), "residual": rng.random() < 0.7}
    group = rng.choice((32, 64, 128))
    scales = rng.choice(("bf16", "bf16", "fp32"))
    if op == "quant":
        k = _size(rng, 64, 28672)
        return {"op": op, "n": _size(rng, 16, min(28672, (1 << 26) // k)), "k": k,
                "type": rng.choice(("bf16", "fp16", "fp32")), "group": group, "scales": scales}
    m = rng.choice((1, 1, _log(rng, 2, 64), _log(rng, 2, 512)))
    k = _size(rng, 128, 28672)
    n = _size(rng, 64, max(64, min(28672, (1 << 27) // k, (512 << 26) // (m * k))))
    return {"op": op, "m": m, "n": n, "k": k, "type": rng.choice(("int8", "int8", "bf16", "fp16")),
            "out": rng.choice(("bf16", "bf16", "fp32")), "group": group, "scales": scales}


def work(case):
    c = case
    if c["op"] == "norm":
        e, b = c["rows"] * c["cols"], _bytes(c["type"])
        # x, the residual and h, the weight; the values leave in 16 bits
        return {"bytes": e * (b * (3 if c["residual"] else 2) + 2) + c["cols"] * b + 4 * c["rows"], "flops": 8 * e}
    nk = c["n"] * c["k"]
    scales = c["n"] * -(-c["k"] // c["group"]) * _bytes(c["scales"])
    if c["op"] == "quant":
        # the weights in, their values out in 16 bits, the scales
        return {"bytes": nk * (_bytes(c["type"]) + 2) + scales, "flops": 4 * nk}
    x = c["m"] * c["k"] * _bytes(c["type"]) + (4 * c["m"] if c["type"] == "int8" else 0)
    return {"bytes": nk / 2 + scales + x + c["m"] * c["n"] * _bytes(c["out"]), "flops": 2 * c["m"] * nk}


def _bytes(t):
    return {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1}[t]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] == "norm":
        # a residual stream: a few channels far larger than the others, rows of different size
        rows, cols, t = c["rows"], c["cols"], TYPES[c["type"]]
        channel = torch.where(torch.rand(cols, device=DEV, generator=g) < 0.003, 8.0, 1.0)
        size = torch.exp(0.5 * torch.randn(rows, 1, device=DEV, generator=g))
        x = torch.randn(rows, cols, device=DEV, generator=g).mul_(channel).mul_(size).to(t)
        res = torch.randn(rows, cols, device=DEV, generator=g).mul_(size).to(t) if c["residual"] else None
        weight = (1 + 0.2 * torch.randn(cols, device=DEV, generator=g)).to(t)
        return {"case": c, "x": x, "residual": res, "weight": weight}
    if c["op"] == "quant":
        # trained weights: about normal, rows of different size, some groups with an outlier
        w = torch.randn(c["n"], c["k"], device=DEV, generator=g)
        w.mul_(0.02 * torch.exp(0.3 * torch.randn(c["n"], 1, device=DEV, generator=g)))
        w.mul_(torch.where(torch.rand(1, c["k"], device=DEV, generator=g) < 0.002, 4.0, 1.0))
        return {"case": c, "w": w.to(TYPES[c["type"]])}
    n, k, m = c["n"], c["k"], c["m"]
    nt, kt = -(-n // 16), -(-k // 128)
    q = torch.randn(n, k, device=DEV, generator=g).mul_(2.6).round_().clamp_(-7, 7).to(torch.int8)
    q = torch.nn.functional.pad(q, (0, kt * 128 - k, 0, nt * 16 - n)).bitwise_and_(15).view(torch.uint8)
    tiles = q[:, 0::2] | (q[:, 1::2] << 4)
    tiles = tiles.view(torch.int32).view(nt, 16, kt, 4, 4).permute(0, 2, 4, 1, 3).contiguous().view(torch.uint8)
    groups, per = -(-k // c["group"]), kt * 128 // c["group"]
    s = torch.zeros(nt * 16, per, device=DEV)
    s[:n, :groups] = 0.004 + 0.008 * torch.rand(n, groups, device=DEV, generator=g)
    scales = s.view(nt, 16, per).permute(0, 2, 1).contiguous().to(TYPES[c["scales"]])
    x = torch.randn(m, k, device=DEV, generator=g)
    x.mul_(torch.where(torch.rand(1, k, device=DEV, generator=g) < 0.003, 8.0, 1.0))
    xs = None
    if c["type"] == "int8":
        xs = x.abs().amax(1) / 127
        x = (x / xs[:, None]).round_()
    return {"case": c, "x": x.to(TYPES[c["type"]]), "x_scale": xs, "tiles": tiles.view(nt, kt, 1024), "scales": scales}


# ---------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"norm": _norm, "quant": _quant, "mv": _mv}[c["op"]](c, state)


def _values_type(c):
    return TYPES[c["type"] if c["type"] != "fp32" else "bf16"]


def _own(c, s):
    import lossless_entropy_coding_byte_amd as lecb

    if c["op"] == "norm":
        q, scale, h = lecb.rmsnorm_q8(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        return {"h": h, "values": lecb.dequantize_q8(q, scale, _values_type(c)), "scale": scale}
    if c["op"] == "quant":
        w4 = lecb.quantize_w4(s["w"], group=c["group"], scale_dtype=TYPES[c["scales"]])
        return {"values": lecb.dequantize_w4(w4, _values_type(c)), "scales": w4.scales}
    w4 = lecb.W4Weights(s["tiles"], s["scales"], c["n"], c["k"], c["group"])
    return lecb.matvec_w4(s["x"], w4, x_scale=s["x_scale"], out_dtype=TYPES[c["out"]])


def _norm(c, s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    scale = y.abs().amax(1, keepdim=True) / 127
    q = torch.where(scale > 0, y / scale, 0.0).round().clamp(-127, 127)
    return {"h": h.to(s["x"].dtype), "values": (q * scale).to(_values_type(c)), "scale": scale[:, 0]}


def _quant(c, s):
    n, k, g = c["n"], c["k"], c["group"]
    nt, per = -(-n // 16), -(-k // 128) * (128 // g)
    w = torch.nn.functional.pad(s["w"], (0, per * g - k, 0, nt * 16 - n)).view(nt * 16, per, g).float()
    # the quotients in 64 bits: a weight half a step between two codes goes to the even one, any other to its nearest
    scales = (w.abs().amax(2).double() / 7).to(TYPES[c["scales"]])
    d = scales.double()[:, :, None]
    q = torch.where(d > 0, w.double() / d, 0.0).round().clamp(-7, 7).float()
    values = (q * scales.float()[:, :, None]).to(_values_type(c)).view(nt * 16, per * g)[:n, :k].contiguous()
    return {"values": values, "scales": scales.view(nt, 16, per).permute(0, 2, 1).contiguous()}


def _mv(c, s):
    n, k, g = c["n"], c["k"], c["group"]
    nt, kt = -(-n // 16), -(-k // 128)
    words = s["tiles"].view(torch.int32).view(nt, kt, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(nt * 16, kt * 16, 1)
    shift = torch.arange(28, -4, -4, device=words.device, dtype=torch.int32)
    q = ((words << shift) >> 28).view(nt * 16, kt * 128 // g, g).float()
    w = (q * s["scales"].float().permute(0, 2, 1).reshape(nt * 16, -1, 1)).view(nt * 16, kt * 128)[:n, :k]
    y = s["x"].float() @ w.t()
    if s["x_scale"] is not None:
        y = y * s["x_scale"][:, None]
    return y.to(TYPES[c["out"]])


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c, f64 = s["case"], torch.float64
    if c["op"] == "norm":
        h = s["x"].to(f64) if s["residual"] is None else s["x"].to(f64).add_(s["residual"])
        r = (h.square().sum(1).div_(c["cols"]).add_(EPS)).sqrt_().reciprocal_()
        y = h * s["weight"].to(f64) * r[:, None]
        step = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 127.0
        codes = torch.round(y / step.clamp_min(1e-300)[:, None])
        return {"h": h, "values": codes * step[:, None], "scale": step}
    n, k, g = c["n"], c["k"], c["group"]
    rows = -(-n // 16) * 16
    per = -(-k // 128) * 128 // g
    if c["op"] == "quant":
        w = torch.zeros(rows, per * g, device=DEV, dtype=f64)
        w[:n, :k] = s["w"]
        w = w.view(rows * per, g)
        step = torch.linalg.vector_norm(w, ord=math.inf, dim=1).div_(7.0).to(TYPES[c["scales"]]).to(f64)
        w = torch.clamp(torch.round(w / step.clamp_min(1e-300)[:, None]), -7, 7).mul_(step[:, None])
        return {"values": w.view(rows, per * g)[:n, :k].clone(),
                "scales": step.view(rows // 16, 16, per).transpose(1, 2).clone()}
    # codes by bytes: two to each, the lower four bits first; the tile's words put back in their rows
    b = s["tiles"].view(rows // 16, per * g // 128, 4, 16, 4, 4)
    b = b.permute(0, 3, 1, 4, 2, 5).reshape(rows, per * g // 2).to(torch.int16)
    codes = torch.stack((b % 16, b // 16), 2).view(rows, per, g)
    w = torch.where(codes > 7, codes - 16, codes).to(f64)
    w.mul_(s["scales"].to(f64).transpose(1, 2).reshape(rows, per, 1))
    y = torch.mm(w.view(rows, per * g)[:n, :k], s["x"].to(f64).t().contiguous()).t().contiguous()
    return y if s["x_scale"] is None else y * s["x_scale"].to(f64)[:, None]
