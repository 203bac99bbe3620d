"""A layer's weights from bf16 to 4 bits, through the codec and back, and the
layer's steps on them.

    python examples/quantised_layer.py [--hidden 4096] [--inner 14336] [--tokens 1]

Each matrix is rounded to 4-bit tiles (``quantize_w4``); the tiles, bytes like any
other, are coded losslessly against one codebook made from them, kept as streams,
and decoded when the layer is loaded.  Then the layer runs: the residual's
addition, its norm in 8 bits, the products with the 4-bit weights, for one token
and for a prompt, the decode step also captured into a graph.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_entropy_coding_byte_amd as lecb  # noqa: E402

CHUNK = 4096


class Stored:
    """A matrix as it is kept: the stream of its 4-bit tiles, and their scales."""

    def __init__(self, w4, codebook):
        flat = w4.tiles.view(-1)
        self.shape = (w4.n, w4.k, w4.group)
        self.count = flat.numel()
        stream, res = lecb.encode(flat, codebook, CHUNK)
        self.bytes = int(lecb.results_to_numpy(res)[0]["bytes"])
        self.stream = stream[: self.bytes].clone()
        self.scales = w4.scales

    def load(self, codebook):
        flat, res = lecb.decode(self.stream, self.bytes, codebook, CHUNK, self.count)
        if int(lecb.results_to_numpy(res)[0]["status"]) != lecb.LECB_OK:
            raise RuntimeError("the stored tiles are damaged")
        n, k, group = self.shape
        return lecb.W4Weights(flat, self.scales, n, k, group)


def codebook_of(matrices):
    """One codebook for the bytes (pairs of codes) of all the matrices."""
    hist = torch.zeros(256, dtype=torch.int64, device=matrices[0].tiles.device)
    for i, w4 in enumerate(matrices):
        lecb.lecb_histogram(w4.tiles.view(-1), hist, accumulate=i > 0)
    return lecb.DeviceCodebook.upload(lecb.lecb_build_codebook(hist.cpu().numpy(), 16, 1), hist.device)


def step(x, residual, norm_weight, up, down):
    """One block: (its output, the residual stream).  x, residual [tokens, hidden] bf16."""
    q, scale, h = lecb.rmsnorm_q8(x, norm_weight, residual=residual)
    inner = torch.nn.functional.silu(lecb.matvec_w4(q, up, x_scale=scale))
    return lecb.matvec_w4(inner, down), h


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--inner", type=int, default=14336)
    p.add_argument("--tokens", type=int, default=1)
    p.add_argument("--prompt", type=int, default=512)
    a = p.parse_args(argv)
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(1)

    def randn(*size):
        return torch.randn(*size, device=dev, generator=g)

    original = [(randn(a.inner, a.hidden) / math.sqrt(a.hidden)).bfloat16(),
                (randn(a.hidden, a.inner) / math.sqrt(a.inner)).bfloat16()]
    norm_weight = (1 + 0.1 * randn(a.hidden)).bfloat16()

    rounded = [lecb.quantize_w4(w) for w in original]
    codebook = codebook_of(rounded)
    stored = [Stored(w4, codebook) for w4 in rounded]
    up, down = (s.load(codebook) for s in stored)
    for w4, back in zip(rounded, (up, down)):
        assert torch.equal(w4.tiles.view(-1), back.tiles.view(-1)), "the codec is lossless"
    plain = sum(w.numel() * 2 for w in original)
    four = sum(s.count + s.scales.numel() * 2 for s in stored)
    kept = sum(s.bytes + s.scales.numel() * 2 for s in stored)
    print(f"weights: {plain / 2**20:.1f} MiB in bf16, {four / 2**20:.1f} in 4 bits, {kept / 2**20:.1f} as streams")

    errors = []
    for tokens in (a.tokens, a.prompt):
        x, r = randn(tokens, a.hidden).bfloat16(), randn(tokens, a.hidden).bfloat16()
        y, h = step(x, r, norm_weight, up, down)
        hf = (x.float() + r.float())
        n = hf * torch.rsqrt(hf.square().mean(1, keepdim=True) + 1e-6) * norm_weight.float()
        want = torch.nn.functional.silu(n @ original[0].float().t()) @ original[1].float().t()
        errors.append(((y.float() - want).norm() / want.norm()).item())
        print(f"{tokens} tokens: relative error {errors[-1]:.3f} against the bf16 layer")

    # the decode step as a graph: its inputs are written into x and r
    x, r = randn(a.tokens, a.hidden).bfloat16(), randn(a.tokens, a.hidden).bfloat16()
    step(x, r, norm_weight, up, down)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = step(x, r, norm_weight, up, down)
    for _ in range(3):
        x.copy_(randn(*x.shape))
        r.copy_(h)
        graph.replay()
        want, _ = step(x, r, norm_weight, up, down)
        assert torch.equal(y, want), "a replay gives what the eager step gives"
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(50):
        graph.replay()
    end.record()
    end.synchronize()
    print(f"decode step of {a.tokens} tokens: {start.elapsed_time(end) * 20:.1f} us a replay")
    return {"kept": kept, "four": four, "plain": plain, "errors": errors}


if __name__ == "__main__":
    main()
