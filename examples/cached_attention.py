"""The attention half of a layer that serves several requests, on 4-bit weights and an
8-bit cache.

    python examples/cached_attention.py [--hidden 2048] [--heads 16] [--kv-heads 4] [--prompt 700] [--steps 24]

Prompts of different lengths go through together: the norm in 8 bits, the products with
4-bit weights, their keys and values into the cache's blocks, attention over them.  Then
the requests decode token by token; the step is one graph, whose lengths count on between
replays.  At last one request is put aside: its blocks, bytes like any other, are coded
losslessly, come back into other blocks of the cache, and its next step gives the same bits.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_entropy_coding_byte_amd as lecb  # noqa: E402

CHUNK, BLOCK = 4096, 64


class Layer:
    def __init__(self, hidden, heads, kv_heads, g, dev):
        self.heads, self.kv_heads, self.dim = heads, kv_heads, hidden // heads
        sizes = [(hidden, hidden), (2 * kv_heads * self.dim, hidden), (hidden, hidden)]
        self.original = [(torch.randn(*s, device=dev, generator=g) / math.sqrt(hidden)).bfloat16() for s in sizes]
        self.wq, self.wkv, self.wo = (lecb.quantize_w4(w) for w in self.original)
        self.norm = torch.ones(hidden, device=dev, dtype=torch.bfloat16)

    def step(self, x, cache, table, lengths, starts=None):
        """(output, queries, keys, values) of the new tokens x [tokens, hidden]."""
        n = x.shape[0]
        h, scale, _ = lecb.rmsnorm_q8(x, self.norm)
        q = lecb.matvec_w4(h, self.wq, x_scale=scale).view(n, self.heads, self.dim)
        kv = lecb.matvec_w4(h, self.wkv, x_scale=scale).view(n, 2 * self.kv_heads, self.dim)
        k, v = kv[:, : self.kv_heads], kv[:, self.kv_heads :]
        lecb.cache_write_q8(cache, k, v, table, lengths, starts)
        out = lecb.attention_q8(q, cache, table, lengths, starts)
        return lecb.matvec_w4(out.view(n, -1), self.wo), q, k, v


def plain(q, k, v):
    """The last tokens' attention over k, v [length, kv heads, dim], in 32 bits and without a cache."""
    n, group = q.shape[0], q.shape[1] // k.shape[1]
    k, v = (t.float().repeat_interleave(group, 1).transpose(0, 1).contiguous() for t in (k, v))
    score = (q.float().transpose(0, 1) @ k.transpose(1, 2).contiguous()) / math.sqrt(q.shape[2])
    length = k.shape[1]
    away = torch.arange(length, device=q.device)[None] > torch.arange(length - n, length, device=q.device)[:, None]
    return (torch.softmax(score.masked_fill(away, -math.inf), 2) @ v).transpose(0, 1)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--heads", type=int, default=16)
    p.add_argument("--kv-heads", type=int, default=4)
    p.add_argument("--prompt", type=int, default=700)
    p.add_argument("--steps", type=int, default=24)
    a = p.parse_args(argv)
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(1)
    layer = Layer(a.hidden, a.heads, a.kv_heads, g, dev)

    # three requests; each is given the blocks that it will come to need, and one's worth more is kept free
    prompts = [a.prompt, a.prompt // 3 + 1, 1]
    width = -(-(a.prompt + a.steps + 1) // BLOCK)
    cache = lecb.new_cache_q8(4 * width, a.kv_heads, layer.dim, BLOCK)
    order = torch.randperm(4 * width, device=dev, generator=g).to(torch.int32).view(4, width)
    table = order[:3].clone()

    def tokens(n):
        return torch.randn(n, a.hidden, device=dev, generator=g).bfloat16()

    def ints(*values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    starts = [0]
    for n in prompts:
        starts.append(starts[-1] + n)
    lengths = ints(*prompts)
    out, q, k, v = layer.step(tokens(starts[-1]), cache, table, lengths, ints(*starts))
    held = [(k[s:e].clone(), v[s:e].clone()) for s, e in zip(starts, starts[1:])]
    errors = []
    seen = lecb.attention_q8(q, cache, table, lengths, ints(*starts))
    for i, (s, e) in enumerate(zip(starts, starts[1:])):
        want = plain(q[s:e], *held[i])
        errors.append(((seen[s:e].float() - want).norm() / want.norm()).item())
    print("prompts of %s tokens: attention off by %s against 32 bits without a cache"
          % (prompts, ", ".join("%.4f" % e for e in errors)))

    # the decoding step as a graph: its tokens are written into x, the lengths count on
    x = tokens(3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lengths.add_(1)
        out, q, k, v = layer.step(x, cache, table, lengths)
    for _ in range(a.steps):
        x.copy_(tokens(3))
        graph.replay()
        held = [(torch.cat((hk, k[i : i + 1])), torch.cat((hv, v[i : i + 1]))) for i, (hk, hv) in enumerate(held)]
        seen = lecb.attention_q8(q, cache, table, lengths)
        assert torch.equal(out, lecb.matvec_w4(seen.view(3, -1), layer.wo)), "a replay gives what the eager step gives"
    assert lengths.tolist() == [n + a.steps for n in prompts]
    for i in range(3):
        want = plain(q[i : i + 1], *held[i])
        errors.append(((seen[i : i + 1].float() - want).norm() / want.norm()).item())
    print("after %d steps: off by %s" % (a.steps, ", ".join("%.4f" % e for e in errors[3:])))

    # request 0 put aside: its blocks' codes as streams, and back into the free blocks
    mine, free = table[0].long(), order[3].long()
    streams, kept, size = [], 0, 0
    for codes in (cache.k, cache.v):
        flat = codes[mine].view(torch.uint8).view(-1)
        hist = torch.zeros(256, dtype=torch.int64, device=dev)
        lecb.lecb_histogram(flat, hist)
        book = lecb.DeviceCodebook.upload(lecb.lecb_build_codebook(hist.cpu().numpy(), 16, 1), dev)
        stream, res = lecb.encode(flat, book, CHUNK)
        used = int(lecb.results_to_numpy(res)[0]["bytes"])
        streams.append((stream[:used].clone(), used, book))
        kept, size = kept + used, size + flat.numel()
    want = lecb.attention_q8(q, cache, table, lengths)
    for codes, (stream, used, book) in zip((cache.k, cache.v), streams):
        back, res = lecb.decode(stream, used, book, CHUNK, codes[mine].numel())
        if int(lecb.results_to_numpy(res)[0]["status"]) != lecb.LECB_OK:
            raise RuntimeError("the stored blocks are damaged")
        codes[free] = back[: codes[mine].numel()].view(torch.int8).view(codes[free].shape)
        codes[mine] = 0
    for scales in (cache.k_scale, cache.v_scale):
        scales[free] = scales[mine]
    table[0] = order[3]
    assert torch.equal(lecb.attention_q8(q, cache, table, lengths), want), "the codec is lossless"
    print(f"one request's blocks: {size / 2**20:.2f} MiB, {kept / 2**20:.2f} as streams")

    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    eight = lengths.clone()
    lengths.copy_((eight - 9).clamp_min(0))
    start.record()
    for _ in range(8):
        graph.replay()
    end.record()
    end.synchronize()
    print(f"decoding step of 3 requests: {start.elapsed_time(end) * 125:.1f} us a replay")
    return {"errors": errors, "kept": kept, "size": size}


if __name__ == "__main__":
    main()
