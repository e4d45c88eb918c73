"""One decoder layer of a decode batch on E4M3 weights and an E4M3 cache.

    python examples/fp8_decode_layer.py [--seqs 16] [--context 4096] [--hidden 2048] [--heads 16] [--kv-heads 4]
                                        [--ffn 1024] [--experts 64] [--top 8]

Every sequence has a prompt in the paged cache and decodes one token a step: the queries and keys are turned by their
positions, the keys and values go into the sequences' pages, the queries attend to them and the
experts that the router chooses take the result, with residuals between.  Lengths, positions and
pages stay on the device, so a step is captured into a graph once and replayed for the tokens after; the example
checks a replay against the eager step and the step against the layer in fp32 on the values that
codes and scales stand for, and prints the time of a replay.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_quantized_matmul_amd import binding as B  # noqa: E402

DIM = 128


class DecodeLayer:
    """Packed projections, router and experts, a cache of `pages` pages and the rotation's frequencies."""

    def __init__(self, qkv, o, router, w13, w2, heads: int, kv_heads: int, top: int, pages: int):
        self.hidden, self.heads, self.kv, self.top, self.router = qkv.shape[1], heads, kv_heads, top, router
        self.qkv, self.o = B.fp8_pack(qkv), B.fp8_pack(o)
        self.w13, self.w2 = B.fp8_pack(w13), B.fp8_pack(w2)
        self.cache = B.kv_cache(pages, kv_heads, DIM)
        self.freqs = torch.from_numpy(B.rope_freqs(DIM)).cuda()

    def attend(self, x, pages, lens, offsets, positions):
        """x [tokens, hidden] -> x and the attention's output through its projection."""
        q, s = B.fp8_quant(x)
        rows = B.fp8_gemm(*self.qkv, self.hidden, q, s).view(-1, self.heads + 2 * self.kv, DIM)
        query, key, value = rows.split([self.heads, self.kv, self.kv], 1)
        query = B.rope(query, positions, self.freqs)
        B.kv_append(self.cache, key, value, pages, lens, offsets, positions, self.freqs)
        a, a_s = B.fp8_quant(B.kv_attention(query, self.cache, pages, lens, offsets).view(x.shape[0], -1))
        return x + B.fp8_gemm(*self.o, self.heads * DIM, a, a_s)

    def __call__(self, x, pages, lens, positions):
        """One token a sequence, up to 32 of them."""
        x = self.attend(x, pages, lens, None, positions)
        return x + B.moe_ffn(x, *self.w13, *self.w2, x @ self.router, self.top)


def values(codes, scale):
    """fp32 of fp8_pack codes [..., rows, 128 kb]."""
    s = scale.repeat_interleave(128, -2)[..., :codes.shape[-2], :].repeat_interleave(128, -1)
    return codes.float() * s


def plain(layer, x, pages, lens):
    """The step after x's keys and values are in the cache, in fp32 (activations unquantized)."""
    x = x.float()
    rows = (x @ values(*layer.qkv)[:, :layer.hidden].t()).view(x.shape[0], -1, DIM)
    angle = (lens - 1).double()[:, None] * layer.freqs
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q1, q2 = rows[:, :layer.heads].chunk(2, -1)
    q = torch.cat((q1 * cos - q2 * sin, q1 * sin + q2 * cos), -1)
    out = torch.zeros_like(q)
    k, v, ks, vs = layer.cache
    for s in range(x.shape[0]):
        n, at = int(lens[s]), pages[s, :(int(lens[s]) + 63) // 64].long()
        keys = (k[at].float() * ks[at][..., None, None]).transpose(0, 1).reshape(layer.kv, -1, DIM)[:, :n]
        vals = (v[at].float() * vs[at][..., None, None]).permute(1, 0, 3, 2).reshape(layer.kv, -1, DIM)[:, :n]
        for h in range(layer.heads):
            g = h * layer.kv // layer.heads
            out[s, h] = torch.softmax(keys[g] @ q[s, h] * DIM ** -0.5, 0) @ vals[g]
    x = x + out.view(x.shape[0], -1) @ values(*layer.o)[:, :layer.heads * DIM].t()
    best, ids = torch.sort((x.bfloat16() @ layer.router).float(), dim=1, descending=True, stable=True)
    y = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for w, e in zip(torch.softmax(best[t, :layer.top], 0), ids[t, :layer.top].tolist()):
            gate, up = (values(layer.w13[0][e], layer.w13[1][e])[:, :layer.hidden] @ x[t]).chunk(2)
            y[t] += w * (values(layer.w2[0][e], layer.w2[1][e])[:, :gate.numel()] @ (torch.nn.functional.silu(gate) * up))
    return x + y


def run(seqs: int, context: int, hidden: int, heads: int, kv_heads: int, ffn: int, experts: int, top: int, replays: int = 50):
    """Returns (relative error against the fp32 layer, microseconds a replay)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    width = (context + replays + 8 + 63) // 64
    layer = DecodeLayer(rand((heads + 2 * kv_heads) * DIM, hidden) * hidden ** -0.5, rand(hidden, heads * DIM) * (heads * DIM) ** -0.5,
                        rand(hidden, experts) * hidden ** -0.5, rand(experts, 2 * ffn, hidden) * hidden ** -0.5,
                        rand(experts, hidden, ffn) * ffn ** -0.5, heads, kv_heads, top, seqs * width)
    pages = torch.randperm(seqs * width, device="cuda", generator=g).int().view(seqs, width)
    # prompts of unlike length, all in one call
    lens = (context - torch.arange(seqs, device="cuda") * (context // (2 * seqs))).int()
    offsets = torch.nn.functional.pad(torch.cumsum(lens, 0), (1, 0)).int()
    tokens = int(offsets[-1])
    positions = torch.arange(tokens, device="cuda").int() - torch.repeat_interleave(offsets[:-1], lens.long())
    layer.attend(rand(tokens, hidden), pages, lens, offsets, positions)

    x, position = rand(seqs, hidden), lens.clone()
    lens += 1
    eager = layer(x, pages, lens, position)                     # the same tokens again change nothing in the cache
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, pages, lens, position)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, pages, lens, position)
    graph.replay()
    torch.cuda.synchronize()
    if not torch.equal(out, eager):
        raise RuntimeError("a replay differs from the eager step")
    want = plain(layer, x, pages, lens)
    rel = ((eager.float() - want).norm() / want.norm()).item()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(replays):
        graph.replay()
        lens += 1
        position += 1
    end.record()
    torch.cuda.synchronize()
    return rel, start.elapsed_time(end) / replays * 1e3


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("seqs", 16), ("context", 4096), ("hidden", 2048), ("heads", 16), ("kv-heads", 4), ("ffn", 1024),
                          ("experts", 64), ("top", 8)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    rel, us = run(a.seqs, a.context, a.hidden, a.heads, a.kv_heads, a.ffn, a.experts, a.top)
    print(f"{a.seqs} sequences of up to {a.context}, {a.heads} heads to {a.kv_heads}, {a.experts} experts of {a.hidden} x {a.ffn}, "
          f"top {a.top}: {us:.1f} us a step of one layer, relative error against fp32 activations {rel:.3f}")


if __name__ == "__main__":
    main()
