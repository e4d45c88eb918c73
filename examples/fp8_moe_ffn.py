"""A mixture-of-experts feed-forward layer on E4M3 weights and activations.

    python examples/fp8_moe_ffn.py [--tokens 512] [--hidden 2048] [--ffn 1024] [--experts 64] [--top 8]

The layer routes each token to `top` of the experts, quantizes the tokens once, runs
the experts' gate and up projections on the rows they were sent, quantizes silu(gate) * up,
runs the down projections and combines each token's rows.  The number of rows of
an expert never leaves the device, so the same calls can be captured into a graph;
the example does that, checks the result against the layer computed in fp32 on
the unquantized weights, and prints the time of a replay.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_quantized_matmul_amd import binding as B  # noqa: E402


class MoeFfn:
    """Packed weights: w13 [experts, 2 ffn, hidden] (gate rows, then up rows), w2 [experts, hidden, ffn]."""

    def __init__(self, w13, w2, router, top: int):
        self.hidden, self.ffn, self.top, self.router = w13.shape[2], w2.shape[2], top, router
        self.w13, self.s13 = B.fp8_pack(w13)
        self.w2, self.s2 = B.fp8_pack(w2)

    def __call__(self, x):
        """x [tokens, hidden] bfloat16 -> [tokens, hidden] bfloat16."""
        r = B.moe_route(x @ self.router, self.top)
        q, qs = B.fp8_quant(x)
        h = B.fp8_gemm_grouped(self.w13, self.s13, self.hidden, q, qs, r.offsets, row_ids=r.row_ids)
        a, a_s = B.fp8_quant(h, swiglu=True)
        y = B.fp8_gemm_grouped(self.w2, self.s2, self.ffn, a, a_s, r.offsets)
        return B.moe_combine(y, r.slots, r.weights)


def plain(x, w13, w2, router, top: int):
    """The same layer on the unquantized weights, in fp32, one expert after the other."""
    logits = (x @ router).float()
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    weights, ids = torch.softmax(best[:, :top], 1), ids[:, :top]
    out = torch.zeros(x.shape, device=x.device)
    for e in range(w13.shape[0]):
        token, place = torch.nonzero(ids == e, as_tuple=True)
        if token.numel():
            gate, up = (x[token].float() @ w13[e].float().t()).chunk(2, 1)
            y = (torch.nn.functional.silu(gate) * up) @ w2[e].float().t()
            out.index_add_(0, token, y * weights[token, place, None])
    return out


def run(tokens: int, hidden: int, ffn: int, experts: int, top: int, replays: int = 50):
    """Returns (relative error against the fp32 layer, microseconds a replay)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    w13, w2 = rand(experts, 2 * ffn, hidden) * hidden ** -0.5, rand(experts, hidden, ffn) * ffn ** -0.5
    router, x = rand(hidden, experts) * hidden ** -0.5, rand(tokens, hidden)
    layer = MoeFfn(w13, w2, router, top)
    want = plain(x, w13, w2, router, top)
    eager = layer(x)
    rel = ((eager.float() - want).norm() / want.norm()).item()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x)
    graph.replay()
    torch.cuda.synchronize()
    if not torch.equal(out, eager):
        raise RuntimeError("a replay differs from the eager layer")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(replays):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return rel, start.elapsed_time(end) / replays * 1e3


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 512), ("hidden", 2048), ("ffn", 1024), ("experts", 64), ("top", 8)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    rel, us = run(a.tokens, a.hidden, a.ffn, a.experts, a.top)
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.ffn}, top {a.top}: {us:.1f} us a layer, "
          f"relative error against fp32 weights and activations {rel:.3f}")


if __name__ == "__main__":
    main()
