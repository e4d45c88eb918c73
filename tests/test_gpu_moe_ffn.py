"""GPU parity of the expert layer of few tokens.

The bound, from the arithmetic.  The 128 products of a block are exact in fp32, or cut at 2^-22 (a row of x in one
or two fp16 terms: its elements below 2^-22 of its largest are off by 2^-33 of that), and added with a rounding of
2^-23 each; the scaling, the blocks' sum and the waves' round kb + 6 times by 2^-24.  silu is within 4 x 2^-23.  The
hidden row is rounded to fp16, half a step of which is up to 2^-11 of it (two terms, 2^-22, for fp32) and goes through the same sums; the experts' weights (6 x
2^-23) and their sum add 6 + top.  All are relative to the oracle's bound of the terms.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_quantized_matmul_amd import binding as B
from oracle import fp8 as of8
from oracle import moe as omoe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def weights(rng, experts, rows, cols):
    """Codes and scales as fp8_pack writes them, on the host, from a few distinct matrices."""
    got = [of8.quant_weight((rng.standard_normal((rows, cols)) * cols ** -0.5 * np.exp(rng.standard_normal((rows, 1)))).astype(np.float32))
           for _ in range(min(experts, 4))]
    q, s = np.stack([got[e % len(got)][0] for e in range(experts)]), np.stack([got[e % len(got)][1] * np.float32(1 + e / 8) for e in range(experts)])
    return q, s


def tol(mag, hidden, ffn, top, dtype):
    sums = lambda k: 128 * 2.0 ** -23 + (of8.blocks(k) + 6) * 2.0 ** -24          # noqa: E731
    return mag * (sums(hidden) + sums(ffn) + (2.0 ** -21 if dtype == torch.float32 else 2.0 ** -11 + 2.0 ** -21) + (16 + top) * 2.0 ** -23)


def check(got, ref, t, dtype, label):
    half, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    # the type's nearest value to what lies half a step past its largest (fp16: 65504 + 16) is an infinity
    over = np.abs(ref) + t >= torch.finfo(dtype).max * (1 + half / 2)
    assert np.all(np.isfinite(got) | over), label
    assert np.all(np.sign(got) == np.sign(ref), where=over), label
    worst = np.max(np.abs(got - ref) / (t + half * (np.abs(ref) + t) + tiny), where=np.isfinite(got), initial=0.0)
    assert worst <= 1.0, f"{label}: {worst:.3g} of the bound"


def run(rng, tokens, experts, top, hidden, ffn, dtype, renorm=True, ltype=None, logits=None, x=None, label=""):
    q13, s13 = weights(rng, experts, 2 * ffn, hidden)
    q2, s2 = weights(rng, experts, hidden, ffn)
    x = rng.standard_normal((tokens, hidden)) * np.exp(rng.standard_normal((tokens, 1))) if x is None else x
    logits = rng.standard_normal((tokens, experts)) if logits is None else logits
    d, dl = torch.from_numpy(x).to(dtype), torch.from_numpy(logits).to(ltype or dtype)
    up = lambda a, t=None: torch.from_numpy(a).to(DEV) if t is None else torch.from_numpy(a).to(DEV).view(t)   # noqa: E731
    args = (up(q13, F8), up(s13), up(q2, F8), up(s2))
    y = B.moe_ffn(d.to(DEV), *args, dl.to(DEV), top, renorm=renorm)
    assert y.dtype == dtype and y.shape == (tokens, hidden)
    ref, mag = omoe.ffn(d.double().numpy(), q13, s13, q2, s2, dl.double().numpy(), top, renorm)
    check(host(y), ref, tol(mag, hidden, ffn, top, dtype), dtype, label or f"{tokens} of {experts} x {hidden} x {ffn}")
    return d, dl, args, y, ref


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,experts,top,hidden,ffn", [
    (1, 1, 1, 1, 1), (1, 8, 2, 128, 128), (3, 4, 4, 100, 65), (7, 12, 3, 312, 1092), (16, 8, 2, 256, 130),
    (17, 3, 2, 129, 127), (32, 6, 6, 384, 96), (32, 64, 8, 64, 64), (2, 130, 5, 72, 40), (5, 1024, 32, 16, 16)])
def test_expert_layer(tokens, experts, top, hidden, ffn, dtype):
    run(np.random.default_rng(tokens + hidden), tokens, experts, top, hidden, ffn, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ltype", TYPES)
@pytest.mark.parametrize("renorm", [True, False])
def test_weights_over_all_and_types_of_logits(dtype, ltype, renorm):
    run(np.random.default_rng(3), 9, 20, 4, 160, 136, dtype, renorm, ltype)


@pytest.mark.parametrize("tokens", [1, 5, 32])
@pytest.mark.parametrize("renorm", [True, False])
def test_routing_is_moe_routes(tokens, renorm):
    """Ties, masks, NaN and infinities among the logits: the experts and weights of moe_route."""
    rng = np.random.default_rng(tokens)
    logits = np.round(rng.standard_normal((tokens, 40)) * 2) / 2
    logits[rng.random(logits.shape) < 0.4] = -np.inf
    logits[0, 3], logits[0, 7] = np.nan, np.inf
    if tokens > 2:
        logits[1] = -np.inf                                              # no expert: a row of zeros
        logits[2] = -np.inf
        logits[2, 39] = -3e38
    _, _, _, y, ref = run(rng, tokens, 40, 6, 64, 48, torch.float32, renorm, logits=logits)
    if tokens > 2:
        assert np.all(host(y)[1] == 0.0) and np.any(ref[2] != 0.0)


@pytest.mark.parametrize("tokens,hidden,ffn", [(1, 64, 64), (32, 200, 130)])
def test_no_token_has_an_expert(tokens, hidden, ffn):
    logits = np.full((tokens, 9), -np.inf)
    *_, y, ref = run(np.random.default_rng(2), tokens, 9, 3, hidden, ffn, torch.bfloat16, logits=logits)
    assert np.all(host(y) == 0.0) and np.all(ref == 0.0)


def test_all_tokens_to_one_expert():
    logits = np.full((32, 70), -np.inf)
    logits[:, 66] = np.arange(32)
    run(np.random.default_rng(4), 32, 70, 4, 260, 140, torch.float16, logits=logits)


@pytest.mark.parametrize("dtype", TYPES)
def test_wide_layers(dtype):
    """More blocks a row than waves, and rows in several turns of every workgroup."""
    run(np.random.default_rng(6), 20, 24, 2, 2200, 1300, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_unlike_size_and_not_finite(dtype):
    rng = np.random.default_rng(9)
    x = rng.standard_normal((6, 200))
    x[1] *= 2.0 ** -14 if dtype == torch.float16 else 2.0 ** -40
    x[2] *= 2.0 ** 7 if dtype == torch.float16 else 2.0 ** 20
    x[3] = 0.0
    d, dl, args, y, _ = run(rng, 6, 5, 2, 200, 90, dtype, x=x)
    assert np.all(host(y)[3] == 0.0)
    base = host(y)
    d = d.to(DEV)
    d[0, 7], d[4, 199] = float("nan"), float("-inf")
    got = host(B.moe_ffn(d, *args, dl.to(DEV), 2))
    assert np.all(np.isnan(got[[0, 4]])) and np.array_equal(got[[1, 2, 3, 5]], base[[1, 2, 3, 5]])


def test_gates_far_out():
    """silu of -200 .. 200: 0 and the gate itself."""
    rng = np.random.default_rng(10)
    run(rng, 4, 3, 1, 64, 64, torch.float32, x=200.0 * rng.standard_normal((4, 64)))


def test_strided_rows_and_given_tensors():
    rng = np.random.default_rng(11)
    d, dl, args, y, _ = run(rng, 5, 9, 3, 136, 72, torch.bfloat16)
    wide = torch.zeros(5, 140, dtype=torch.bfloat16, device=DEV)
    wide[:, 3:139] = d.to(DEV)
    logits = torch.zeros(5, 11, dtype=torch.bfloat16, device=DEV)
    logits[:, 1:10] = dl.to(DEV)
    ws = torch.full((B.moe_ffn_workspace(5, 9, 3, 136, 72),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(y)
    for _ in range(2):
        assert torch.equal(B.moe_ffn(wide[:, 3:139], *args, logits[:, 1:10], 3, out=out, workspace=ws), y)
    with pytest.raises(ValueError, match="workspace"):
        B.moe_ffn(wide[:, 3:139], *args, logits[:, 1:10], 3, workspace=ws[:-1])
    with pytest.raises(B.BqmError):
        B.moe_ffn(wide[:, 3:139], *args, logits[:, 1:10], 10)


def test_beside_the_calls_it_joins():
    """The same layer by moe_route, fp8_gemm_grouped and moe_combine: activations quantized there, so the two differ by
    that alone.  A code is off by half a step (2^-4 of it, rms about 2^-5.3): both layers' roundings of
    random sign leave a relative difference of a few hundredths, far from a wrong expert's."""
    torch.manual_seed(1)
    x = torch.randn(8, 256, device=DEV).bfloat16()
    w13, s13 = B.fp8_pack(torch.randn(16, 2 * 192, 256, device=DEV) / 16)
    w2, s2 = B.fp8_pack(torch.randn(16, 256, 192, device=DEV) / 14)
    logits = torch.randn(8, 16, device=DEV)
    r = B.moe_route(logits, 4)
    q, qs = B.fp8_quant(x)
    h = B.fp8_gemm_grouped(w13, s13, 256, q, qs, r.offsets, row_ids=r.row_ids)
    a, a_s = B.fp8_quant(h, swiglu=True)
    want = B.moe_combine(B.fp8_gemm_grouped(w2, s2, 192, a, a_s, r.offsets), r.slots, r.weights).float()
    got = B.moe_ffn(x, w13, s13, w2, s2, logits, 4).float()
    assert ((got - want).norm() / want.norm()).item() < 0.1


def test_graphs_that_share_a_workspace():
    rng = np.random.default_rng(13)
    layers = [run(rng, 3, 10, 3, 200, 150, torch.bfloat16), run(rng, 20, 5, 2, 1100, 70, torch.float32)]
    calls = [(d.to(DEV), *args, dl.to(DEV), top) for (d, dl, args, *_), top in zip(layers, (3, 2))]
    want = [B.moe_ffn(*c) for c in calls]
    need = max(B.moe_ffn_workspace(3, 10, 3, 200, 150), B.moe_ffn_workspace(20, 5, 2, 1100, 70))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in calls], []
    for g, c in zip(graphs, calls):
        with torch.cuda.graph(g):
            outs.append(B.moe_ffn(*c, workspace=ws))
    for i in range(6):
        outs[i % 2].zero_()
        graphs[i % 2].replay()
        assert torch.equal(outs[i % 2], want[i % 2])
        assert torch.equal(B.moe_ffn(*calls[i % 2], workspace=ws), want[i % 2])


def test_graph_replays_and_other_streams():
    rng = np.random.default_rng(12)
    d, dl, args, y, _ = run(rng, 6, 10, 3, 200, 150, torch.bfloat16)
    x, logits = d.to(DEV), dl.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(B.moe_ffn(x, *args, logits, 3), y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = B.moe_ffn(x, *args, logits, 3)
    for i in range(4):
        x.copy_(torch.randn(6, 200, device=DEV))
        logits.copy_(torch.randn(6, 10, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, B.moe_ffn(x, *args, logits, 3))
