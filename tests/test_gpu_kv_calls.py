"""Rotary positions, the 8-bit cache and its attention as programs call them: given tensors, views that start anywhere, batches
that change under a captured graph, prompts beside single tokens, and steps against one call.  Bounds as in test_gpu_kv.py.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_quantized_matmul_amd import binding as B
from oracle import fp8 as of8
from oracle import kv as okv
from tests.test_gpu_kv import (DEV, F8, TYPES, WIDE, attention_tol, batch, check, check_attention, dev, filled, host, ints, on_device, rounded,
                               same_cache, widened)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
def test_rope_returns_the_given_tensor(dtype):
    x, f, pos = torch.randn(6, 3, 32, device=DEV).to(dtype), dev(B.rope_freqs(32)), ints(np.arange(6))
    want = B.rope(x, pos, f)
    out = torch.empty(3, 6, 32, dtype=dtype, device=DEV).transpose(0, 1)
    got = B.rope(x, pos, f, out=out)
    assert got.data_ptr() == out.data_ptr() and got.stride() == out.stride() and torch.equal(out, want)
    assert B.rope(x, pos, f, out=x).data_ptr() == x.data_ptr() and torch.equal(x, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,rotary", [(128, 128), (256, 64), (192, 0), (96, 48), (8, 8)])
def test_append_of_rows_that_start_anywhere(dim, rotary, dtype):
    """Elements one by one give the codes and scales that loads of eight columns do."""
    rng = np.random.default_rng(dim)
    lens, news = [130, 9, 64, 0], [90, 2, 64, 0]
    pages, off, count = batch(rng, lens, news)
    f = dict(positions=ints(rng.integers(0, 9999, 156)), freqs=dev(B.rope_freqs(rotary))) if rotary else {}
    first, tokens = filled(rng, count, 2, dim), 156
    rows = torch.randn(tokens, 4, dim, device=DEV).to(dtype)
    odd = torch.empty(tokens * 4 * dim + 1, dtype=dtype, device=DEV)[1:].view(tokens, 4, dim)
    odd.copy_(rows)
    caches = [on_device(first), on_device(first)]
    for cache, x in zip(caches, (rows, odd)):
        B.kv_append(cache, x[:, :2], x[:, 2:], ints(pages), ints(lens), ints(off), **f)
    for a, b in zip(*caches):
        assert np.array_equal(host(a), host(b))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [0.0, -0.4, 5.0])
@pytest.mark.parametrize("width", [0, WIDE])
def test_attention_scales(width, scale, dtype):
    check_attention(np.random.default_rng(3), [200, 70, 1], [150, 2, 1], 4, 2, 64, dtype, scale=scale, width=width)
    check_attention(np.random.default_rng(4), [200, 70, 1], [1, 1, 1], 4, 2, 64, dtype, scale=scale, width=width)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width,window", [(40, 0), (4000, 0), (40, 700)])
def test_prompts_beside_single_tokens(width, window, dtype):
    """A prompt and pieces of two others among 30 single tokens at up to 2000 positions."""
    rng = np.random.default_rng(90)
    news = [1] * 15 + [300] + [1] * 10 + [70, 0] + [1] * 5 + [129]
    lens = [int(n + rng.integers(0, 2001 - n)) for n in news]
    check_attention(rng, lens, news, 8, 2, 64, dtype, window, width=width)


@pytest.mark.parametrize("width", [0, WIDE])
def test_a_captured_call_of_batches_that_change(width):
    """Lengths, offsets and tables change in place between replays, within the captured shapes: single tokens, then a prompt, then
    rows of no sequence; each replay is the eager call's."""
    rng = np.random.default_rng(91)
    heads, kv, dim, tokens, seqs = 8, 2, 64, 150, 6
    plans = [([90, 300, 5, 64, 200, 1], [1, 1, 1, 1, 1, 1]), ([150, 0, 0, 0, 0, 0], [150, 0, 0, 0, 0, 0]),
             ([120, 40, 260, 33, 1, 70], [20, 40, 60, 3, 1, 20]), ([0] * 6, [0] * 6)]
    tables = [batch(rng, lens, news, width=5) for lens, news in plans]
    count = max(c for *_, c in tables)
    cache = on_device(filled(rng, count, kv, dim))
    x = torch.randn(tokens, heads + 2 * kv, dim, device=DEV).bfloat16()
    f = dev(B.rope_freqs(dim))
    put = lambda i: [ints(widened(tables[i][0], width)), ints(plans[i][0]), ints(tables[i][1]), ints(rng.integers(0, 5000, tokens))]   # noqa: E731
    pages, lens, offsets, positions = put(0)

    def step(out):
        B.kv_append(cache, x[:, heads:heads + kv], x[:, heads + kv:], pages, lens, offsets, positions, f)
        return B.kv_attention(B.rope(x[:, :heads], positions, f), cache, pages, lens, offsets, out=out)

    out = torch.zeros(tokens, heads, dim, dtype=torch.bfloat16, device=DEV)
    state = [t.clone() for t in cache]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for i in (0, 1, 2, 3, 1, 0):
        for t, new in zip((pages, lens, offsets, positions), put(i)):
            t.copy_(new)
        x.copy_(torch.randn_like(x))
        got = []
        for run in (graph.replay, lambda: step(out)):
            for t, s in zip(cache, state):
                t.copy_(s)
            out.fill_(5.0)
            run()
            got.append([out.clone()] + [t.clone() for t in cache])
            torch.cuda.synchronize()
        for a, b in zip(*got):
            assert np.array_equal(host(a), host(b))
        assert np.all(host(out)[sum(plans[i][1]):] == 5.0)


def test_calls_on_two_streams():
    """Two batches over one cache at once, each on a stream and with a workspace of its own."""
    rng = np.random.default_rng(92)
    jobs = []
    lens, news = [3000, 400], [1, 1]
    pages, off, count = batch(rng, lens, news)
    cache = on_device(filled(rng, count, 2, 128))
    for n in ([1, 1], [100, 300]):
        _, o, _ = batch(rng, lens, n)
        jobs.append((torch.randn(sum(n), 8, 128, device=DEV).bfloat16(), cache, ints(widened(pages, 500)), ints(lens), ints(o)))
    want = [B.kv_attention(*j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (s, j) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(s):
                outs[i].append(B.kv_attention(*j))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


def test_cache_of_one_call_is_the_oracles():
    """Turned keys beside values: what one call over three sequences leaves, codes, scales and untouched pages."""
    rng = np.random.default_rng(93)
    lens, news, dim = [130, 64, 1], [70, 64, 1], 64
    pages, off, count = batch(rng, lens, news)
    want = filled(rng, count, 2, dim)
    cache = on_device(want)
    x, d = rounded(rng.standard_normal((135, 2, dim)), torch.float32)
    okv.append(want, x, -x, pages, lens, off)
    B.kv_append(cache, d, -d, ints(pages), ints(lens), ints(off), ints(np.zeros(135)), dev(B.rope_freqs(dim)))   # angles of 0
    same_cache(cache, want, dim)


def test_prompts_and_replayed_steps_against_the_whole_in_one_call():
    """Two prompts, then tokens one by one through two captured steps, each with a workspace of its own, in a table wide enough
    for parts; every step against an oracle that appends the same keys and values itself, and against one call of all
    tokens over a second cache."""
    torch.manual_seed(2)
    rng = np.random.default_rng(80)
    heads, kv, dim, steps, width = 8, 2, 64, 6, 600
    news = [100, 37]
    total = [n + steps for n in news]
    f = B.rope_freqs(dim)
    df = dev(f)
    pages, off, count = batch(rng, total, news)
    pages = widened(pages, width)
    tables = ints(pages)
    need = B.kv_attention_workspace(2, 2, heads, kv, dim, width)
    assert need > 0
    rows = [torch.randn(n, heads + 2 * kv, dim, device=DEV).bfloat16() for n in total]     # of each sequence
    cache = B.kv_cache(count, kv, dim)

    def step(x, positions, lens, offsets, into, workspace=None):
        q = B.rope(x[:, :heads], positions, df)
        B.kv_append(into, x[:, heads:heads + kv], x[:, heads + kv:], tables, lens, offsets, positions, df)
        return B.kv_attention(q, into, tables, lens, offsets, workspace=workspace)

    # the oracle's cache: keys turned in 64 bits from the same rows
    want = okv.empty(count, kv, dim)

    def put(xs, positions, lens, offsets):
        x = torch.cat(xs).double().cpu().numpy()
        okv.append(want, okv.rope(x[:, heads:heads + kv], positions, f), x[:, heads + kv:], pages, lens, offsets)

    prompt = [r[:n] for r, n in zip(rows, news)]
    at = np.concatenate([np.arange(n) for n in news])
    step(torch.cat(prompt), ints(at), ints(news), ints(off), cache)
    put(prompt, at, news, off)
    x, positions, lens = torch.stack([r[n] for r, n in zip(rows, news)]), ints(news), ints(news) + 1
    state = [t.clone() for t in cache]
    spaces = [torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, positions, lens, None, cache, spaces[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, ws in zip(graphs, spaces):
        with torch.cuda.graph(g):
            outs.append(step(x, positions, lens, None, cache, ws))
    for t, s in zip(cache, state):
        t.copy_(s)
    got = []
    for i in range(steps):
        x.copy_(torch.stack([r[n + i] for r, n in zip(rows, news)]))
        graphs[i % 2].replay()
        got.append(outs[i % 2].clone())
        (rows[0].float() @ rows[0].float().transpose(1, 2)).sum()        # the program's own work between
        spaces[1 - i % 2].fill_(0xFF)
        put([r[n + i:n + i + 1] for r, n in zip(rows, news)], [n + i for n in news], [n + i + 1 for n in news], None)
        # scales and values are the oracle's; a turned key may be the neighbouring code (rope's error beside a border)
        held = {"k": host(cache.k), "v": host(cache.v), "k_scale": host(cache.k_scale), "v_scale": host(cache.v_scale)}
        assert np.array_equal(held["v_scale"], want["v_scale"]) and np.array_equal(held["v"], want["v"])
        assert np.array_equal(held["k_scale"], want["k_scale"])
        a, b = of8.decode(held["k"]), of8.decode(want["k"])
        near = np.maximum(np.maximum(np.abs(a), np.abs(b)) * 2.0 ** -3, 2.0 ** -9)
        assert np.all(np.abs(a - b) <= near) and np.mean(a != b) < 1e-3
        q = host(B.rope(x[:, :heads], positions, df))
        ref, mag, most, small = okv.attention(q, held, pages, [n + i + 1 for n in news])
        check(host(got[-1]), ref, attention_tol(mag, most, small, 64, 120, torch.bfloat16), torch.bfloat16, f"step {i}")
        positions += 1
        lens += 1
    # all tokens in one call: the same scales, and codes but for those that were rounded again when a scale grew
    whole = B.kv_cache(count, kv, dim)
    places = np.concatenate([np.arange(n) for n in total])
    ends = np.concatenate([[0], np.cumsum(total)]).astype(np.int32)
    out = step(torch.cat(rows), ints(places), ints(total), ints(ends), whole)
    assert torch.equal(whole.k_scale, cache.k_scale) and torch.equal(whole.v_scale, cache.v_scale)
    held = {"k": host(whole.k), "v": host(whole.v), "k_scale": host(whole.k_scale), "v_scale": host(whole.v_scale)}
    for name, steps_wrote in (("k", host(cache.k)), ("v", host(cache.v))):
        a, b = of8.decode(held[name]), of8.decode(steps_wrote)
        assert np.all(np.abs(a - b) <= np.maximum(np.abs(a) * 2.0 ** -3, 2.0 ** -9))
    q = host(B.rope(torch.cat(rows)[:, :heads], ints(places), df))
    ref, mag, most, small = okv.attention(q, held, pages, total, ends)
    check(host(out), ref, attention_tol(mag, most, small, 64, 120, torch.bfloat16), torch.bfloat16, "whole")
