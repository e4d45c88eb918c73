"""GPU parity of rotary positions, the paged 8-bit cache and its attention.

Bounds, from the arithmetic.

rope: the angle is formed in fp64 (4 roundings of 2^-53 of it, in the oracle too), cos and sin are within 4 x 2^-24 of
the scale, the two products and their sum round twice: (7 x 2^-24 + 2^-50 angle) mscale (|x1| + |x2|), then
half a step of the type.

append: scales and codes of values that are not turned are exact.  A turned key is within rope's bound in fp32, and
its code is the nearest to that: half a step (2^-4 of it, 2^-10 of the scale below 2^-6 of it) and that bound.

attention: a row's scores.  dp products, exact in fp32 or cut at 2^-23 where q has two terms, with a rounding of 2^-23
each (the matrix cores may truncate), and 8 more: e = (2 dp + 16) 2^-23 times the sum of |scale q k|,
absolute.  exp adds 2^-22.  p is rounded to fp16, of 11 bits, half a step of which is up to 2^-11 of it (two terms,
2^-22, for fp32), the products p v are
summed within a page (66 roundings of 2^-23) and over pages and parts (2^-23 each), the sum of p likewise: with L
positions in all, out is off by at most
    (2 e + 2^-21 + p's + (66 + L / 16) 2^-22) sum p |v| + 2^-40 sum |v|
and half a step of the type: p times 2^15 in fp16 is in steps of 2^-24 below 2^-14, so a p below 2^-29 of the largest is
off by up to 2^-40 of it, in two terms too.  With 16-bit rows p is times 2^11 of a maximum that may lag behind by 2^4: 2^-36.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_quantized_matmul_amd import binding as B
from oracle import fp8 as of8
from oracle import kv as okv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def ints(a):
    return dev(np.asarray(a, dtype=np.int32))


def host(t):
    torch.cuda.synchronize()
    t = t.view(torch.uint8) if t.dtype == F8 else t.double() if t.is_floating_point() else t
    return t.cpu().numpy()


def rounded(x, dtype):
    """x as the type holds it, on the host, in fp64, and on the device."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(dtype)
    return t.double().numpy(), t.to(DEV)


def check(got, ref, tol, dtype, label=""):
    bound = tol + torch.finfo(dtype).eps / 2 * (np.abs(ref) + tol) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    assert np.all(np.isfinite(got)), label
    worst = np.max(np.abs(got - ref) / bound)
    assert worst <= 1.0, f"{label}: {worst:.3g} of the bound"


# ------------------------------------------------------------------ rope

def rope_tol(x, positions, freqs, interleaved, mscale):
    r = 2 * len(freqs)
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    tol = np.zeros(x.shape)
    angle = np.abs(np.asarray(positions, dtype=np.float64))[:, None, None] * np.asarray(freqs)
    tol[..., i] = tol[..., j] = (7 * 2.0 ** -24 + 2.0 ** -50 * angle) * mscale * (np.abs(x[..., i]) + np.abs(x[..., j]))
    return tol


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rotary", [(1, 1, 2, 2), (1, 32, 128, 128), (5, 3, 26, 26), (70, 12, 26, 12),
                                                     (3, 2, 80, 32), (129, 5, 64, 64), (600, 3, 128, 64), (2, 1, 1024, 1024),
                                                     (7, 2, 40, 16), (513, 2, 256, 256)])
def test_rope(tokens, heads, dim, rotary, interleaved, dtype):
    rng = np.random.default_rng(tokens * 100 + dim)
    x, d = rounded(rng.standard_normal((tokens, heads, dim)), dtype)
    pos = rng.integers(0, 1 << 20, tokens)
    pos[0] = 0 if tokens > 1 else 131071
    f = B.rope_freqs(rotary)
    for backward in (False, True):
        y = B.rope(d, ints(pos), dev(f), interleaved=interleaved, mscale=1.25, backward=backward)
        assert y.dtype == dtype and y.is_contiguous()
        check(host(y), okv.rope(x, pos, f, interleaved, 1.25, backward), rope_tol(x, pos, f, interleaved, 1.25), dtype)


def test_rope_of_far_positions():
    """Position 2^31 - 1 turns by 2^31 radians: 2^-22 of one remains of fp64."""
    x, d = rounded(np.random.default_rng(3).standard_normal((4, 2, 64)), torch.float32)
    pos, f = [2 ** 31 - 1, 2 ** 30, -5, -2 ** 31], B.rope_freqs(64)
    check(host(B.rope(d, ints(pos), dev(f))), okv.rope(x, pos, f), rope_tol(x, pos, f, False, 1.0), torch.float32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,rotary", [(64, 64), (64, 16), (26, 26)])
def test_rope_views_in_place_and_heads_first(dim, rotary, dtype):
    rng = np.random.default_rng(dim + rotary)
    wide_h, wide = rounded(rng.standard_normal((9, 7, dim)), dtype)
    pos, f = rng.integers(0, 5000, 9), B.rope_freqs(rotary)
    want = host(B.rope(wide, ints(pos), dev(f)))
    part = B.rope(wide[:, 2:5], ints(pos), dev(f))                       # part of the projections' rows
    assert np.array_equal(host(part), want[:, 2:5])
    odd = torch.empty(9 * 7 * dim + 1, dtype=dtype, device=DEV)[1:].view(9, 7, dim)
    odd.copy_(wide)
    assert np.array_equal(host(B.rope(odd, ints(pos), dev(f))), want)     # rows that start anywhere
    first = wide.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty(7, 9, dim, dtype=dtype, device=DEV).transpose(0, 1)
    assert B.rope(first, ints(pos), dev(f), out=out) is out or True
    assert np.array_equal(host(out), want)
    inside = wide.clone()
    B.rope(inside[:, 2:5], ints(pos), dev(f), out=inside[:, 2:5])
    got = host(inside)
    assert np.array_equal(got[:, 2:5], want[:, 2:5])
    assert np.array_equal(got[:, :2], wide_h[:, :2]) and np.array_equal(got[:, 5:], wide_h[:, 5:])
    with pytest.raises(B.BqmError):
        B.rope(wide, ints(pos), dev(f), out=wide[:1].expand(9, 7, dim))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """<g, rope(x + h e) - rope(x - h e)> / 2 h, element by element, in the fp32 of the op with h = 1: rope is linear, so the
    difference is off by the roundings of both alone (2 x 8 x 2^-24 of |x| + 1 each, summed over a row's 16 outputs)."""
    rng = np.random.default_rng(8)
    x, d = rounded(rng.standard_normal((3, 1, 16)), torch.float32)
    g, dg = rounded(rng.standard_normal((3, 1, 16)), torch.float32)
    pos, f = [3, 1000, 77777], B.rope_freqs(12)
    kw = dict(interleaved=interleaved, mscale=1.3)
    got = host(B.rope(dg, ints(pos), dev(f), backward=True, **kw))
    check(got, okv.rope(g, pos, f, interleaved, 1.3, True), rope_tol(g, pos, f, interleaved, 1.3), torch.float32)
    for c in range(16):
        e = torch.zeros(1, 1, 16, device=DEV)
        e[..., c] = 1.0
        diff = host(B.rope(d + e, ints(pos), dev(f), **kw)) - host(B.rope(d - e, ints(pos), dev(f), **kw))
        num = (g * diff / 2).sum((1, 2))
        assert np.all(np.abs(num - got[:, 0, c]) <= 16 * 1.3 * 2.0 ** -23 * 16 * (np.abs(x).max() + 1) * np.abs(g).max())


# ------------------------------------------------------------------ the cache

def batch(rng, lens, news, spare=3, width=None):
    """pages [seqs, width] in a random order (-1 past a sequence's), offsets, and the pages of the cache."""
    need = [max(1, -(-n // 64)) for n in lens]
    width = width or max(need)
    count = sum(need) + spare
    order = rng.permutation(count)
    pages, at = np.full((len(lens), width), -1, dtype=np.int32), 0
    for s, n in enumerate(need):
        pages[s, :min(n, width)] = order[at:at + n][:width]
        at += n
    return pages, np.concatenate([[0], np.cumsum(news)]).astype(np.int32), count


def on_device(c):
    return B.KvCache(dev(c["k"]).view(F8), dev(c["v"]).view(F8), dev(c["k_scale"], torch.float32), dev(c["v_scale"], torch.float32))


def filled(rng, count, heads, dim):
    """A cache whose pages are full of codes, NaN among them in no page."""
    c = okv.empty(count, heads, dim)
    c["k"][..., :dim] = rng.integers(0, 0x7E, c["k"][..., :dim].shape) | (rng.integers(0, 2, c["k"][..., :dim].shape) << 7)
    c["v"][..., :dim, :] = rng.integers(0, 0x7E, c["v"][..., :dim, :].shape) | (rng.integers(0, 2, c["v"][..., :dim, :].shape) << 7)
    for n in ("k_scale", "v_scale"):
        c[n][:] = 2.0 ** rng.integers(-11, -6, c[n].shape)
    return c


def same_cache(got: B.KvCache, want: dict, dim: int):
    for name, t in zip(("k_scale", "v_scale"), got[2:]):
        assert np.array_equal(host(t), want[name]), name
    for name, t in zip(("k", "v"), got[:2]):
        g, w = host(t), want[name]
        g, w = (g[..., :dim], w[..., :dim]) if name == "k" else (g[..., :dim, :], w[..., :dim, :])
        assert np.array_equal(of8.decode(g), of8.decode(w), equal_nan=True), name


LENS = [([1], [1]), ([64], [64]), ([65], [2]), ([3, 0, 130, 64, 129], [1, 0, 70, 64, 1]), ([200, 7, 64], [137, 7, 3]),
        ([500], [500])]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,heads", [(26, 3), (32, 1), (64, 2), (80, 2), (128, 2), (192, 1), (256, 1), (1, 2), (129, 1)])
@pytest.mark.parametrize("lens,news", LENS)
def test_append_is_exact(lens, news, dim, heads, dtype):
    rng = np.random.default_rng(sum(lens) + dim)
    pages, off, count = batch(rng, lens, news)
    want = filled(rng, count, heads, dim)
    cache = on_device(want)
    tokens = int(off[-1])
    x, d = rounded(rng.standard_normal((tokens, 2 * heads, dim)) * np.exp(2 * rng.standard_normal((tokens, 2 * heads, 1))), dtype)
    before = {n: a.copy() for n, a in want.items()}
    okv.append(want, x[:, :heads], x[:, heads:], pages, lens, off)
    B.kv_append(cache, d[:, :heads], d[:, heads:], ints(pages), ints(lens), offsets=ints(off))
    same_cache(cache, want, dim)
    assert any(not np.array_equal(before[n], want[n]) for n in want)
    # once more: the same tokens change nothing
    B.kv_append(cache, d[:, :heads], d[:, heads:], ints(pages), ints(lens), offsets=ints(off))
    same_cache(cache, want, dim)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary", [(26, 26), (128, 128), (128, 64), (96, 48), (80, 32)])
def test_append_turns_keys(dim, rotary, interleaved, dtype):
    rng = np.random.default_rng(dim + rotary)
    lens, news = [90, 5, 64], [40, 1, 64]
    pages, off, count = batch(rng, lens, news)
    cache = B.kv_cache(count, 2, dim)
    x, d = rounded(rng.standard_normal((105, 2, dim)), dtype)
    pos, f = rng.integers(0, 1 << 17, 105), B.rope_freqs(rotary, kind="linear", factor=2.0)
    B.kv_append(cache, d, d, ints(pages), ints(lens), ints(off), ints(pos), dev(f), interleaved=interleaved, mscale=1.1)
    turned, tol = okv.rope(x, pos, f, interleaved, 1.1), rope_tol(x, pos, f, interleaved, 1.1)
    k, ks = of8.decode(host(cache.k)), host(cache.k_scale)
    for s, i, p in okv.rows_of(off, lens, 105):
        page = pages[s, p // 64]
        got = k[page, :, p % 64, :dim] * ks[page][:, None]
        step = np.maximum(np.abs(turned[i]) + tol[i], 2.0 ** -6 * ks[page][:, None]) * 2.0 ** -4
        assert np.all(np.abs(got - turned[i]) <= step + tol[i])
        assert np.all(k[page, :, p % 64, dim:] == 0.0)
    want = okv.empty(count, 2, dim)
    okv.append(want, turned, x, pages, lens, off)
    assert np.array_equal(host(cache.k_scale)[pages[0, 0]], want["k_scale"][pages[0, 0]])
    assert np.array_equal(host(cache.v_scale), want["v_scale"])


def test_append_one_token_a_sequence_and_growth():
    rng = np.random.default_rng(12)
    lens = np.array([1, 64, 65, 130, 17], dtype=np.int32)
    pages, _, count = batch(rng, lens + 20, [1] * 5)
    want = filled(rng, count, 2, 48)
    cache = on_device(want)
    for step in range(20):                                               # each token twice as large as the one before
        x, d = rounded(rng.standard_normal((5, 2, 48)) * 2.0 ** (step - 9), torch.bfloat16)
        okv.append(want, x, -x, pages, lens, None)
        B.kv_append(cache, d, -d, ints(pages), ints(lens))
        same_cache(cache, want, 48)
        lens = lens + 1


def test_append_infinities_and_nan():
    rng = np.random.default_rng(13)
    x, _ = rounded(rng.standard_normal((70, 1, 32)), torch.float32)
    x[3, 0, 4], x[3, 0, 5], x[66, 0, 0] = np.inf, -np.inf, np.nan
    x[5, 0] = 3e38
    x[69, 0] = 1e-42
    pages, off, count = batch(rng, [70], [70])
    want, cache = okv.empty(count, 1, 32), B.kv_cache(count, 1, 32)
    okv.append(want, x, x, pages, [70], off)
    B.kv_append(cache, dev(x, torch.float32), dev(x, torch.float32), ints(pages), ints([70]), ints(off))
    same_cache(cache, want, 32)


def test_append_leaves_out_what_has_no_place():
    """Pages outside the cache, positions before 0 and past the table, rows of no sequence."""
    rng = np.random.default_rng(14)
    lens, off = [130, 200, 3, -4], [0, 130, 140, 147, 149]               # the third: 7 rows of 3 positions
    pages = np.array([[0, 9, 2, -1], [3, 4, 1 << 30, -1], [5, -1, -1, -1], [6, 6, 6, 6]], dtype=np.int32)[:, :3]
    want = filled(rng, 9, 2, 64)
    cache = on_device(want)
    x, d = rounded(rng.standard_normal((160, 2, 64)), torch.float16)
    okv.append(want, x, x, pages, lens, off)
    B.kv_append(cache, d, d, ints(pages), ints(lens), ints(off))
    same_cache(cache, want, 64)
    wide = torch.full((4, 50), 7, dtype=torch.int32, device=DEV)          # a row of a wider table
    wide[:, :3] = ints(pages)
    B.kv_append(cache, d, d, wide[:, :3], ints(lens), ints(off))
    same_cache(cache, want, 64)
    B.kv_append(cache, d, d, ints(pages), ints(lens), ints([-5, -1, 0, 0, 0]))   # nothing
    same_cache(cache, want, 64)


# ------------------------------------------------------------------ attention

def attention_tol(mag, most, small, dp, length, dtype):
    e = (2 * dp + 16) * 2.0 ** -23 * most[..., None]
    p = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -11
    return (2 * e + 2.0 ** -21 + p + (66 + length / 16) * 2.0 ** -22) * mag + small * (1 if dtype == torch.float32 else 16)


WIDE = 8192      # pages of a table for which a few rows are taken in tiles of 128 queries, in parts


def widened(pages, width):
    """The table with columns of no page behind the others."""
    return np.pad(pages, ((0, 0), (0, max(0, width - pages.shape[1]))), constant_values=-1)


def check_attention(rng, lens, news, heads, kv, dim, dtype, window=0, scale=None, cache=None, pages=None, count=None, q=None, off=None, width=0):
    if pages is None:
        pages, off, count = batch(rng, lens, news)
    pages = widened(pages, width)
    cache = cache or filled(rng, count, kv, dim)
    tokens = int(off[-1])
    q, d = rounded(rng.standard_normal((tokens, heads, dim)), dtype) if q is None else rounded(q, dtype)
    out = torch.full((tokens, heads, dim), 77.0, dtype=dtype, device=DEV)
    got = B.kv_attention(d, on_device(cache), ints(pages), ints(lens), ints(off), scale=scale, window=window, out=out)
    ref, mag, most, small = okv.attention(q, cache, pages, lens, off, scale, window)
    rows = ~np.isnan(ref).any((1, 2))
    tol = attention_tol(mag, most, small, okv.padded_dim(dim), max(max(lens), 1), dtype)
    check(host(got)[rows], ref[rows], tol[rows], dtype, f"{lens} {news} {heads}/{kv} x {dim}")
    assert np.all(host(got)[~rows] == 77.0)
    return host(got), ref


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv,dim", [(1, 1, 64), (12, 4, 26), (8, 2, 128), (4, 4, 80), (3, 1, 96), (34, 2, 32),
                                          (2, 1, 192), (4, 1, 256), (1, 1, 1)])
@pytest.mark.parametrize("lens,news", [([1], [1]), ([64], [1]), ([65], [1]), ([300, 1, 64, 129, 0, 63], [1, 1, 1, 1, 0, 1])])
def test_attention_decode(lens, news, heads, kv, dim, dtype):
    check_attention(np.random.default_rng(sum(lens) + dim), lens, news, heads, kv, dim, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [0, 1, 50, 64])
@pytest.mark.parametrize("heads,kv,dim", [(6, 2, 26), (4, 1, 128), (2, 2, 64), (20, 1, 32)])
@pytest.mark.parametrize("lens,news", [([70], [70]), ([200, 64, 9, 130], [5, 64, 0, 67]), ([260], [3])])
@pytest.mark.parametrize("width", [0, WIDE])
def test_attention_of_several_rows(lens, news, heads, kv, dim, window, width, dtype):
    check_attention(np.random.default_rng(sum(lens) + dim + window), lens, news, heads, kv, dim, dtype, window, width=width)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv,dim,lens,news,window", [
    (8, 2, 128, [5000], [1], 0), (4, 1, 64, [3000, 100, 4097], [1, 1, 1], 1000), (8, 8, 128, [1500], [200], 0),
    (4, 1, 128, [700, 900], [600, 300], 0), (16, 2, 128, [2100], [64], 300), (3, 3, 26, [600], [600], 0),
    (4, 2, 96, [1100], [260], 0), (2, 1, 192, [900], [257], 0), (2, 1, 256, [700], [300], 100)])
@pytest.mark.parametrize("width", [0, WIDE])
def test_attention_of_long_sequences(heads, kv, dim, lens, news, window, width, dtype):
    rng = np.random.default_rng(sum(lens))
    q = rng.standard_normal((sum(news), heads, dim)) * np.exp(rng.standard_normal((sum(news), heads, 1)))
    check_attention(rng, lens, news, heads, kv, dim, dtype, window, q=q, width=width)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,window", [(32, 0), (26, 70), (128, 0)])
def test_attention_of_many_sequences(dim, window, dtype):
    """Tiles of 128 queries without parts: 64 sequences of 0 .. 40 rows, some of one or none."""
    rng = np.random.default_rng(dim)
    news = rng.integers(0, 41, 64)
    news[:3] = 0, 1, 40
    lens = [int(n + rng.integers(0, 300)) for n in news]
    check_attention(rng, lens, news.tolist(), 16, 8, dim, dtype, window, width=16)


@pytest.mark.parametrize("width", [0, WIDE])
def test_attention_rows_without_positions_are_zero(width):
    rng = np.random.default_rng(21)
    pages = np.array([[-1, 3], [2, 99], [-1, -1], [4, 5]], dtype=np.int32)
    lens, off = [100, 100, 64, 2], np.array([0, 70, 75, 78, 84], dtype=np.int32)  # the last: 6 rows of 2 positions
    got, ref = check_attention(rng, lens, None, 4, 2, 64, torch.bfloat16, pages=pages, off=off, count=6, width=width)
    assert np.all(got[:34] == 0.0) and np.all(got[75:78] == 0.0) and np.all(got[78:82] == 0.0)


def test_attention_leaves_rows_of_no_sequence():
    rng = np.random.default_rng(22)
    pages, _, count = batch(rng, [80, 90], [1, 1])
    cache = filled(rng, count, 2, 64)
    q, d = rounded(rng.standard_normal((40, 2, 64)), torch.float16)
    for off, width in (([3, 5, 30], 0), ([3, 25, 30], 0), ([3, 25, 30], WIDE)):
        pages = widened(pages, width)
        out = torch.full((40, 2, 64), -3.0, dtype=torch.float16, device=DEV)
        B.kv_attention(d, on_device(cache), ints(pages), ints([80, 90]), ints(off), out=out)
        ref, mag, most, small = okv.attention(q, cache, pages, [80, 90], off)
        rows = ~np.isnan(ref).any((1, 2))
        assert np.array_equal(np.nonzero(rows)[0], np.arange(3, 30))
        check(host(out)[rows], ref[rows], attention_tol(mag, most, small, 64, 90, torch.float16)[rows], torch.float16)
        assert np.all(host(out)[~rows] == -3.0)


@pytest.mark.parametrize("width", [0, WIDE])
@pytest.mark.parametrize("news,window", [(1, 0), (1, 30), (40, 0), (150, 40), (200, 0)])
def test_attention_ignores_what_is_masked(news, window, width):
    """NaN codes past the end, before the window and ahead of a row; slots after the end hold whatever they did."""
    rng = np.random.default_rng(news + window)
    length = 200
    pages, off, count = batch(rng, [length], [news])
    pages = widened(pages, width)
    clean = filled(rng, count, 2, 64)
    q = rng.standard_normal((news, 4, 64))
    base, _ = check_attention(rng, [length], [news], 4, 2, 64, torch.bfloat16, window, cache=clean, pages=pages, off=off, q=q)
    dirty = {n: a.copy() for n, a in clean.items()}
    last, mid = pages[0, 3], pages[0, 1]
    dirty["k"][last, :, 8:], dirty["v"][last, :, :, 8:] = 0x7F, 0xFF      # positions from 200 on
    for p in range(count):
        if p not in pages:
            dirty["k"][p], dirty["v"][p], dirty["k_scale"][p] = 0x7F, 0x7F, np.nan
    first = length - news - window + 1 if window else 0
    if window and first > 64:                                            # before every row's window
        dirty["k"][pages[0, 0]], dirty["v"][pages[0, 0]] = 0x7F, 0x7F
        dirty["v_scale"][pages[0, 0]] = np.nan
    got, _ = check_attention(rng, [length], [news], 4, 2, 64, torch.bfloat16, window, cache=dirty, pages=pages, off=off, q=q)
    assert np.array_equal(got, base)
    if news < 2:
        return
    # a key and a value that only the rows from its position on (within the window) see
    at = length - news // 2
    page, slot = pages[0, at // 64], at % 64
    for name in ("k", "v"):
        spoiled = {n: a.copy() for n, a in clean.items()}
        if name == "k":
            spoiled["k"][page, 0, slot, 3] = 0x7F
        else:
            spoiled["v"][page, 0, 3, slot] = 0xFF
        _, d = rounded(q, torch.bfloat16)
        got = host(B.kv_attention(d, on_device(spoiled), ints(pages), ints([length]), ints(off), window=window))
        pos = length - news + np.arange(news)
        sees = (pos >= at) & ((pos < at + window) if window else True)
        heads, cols = slice(0, 2), slice(None) if name == "k" else 3      # heads 0 and 1 read head 0 of the cache
        assert np.all(np.isnan(got[sees][:, heads][..., cols])), name
        got[sees, heads, cols] = base[sees, heads, cols] if name == "v" else base[sees][:, heads]
        assert np.array_equal(got, base), name


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news,width", [(3, 0), (40, WIDE)])
def test_attention_of_a_row_that_is_not_finite(news, width, dtype):
    rng = np.random.default_rng(5)
    pages, off, count = batch(rng, [100], [news])
    pages = widened(pages, width)
    cache = filled(rng, count, 2, 32)
    _, d = rounded(rng.standard_normal((news, 4, 32)), dtype)
    base = host(B.kv_attention(d, on_device(cache), ints(pages), ints([100]), ints(off)))
    d[0, 1, 5], d[2, 3, 0] = float("inf"), float("nan")
    got = host(B.kv_attention(d, on_device(cache), ints(pages), ints([100]), ints(off)))
    assert np.all(np.isnan(got[0, 1])) and np.all(np.isnan(got[2, 3]))
    got[0, 1], got[2, 3] = base[0, 1], base[2, 3]
    assert np.array_equal(got, base)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news,width", [(1, 0), (90, 0), (90, WIDE)])
def test_attention_of_far_scales(news, width, dtype):
    """Pages whose scales are 2^40 apart, in keys (a softmax of one key) and in values."""
    rng = np.random.default_rng(31)
    lens = [700]
    pages, off, count = batch(rng, lens, [news])
    pages = widened(pages, width)
    cache = filled(rng, count, 2, 64)
    cache["v_scale"][:] = 2.0 ** rng.integers(-60, 60, cache["v_scale"].shape) if dtype != torch.float16 else 2.0 ** rng.integers(-30, 3, cache["v_scale"].shape)
    cache["k_scale"][:] = 2.0 ** rng.integers(-40, -6, cache["k_scale"].shape)
    check_attention(rng, lens, [news], 4, 2, 64, dtype, cache=cache, pages=pages, off=off)
    q = rng.standard_normal((news, 4, 64)) * 2.0 ** rng.integers(-30, 5, (news, 4, 1))
    check_attention(rng, lens, [news], 4, 2, 64, dtype, cache=cache, pages=pages, off=off, scale=0.7, q=q)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("large", [0, 1, 2])
@pytest.mark.parametrize("width", [0, WIDE])
def test_attention_of_a_page_near_the_largest_number(width, large, window, dtype):
    """Rows that do not see the page keep their sums, 2^157 smaller, as they are."""
    rng = np.random.default_rng(36)
    lens, news = [200], [150]
    pages, off, count = batch(rng, lens, news)
    cache = filled(rng, count, 2, 64)
    cache["v_scale"][:] = 2.0 ** -50
    cache["v_scale"][pages[0, large]] = 2.0 ** 107
    check_attention(rng, lens, news, 4, 2, 64, dtype, window, cache=cache, pages=pages, off=off, width=width)


@pytest.mark.parametrize("width", [0, WIDE])
def test_attention_of_shared_pages(width):
    """Two sequences whose first pages are the same, and a page that a table names twice."""
    rng = np.random.default_rng(34)
    lens, news = [150, 200, 192], [20, 77, 30]
    pages, off, count = batch(rng, lens, news)
    pages[1, :2] = pages[0, :2]
    pages[2, 2] = pages[2, 0]
    check_attention(rng, lens, news, 4, 2, 64, torch.bfloat16, pages=pages, off=off, count=count, width=width)


@pytest.mark.parametrize("width", [0, WIDE])
def test_attention_of_many_heads_to_one(width):
    rng = np.random.default_rng(35)
    check_attention(rng, [70, 9, 130], [3, 0, 2], 200, 1, 32, torch.float16, width=width)
    check_attention(rng, [70, 9, 130], [1, 1, 1], 260, 2, 26, torch.bfloat16, width=width)


@pytest.mark.parametrize("width", [0, WIDE])
def test_attention_strided_queries(width):
    rng = np.random.default_rng(33)
    lens, news = [150, 77], [20, 77]
    pages, off, count = batch(rng, lens, news)
    pages = widened(pages, width)
    cache = on_device(filled(rng, count, 2, 80))
    wide = torch.randn(97, 9, 81, device=DEV).half()
    args = (cache, ints(pages), ints(lens), ints(off))
    want = B.kv_attention(wide[:, 1:5, :80].contiguous(), *args)
    assert torch.equal(B.kv_attention(wide[:, 1:5, :80], *args), want)
    first = wide[:, 1:5, :80].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(B.kv_attention(first, *args), want)


# ------------------------------------------------------------------ as they are used

def test_prompt_then_tokens_as_a_graph():
    """Two prompts, then tokens one by one through a captured step, against attention over the whole in one call
    and against the oracle; other work and a second graph with a workspace of its own between the replays."""
    torch.manual_seed(0)
    rng = np.random.default_rng(40)
    heads, kv, dim, steps = 8, 2, 64, 6
    news = [100, 37]
    f = dev(B.rope_freqs(dim))
    pages, off, count = batch(rng, [n + steps for n in news], news)
    tables = ints(pages)
    qkv = torch.randn(137 + 2 * steps, heads + 2 * kv, dim, device=DEV).bfloat16()
    cache = B.kv_cache(count, kv, dim)

    def step(x, positions, lens, offsets, out=None, workspace=None):
        q = B.rope(x[:, :heads], positions, f)
        B.kv_append(cache, x[:, heads:heads + kv], x[:, heads + kv:], tables, lens, offsets, positions, f)
        return B.kv_attention(q, cache, tables, lens, offsets, out=out, workspace=workspace)

    pos = ints(np.concatenate([np.arange(n) for n in news]))
    step(qkv[:137], pos, ints(news), ints(off))
    x, positions, lens = qkv[137:139].clone(), ints(news), ints(news) + 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = [t.clone() for t in cache]
    with torch.cuda.stream(side):
        step(x, positions, lens, None)
    torch.cuda.current_stream().wait_stream(side)
    for t, s in zip(cache, state):
        t.copy_(s)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(step(x, positions, lens, None))
    for t, s in zip(cache, state):
        t.copy_(s)
    got = []
    for i in range(steps):
        x.copy_(qkv[137 + 2 * i:139 + 2 * i])
        graphs[i % 2].replay()
        got.append(outs[i % 2].clone())
        torch.cuda.synchronize()
        (qkv.float() @ qkv.float().transpose(1, 2)).sum()                # the program's own work between
        graphs[i % 2].replay()                                           # the same tokens again: the same result
        assert torch.equal(outs[i % 2], got[-1])
        positions += 1
        lens += 1
    # the oracle reads the cache that the steps wrote
    held = {"k": host(cache.k), "v": host(cache.v), "k_scale": host(cache.k_scale), "v_scale": host(cache.v_scale)}
    q = host(B.rope(qkv[137 + 2 * steps - 2:, :heads], positions - 1, f))
    ref, mag, most, small = okv.attention(q, held, pages, [n + steps for n in news])
    check(host(got[-1]), ref, attention_tol(mag, most, small, 64, 120, torch.bfloat16), torch.bfloat16)
    # an eager call on a stream of its own
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.current_stream())
        again = B.kv_attention(B.rope(x[:, :heads], positions - 1, f), cache, tables, lens - 1)
    side.synchronize()
    assert torch.equal(again, got[-1])


@pytest.mark.parametrize("seqs,most", [(65, 3), (128, 40), (1000, 2), (4097, 1), (4200, 3)])
def test_many_sequences(seqs, most):
    """Workgroups find their sequence among many, with ones without rows between, at the start and at the end."""
    rng = np.random.default_rng(seqs)
    news = rng.integers(0, most + 1, seqs)
    news[[0, 1, -1, seqs // 2]] = 0
    news[2] = most
    lens = (news + rng.integers(0, 70, seqs)).tolist()
    pages, off, count = batch(rng, lens, news)
    want = filled(rng, count, 1, 32)
    cache = on_device(want)
    x, d = rounded(rng.standard_normal((int(off[-1]), 1, 32)), torch.bfloat16)
    okv.append(want, x, -x, pages, lens, off)
    B.kv_append(cache, d, -d, ints(pages), ints(lens), ints(off))
    same_cache(cache, want, 32)
    some = rng.permutation(np.flatnonzero(news))[:40].tolist() + [2]
    got = host(B.kv_attention(d, cache, ints(pages), ints(lens), ints(off)))
    for s in some:
        rows = slice(off[s], off[s + 1])
        ref, mag, most_, small = okv.attention(x[rows], want, pages[s:s + 1], [lens[s]], [0, int(news[s])])
        check(got[rows], ref, attention_tol(mag, most_, small, 32, lens[s], torch.bfloat16), torch.bfloat16, f"sequence {s}")
    assert np.all(np.isfinite(got))


def test_windows_as_large_as_integers():
    rng = np.random.default_rng(60)
    lens, news = [300, 40], [100, 40]
    pages, off, count = batch(rng, lens, news)
    cache, q = on_device(filled(rng, count, 2, 64)), torch.randn(140, 4, 64, device=DEV).bfloat16()
    for width in (0, WIDE):
        args = (q, cache, ints(widened(pages, width)), ints(lens), ints(off))
        want = B.kv_attention(*args)
        for window in (300, 2 ** 30, 2 ** 31 - 1):
            got, ref = host(B.kv_attention(*args, window=window)), host(want)
            # other parts, other orders of the same sums: a step of bf16 at most
            assert np.all(np.abs(got - ref) <= 2.0 ** -7 * np.abs(ref) + 2.0 ** -12)


def test_codes_past_32_bits():
    """Pages whose codes begin past 2^32 bytes hold and give what the same pages of a small cache do."""
    rng = np.random.default_rng(61)
    heads, dim, far = 8, 128, 70000                                       # 64 KiB a page
    lens, news = [200, 130], [200, 130]
    pages, off, count = batch(rng, lens, news)
    small, large = B.kv_cache(count, heads, dim), B.kv_cache(far + count, heads, dim)
    k, v, q = (torch.randn(330, heads, dim, device=DEV).bfloat16() for _ in range(3))
    pos, f = ints(np.concatenate([np.arange(n) for n in news])), dev(B.rope_freqs(dim))
    out = []
    for cache, shift in ((small, 0), (large, far)):
        table = ints(np.where(pages >= 0, pages + shift, -1))
        B.kv_append(cache, k, v, table, ints(lens), ints(off), pos, f)
        out.append([B.kv_attention(q, cache, ints(widened(table.cpu().numpy(), w)), ints(lens), ints(off)) for w in (0, WIDE)])
        out[-1].append(B.kv_attention(q[:2], cache, table, ints(lens)))
    for a, b in zip(*out):
        assert torch.equal(a, b)
    for a, b in zip(small, large):
        assert torch.equal(a.view(torch.uint8) if a.dtype == F8 else a, (b.view(torch.uint8) if b.dtype == F8 else b)[far:])
    assert not large.k[:far].view(torch.uint8).any() and not large.v[:far].view(torch.uint8).any()


def test_graphs_that_share_a_workspace():
    """Two captured calls of unlike sizes with one workspace, replayed in turn with eager work between."""
    rng = np.random.default_rng(51)
    calls = []
    for lens, news in (([5000, 300], [1, 1]), ([900, 2000, 70], [60, 1, 70])):
        pages, off, count = batch(rng, lens, news)
        calls.append((torch.randn(sum(news), 8, 128, device=DEV).bfloat16(), on_device(filled(rng, count, 2, 128)),
                      ints(widened(pages, 3000)), ints(lens), ints(off)))
    want = [B.kv_attention(*c) for c in calls]
    need = max(B.kv_attention_workspace(c[0].shape[0], c[2].shape[0], 8, 2, 128, 3000) for c in calls)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in calls], []
    for g, c in zip(graphs, calls):
        with torch.cuda.graph(g):
            outs.append(B.kv_attention(*c, workspace=ws))
    for i in range(6):
        outs[i % 2].zero_()
        graphs[i % 2].replay()
        assert torch.equal(outs[i % 2], want[i % 2])
        assert torch.equal(B.kv_attention(*calls[i % 2], workspace=ws), want[i % 2])


def test_attention_given_workspace_and_refusals():
    rng = np.random.default_rng(50)
    lens = [20000]
    pages, off, count = batch(rng, lens, [1])
    cache, q = on_device(filled(rng, count, 2, 128)), torch.randn(1, 8, 128, device=DEV)
    want = B.kv_attention(q, cache, ints(pages), ints(lens))
    need = B.kv_attention_workspace(1, 1, 8, 2, 128, pages.shape[1])
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device=DEV)
    for _ in range(2):                                                   # whatever the workspace holds
        assert torch.equal(B.kv_attention(q, cache, ints(pages), ints(lens), workspace=ws), want)
    if need:
        with pytest.raises(ValueError, match="workspace"):
            B.kv_attention(q, cache, ints(pages), ints(lens), workspace=ws[:need - 1])
    with pytest.raises(ValueError, match="Float8_e4m3fn"):
        B.kv_attention(q, cache._replace(k=cache.k.view(torch.uint8)), ints(pages), ints(lens))
    with pytest.raises(ValueError, match="pages must be Int"):
        B.kv_attention(q, cache, ints(pages).long(), ints(lens))
    with pytest.raises(ValueError, match="out must"):
        B.kv_attention(q, cache, ints(pages), ints(lens), out=q[:, :4])
