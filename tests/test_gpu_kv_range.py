"""The attention over the 8-bit cache at the ends of its range, and how many bits its probabilities hold.

``sharp`` is the attention's bound with probabilities of 22 bits (two fp16 terms): with e as in test_gpu_kv.py, out is off by at most
    (2 e + 2^-21 + 2^-22 + (66 + L / 16) 2^-22) sum p |v| + 2^-40 sum |v|.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_quantized_matmul_amd import binding as B
from oracle import fp8 as of8
from oracle import kv as okv
from tests.test_gpu_kv import DEV, F8, TYPES, WIDE, attention_tol, batch, check, check_attention, dev, filled, host, ints, on_device, rounded, widened

pytestmark = pytest.mark.gpu


def sharp(mag, most, small, dp, length, dtype):
    return attention_tol(mag, most, small / (1 if dtype == torch.float32 else 16), dp, length, dtype) - (0 if dtype == torch.float32 else (2.0 ** -11 - 2.0 ** -22) * mag)


# ------------------------------------------------------------------ masked scales, far parts

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
@pytest.mark.parametrize("news,window", [(10, 0), (10, 40), (150, 0), (150, 30)])
@pytest.mark.parametrize("width", [0, WIDE])
def test_scales_of_pages_that_only_some_rows_see(width, news, window, which, bad, dtype):
    """A page with a scale that is not finite beside rows of the same tile that end before it or begin after it."""
    rng = np.random.default_rng(news + window)
    length, heads, kv, dim = 198, 4, 2, 64
    pages, off, count = batch(rng, [length], [news])
    pages = widened(pages, width)
    clean = filled(rng, count, kv, dim)
    q = rng.standard_normal((news, heads, dim))
    base, _ = check_attention(rng, [length], [news], heads, kv, dim, dtype, window, cache=clean, pages=pages, off=off, q=q)
    _, d = rounded(q, dtype)
    pos = length - news + np.arange(news)
    for page in range(4):
        spoiled = {n: a.copy() for n, a in clean.items()}
        spoiled[which][pages[0, page], 1] = bad                          # read by heads 2 and 3
        got = host(B.kv_attention(d, on_device(spoiled), ints(pages), ints([length]), ints(off), window=window))
        sees = (pos >= 64 * page) & ((pos - window < 64 * page + 63) if window else True)
        assert np.array_equal(got[:, :2], base[:, :2]) and np.array_equal(got[~sees], base[~sees])
        gone = ~np.isfinite(got[sees][:, 2:])
        assert gone.all() or which == "k_scale" and bad == float("inf")   # scores of -inf beside +inf may leave one key


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news,heads,kv,width", [(1, 4, 2, 64), (1, 1, 1, 2000), (40, 4, 2, 2000), (200, 4, 1, 64)])
def test_nan_values_of_far_scores(news, heads, kv, width, dtype):
    """A NaN value whose probability is below fp32's numbers is attended to all the same: its column is NaN, also where its
    page is in another part than the row's largest score."""
    rng = np.random.default_rng(width + news)
    dim, length = 64, 64 * 40 + news
    pages, off, count = batch(rng, [length], [news])
    pages = widened(pages, width)
    cache = okv.empty(count, kv, dim)
    cache["v"][:] = of8.encode(rng.standard_normal(cache["v"].shape))
    cache["k_scale"][:], cache["v_scale"][:] = 1.0, 1.0
    near, far = pages[0, 3], pages[0, 30]
    cache["k"][..., 0] = of8.encode(-448.0)                              # scores of -448 and, on page 3, of 0
    cache["k"][near, ..., 0] = 0
    q = np.zeros((news, heads, dim))
    q[..., 0] = 1.0
    args = (rounded(q, dtype)[1], ints(pages), ints([length]), ints(off))
    run = lambda c: host(B.kv_attention(args[0], on_device(c), *args[1:], scale=1.0))   # noqa: E731
    base = run(cache)
    assert np.all(np.isfinite(base))
    cache["v"][far, :, 5, 17] = 0x7F
    got = run(cache)
    assert np.all(np.isnan(got[..., 5]))
    keep = np.arange(dim) != 5
    assert np.array_equal(got[..., keep], base[..., keep])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rise", [[0, 0, 0, 3.97, 3.97, 3.97, 3.97, 3.97], [0, 3.97, 7.9, 8, 11.5, 11.5, 15, 16], [0, 0, 0, 0, 0, 0, 0, 3.97]])
@pytest.mark.parametrize("news,width", [(1, 0), (1, 2000), (130, 0), (130, WIDE)])
def test_values_at_the_limit_with_rising_scores(news, width, rise, dtype):
    """Values times positions just below fp32's largest number, all of one sign, and scores that rise by up to 4 a page in the
    base of two: as far as the tiles' maxima may lag behind."""
    rng = np.random.default_rng(70)
    length, dim = 64 * 8, 32
    pages, off, count = batch(rng, [length], [news])
    pages = widened(pages, width)
    cache = okv.empty(count, 1, dim)
    order = pages[0, :8]
    cache["v"][:] = of8.encode(448.0)
    cache["v_scale"][:] = 2.0 ** 110                                     # 448 x 2^110 x 512 = 1.75 x 2^127
    cache["k_scale"][:] = 1.0
    cache["k"][order, 0, :, 0] = of8.encode(np.log(2.0) * np.array(rise, dtype=np.float64))[:, None]
    q = np.zeros((news, 2, dim))
    q[..., 0] = rng.uniform(0.9, 1.0, (news, 2))
    run = lambda: check_attention(rng, [length], [news], 2, 1, dim, dtype, scale=1.0, cache=cache, pages=pages, off=off, q=q)   # noqa: E731
    run()
    cache["v_scale"][order[::2]] = 2.0 ** -40                            # and beside the smallest units
    run()
    cache["v_scale"][order, 0] = 2.0 ** np.array([15.0, -40, 15, 16, 17, -41, 110, -126])
    run()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("exponent", [0, 17, 20, 26, 60, 115])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("news,width,window", [(1, 0, 0), (1, 2000, 0), (150, 0, 0), (150, 0, 30), (150, WIDE, 0), (150, WIDE, 30)])
def test_scores_far_past_their_differences(news, width, window, sign, exponent, dtype):
    """Scores of up to 448 x 2^exponent, whose steps in fp32 are larger than a probability's whole range: one column of keys, so that
    they are exact.  All weight is on a row's largest, or shared among equal ones."""
    rng = np.random.default_rng(exponent)
    length, dim, heads, kv = 300, 32, 4, 2
    pages, off, count = batch(rng, [length], [news])
    pages = widened(pages, width)
    cache = okv.empty(count, kv, dim)
    cache["k"][..., 0] = rng.choice([0x7E, 0x7C, 0x76, 0x30, 0xF0, 0xFE], cache["k"][..., 0].shape, p=[0.02, 0.08, 0.2, 0.3, 0.2, 0.2])
    cache["v"][:] = of8.encode(rng.integers(-8, 9, cache["v"].shape))
    cache["k_scale"][:], cache["v_scale"][:] = 1.0, 1.0
    q = np.zeros((news, heads, dim))
    q[..., 0] = sign * 2.0 ** rng.integers(0, 2, (news, heads))
    _, d = rounded(q, dtype)
    got = host(B.kv_attention(d, on_device(cache), ints(pages), ints([length]), ints(off), scale=16.0 * 2.0 ** (exponent - 8), window=window))
    for i in range(news):
        for h in range(heads):
            k, v, _ = okv.values(cache, pages, 0, length, h // 2, dim)
            j = np.arange(length)
            p = length - news + i
            see = (j <= p) & ((j > p - window) if window else True)
            s = 16.0 * 2.0 ** (exponent - 8) * k[see, 0] * q[i, h, 0]
            e = np.exp(s - s.max())
            e /= e.sum()
            want, mag = e @ v[see], e @ np.abs(v[see])
            # scores are exact; times log2(e) their differences, below 100 where they count, are off by 2^-23 of them.  p is off by up to
            # 2^-11 of it where it is one term: sum p d (v - o), |d| <= 2^-11, is at most 2^-11 (sum p |v| + |o|) <= 2^-10 sum p |v|
            t = (2.0 ** -10 + 2.0 ** -16) * mag + 2.0 ** -36 * np.abs(v[see]).sum(0)
            # and half a step of the type, below its normal numbers too
            half = torch.finfo(dtype).eps / 2 * np.maximum(np.abs(want) + t, torch.finfo(dtype).smallest_normal)
            assert np.all(np.abs(got[i, h] - want) <= t + half), (i, h)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news,width", [(1, 0), (1, 2000), (150, 0), (150, WIDE)])
@pytest.mark.parametrize("low", [[0], [1], [0, 1, 3]])
def test_scores_below_fp32_beside_others(low, news, width, dtype):
    """Pages whose scores are below -2^128 weigh nothing, also as a row's first; a row that sees no other key is not looked at."""
    rng = np.random.default_rng(news)
    length, dim = 250, 32
    pages, off, count = batch(rng, [length], [news])
    pages = widened(pages, width)
    cache = okv.empty(count, 1, dim)
    cache["k"][pages[0, low], ..., 0] = of8.encode(-448.0)               # times 2^125
    cache["v"][:] = of8.encode(rng.integers(-8, 9, cache["v"].shape))
    cache["k_scale"][:], cache["v_scale"][:] = 1.0, 1.0
    q = np.zeros((news, 2, dim))
    q[..., 0] = 1.0
    _, d = rounded(q, dtype)
    got = host(B.kv_attention(d, on_device(cache), ints(pages), ints([length]), ints(off), scale=2.0 ** 125))
    k, v, _ = okv.values(cache, pages, 0, length, 0, dim)
    for i in range(news):
        see = (np.arange(length) <= length - news + i) & (k[:, 0] == 0.0)
        if not see.any():
            continue
        want, mag = v[see].mean(0), np.abs(v[see]).mean(0)
        t = 2.0 ** -18 * mag                                             # equal probabilities, exact; their sums and the quotient
        assert np.all(np.abs(got[i] - want) <= t + torch.finfo(dtype).eps / 2 * (np.abs(want) + t)), i


# ------------------------------------------------------------------ bits of the probabilities

def cancelling(rng, count, kv, dim):
    """Neighbouring tokens' values are each other's negatives, and their keys alike but for one column."""
    cache = filled(rng, count, kv, dim)
    cache["v"][..., 1::2] = cache["v"][..., 0::2] ^ 0x80
    cache["k"][..., 1::2, :] = cache["k"][..., 0::2, :]
    cache["k"][..., 1::2, 0] = of8.encode(0.0)
    cache["k"][..., 0::2, 0] = of8.encode(448.0)
    cache["k_scale"][:], cache["v_scale"][:] = 2.0 ** -9, 1.0
    return cache


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,heads,kv", [(32, 6, 2), (128, 4, 1), (80, 8, 8), (256, 2, 1)])
@pytest.mark.parametrize("length,news", [(20, 1), (64, 1), (40, 3), (2000, 1)])
def test_probabilities_of_few_rows_hold_22_bits(length, news, dim, heads, kv, dtype):
    """Values of both signs that nearly cancel, so that a result is as small as the errors of its probabilities: half a step of the
    result's type hides none of them."""
    rng = np.random.default_rng(length + dim)
    pages, off, count = batch(rng, [length], [news])
    cache = cancelling(rng, count, kv, dim)
    q = 0.05 * rng.standard_normal((news, heads, dim))
    q[..., 0] = 0.02
    q, d = rounded(q, dtype)
    got = B.kv_attention(d, on_device(cache), ints(pages), ints([length]), ints(off))
    ref, mag, most, small = okv.attention(q, cache, pages, [length], off)
    check(host(got), ref, sharp(mag, most, small, okv.padded_dim(dim), length, dtype), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,news,width", [(192, 8, 100), (256, 16, 100), (160, 5, 100)])
def test_wide_heads_of_few_rows_hold_22_bits(dim, news, width, dtype):
    """Past 128 columns a few rows of many sequences are no work for tiles of 128 queries: probabilities hold 22 bits there too."""
    rng = np.random.default_rng(dim)
    seqs, heads, kv = 64, 8, 2
    lens = rng.integers(news, 41, seqs).tolist()
    pages, off, count = batch(rng, lens, [news] * seqs)
    pages = widened(pages, width)
    cache = cancelling(rng, count, kv, dim)
    q = 0.05 * rng.standard_normal((news * seqs, heads, dim))
    q[..., 0] = 0.02
    q, d = rounded(q, dtype)
    got = host(B.kv_attention(d, on_device(cache), ints(pages), ints(lens), ints(off)))
    for s in (0, 13, 63):
        rows = slice(off[s], off[s + 1])
        ref, mag, most, small = okv.attention(q[rows], cache, pages[s:s + 1], [lens[s]], [0, news])
        check(got[rows], ref, sharp(mag, most, small, okv.padded_dim(dim), lens[s], dtype), dtype)
    assert np.all(np.isfinite(got))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,window", [(64, 0), (96, 50), (128, 0), (192, 90), (256, 0)])
def test_ragged_prompts_in_both_routes(dim, window, dtype):
    """Sequences of 0 to 200 rows, none and single ones among them, in a narrow table and in one that is wide enough for tiles of
    128 queries whatever the type."""
    rng = np.random.default_rng(dim + 1)
    news = rng.integers(60, 201, 9)
    news[[0, 3, 8]] = 0, 1, 200
    lens = [int(n + rng.integers(0, 200)) for n in news]
    for width in (0, 1000):
        check_attention(rng, lens, news.tolist(), 4, 2, dim, dtype, window, width=width)
