"""The expert layer of few tokens at the ends of its types' ranges, and how many bits its terms hold.

Operands enter the matrix cores as 16-bit terms: x as it is (fp32 in three bf16 terms, 24 bits), hidden rows as two bf16
terms of 16 bits in all (2^-17 of the value) or, for an fp32 x, three.  A product with a code is exact.  ``few``
bounds layers in which a result is the sum of a few products, so that a term left out shows:

* gate and up of one column: up to 3 products of fp32's terms, added with two roundings of 2^-23; else exact.
* silu: 4 x 2^-23 of its own, and 1.28 times the gate's error where the gate is 0.5 to 8 (1 + g (1 - s(g)) <= 1.28); times up
  2^-24 and up's error; the weight of a token's only expert is 1.
* the hidden row's terms: 2^-17, or 2^-24 for fp32; their products with W2's codes exact, n columns in up to 3 n
  products added with 2^-23 each, and the scale and the waves' sums, exact zeros but for one: 2^-23.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_quantized_matmul_amd import binding as B
from oracle import fp8 as of8
from oracle import moe as omoe
from tests.test_gpu_moe_ffn import DEV, F8, TYPES, host, tol, weights
from tests.test_gpu_moe_ffn import check as check_labelled

pytestmark = pytest.mark.gpu


def check(got, ref, t, dtype):
    check_labelled(got, ref, t, dtype, "")


def layer(x, w13, s13, w2, s2, logits, top, dtype):
    """(out, the oracle's, its bound) of codes and scales on the host."""
    d, dl = torch.from_numpy(x).to(dtype), torch.from_numpy(logits).float()
    up = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a)).to(DEV) if t is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV).view(t)  # noqa: E731
    y = B.moe_ffn(d.to(DEV), up(w13, F8), up(s13), up(w2, F8), up(s2), dl.to(DEV), top)
    ref, mag = omoe.ffn(d.double().numpy(), w13, s13, w2, s2, dl.double().numpy(), top)
    return host(y), ref, mag


def codes(rows, cols, values, at=slice(None)):
    """One expert's codes [1, rows, 128 ceil(cols / 128)]: `values` at `at`, zeros elsewhere."""
    m = np.zeros((rows, of8.blocks(cols) * 128))
    m[at] = values
    return of8.encode(m)[None]


def ones(rows, cols, s=1.0):
    return np.full((1, of8.blocks(rows), of8.blocks(cols)), s, dtype=np.float32)


# ------------------------------------------------------------------ range

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hidden", [1, 40, 300])
def test_largest_numbers_in_a_row(hidden, dtype):
    """A row that holds the type's largest numbers, with scales that bring its products back: codes up to 1, so that a
    block's sum of one column stays in fp32 unscaled too."""
    rng = np.random.default_rng(hidden)
    big = torch.finfo(dtype).max
    x = np.zeros((3, hidden))
    x[0, 0], x[1, hidden // 2], x[2, -1] = big, -big, big * (1 - 2.0 ** -7)
    ffn = 20
    w13 = codes(2 * ffn, hidden, rng.choice([-1.0, -0.625, 0.25, 0.5, 1.0], (2 * ffn, hidden)), np.s_[:, :hidden])
    w2 = codes(hidden, ffn, rng.standard_normal((hidden, ffn)), np.s_[:, :ffn])
    got, ref, mag = layer(x, w13, ones(2 * ffn, hidden, 2.0 ** -126), w2, ones(hidden, ffn), np.zeros((3, 1)), 1, dtype)
    check(got, ref, tol(mag, hidden, ffn, 1, dtype), dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_numbers(dtype):
    """Rows and hidden rows of 2^-85, whose last terms lie far below: nothing of them is lost."""
    rng = np.random.default_rng(4)
    hidden, ffn = 300, 140
    q13, s13 = weights(rng, 2, 2 * ffn, hidden)
    q2, s2 = weights(rng, 2, hidden, ffn)
    x = rng.standard_normal((3, hidden)) * 2.0 ** -85
    for up, down in ((85, 0), (40, 90)):
        got, ref, mag = layer(x, q13, (s13 * np.float32(2.0 ** up)).astype(np.float32), q2, (s2 * np.float32(2.0 ** down)).astype(np.float32),
                              rng.standard_normal((3, 2)), 2, dtype)
        assert np.abs(ref).max() > 0.01
        check(got, ref, tol(mag, hidden, ffn, 2, dtype), dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,experts,top,hidden,ffn", [(2, 3, 2, 130, 70), (20, 4, 1, 700, 130)])
def test_sums_of_large_numbers(tokens, experts, top, hidden, ffn, dtype):
    """Rows near the largest number and packed weights of small scales: the sums of a block, codes up to 448, are
    past fp32 before the scale."""
    rng = np.random.default_rng(tokens)
    q13, s13 = weights(rng, experts, 2 * ffn, hidden)
    q2, s2 = weights(rng, experts, hidden, ffn)
    x = rng.uniform(0.25, 0.99, (tokens, hidden)) * rng.choice([-1.0, 1.0], (tokens, hidden)) * 2.0 ** 128
    s13 = np.maximum(s13 * np.float32(2.0 ** -118), np.float32(2.0 ** -126))
    got, ref, mag = layer(x, q13, s13, q2, (s2 * np.float32(2.0 ** -20)).astype(np.float32), rng.standard_normal((tokens, experts)), top, dtype)
    assert np.all(np.isfinite(ref)) and np.abs(ref).max() < 2.0 ** 100
    check(got, ref, tol(mag, hidden, ffn, top, dtype), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ffn", [1, 33, 129])
def test_hidden_rows_near_the_largest_number(ffn, dtype):
    """silu(gate) * up = 0.999 x 2^128, past the nearest bf16 that is finite."""
    x = np.ones((1, 1))
    s13 = ones(2 * ffn, 1, np.float32(np.sqrt(0.999) * 2.0 ** 64))
    w13 = codes(2 * ffn, 1, 1.0, np.s_[:, :1])
    signs = np.where(np.arange(ffn) % 2, -1.0, 1.0) * np.where(np.arange(ffn) % 3, 0.5, 1.0)
    w2 = codes(1, ffn, signs, np.s_[0, :ffn])
    got, ref, mag = layer(x, w13, s13, w2, ones(1, ffn, 2.0 ** -120), np.zeros((1, 1)), 1, dtype)
    assert np.all(np.abs(ref) > 1.0)
    check(got, ref, tol(mag, 1, ffn, 1, dtype), dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_sums_of_large_hidden_rows(dtype):
    rng = np.random.default_rng(5)
    hidden, ffn = 60, 200
    q13, s13 = weights(rng, 2, 2 * ffn, hidden)
    q2, s2 = weights(rng, 2, hidden, ffn)
    x = np.abs(rng.standard_normal((4, hidden))) + 0.5
    got, ref, mag = layer(x, q13, (s13 * np.float32(2.0 ** 58)).astype(np.float32), q2, (s2 * np.float32(2.0 ** -112)).astype(np.float32),
                          rng.standard_normal((4, 2)), 2, dtype)
    assert np.all(np.isfinite(ref)) and np.abs(ref).max() > 1.0
    check(got, ref, tol(mag, hidden, ffn, 2, dtype), dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_what_leaves_fp32_is_nan(dtype):
    """Gates, up rows and hidden rows past fp32: rows of NaN, and the other tokens' as they were."""
    rng = np.random.default_rng(6)
    hidden, ffn = 64, 48
    q13, s13 = weights(rng, 1, 2 * ffn, hidden)
    q2, s2 = weights(rng, 1, hidden, ffn)
    s13 = (s13 * np.float32(2.0 ** 60)).astype(np.float32)
    s2 = (s2 * np.float32(2.0 ** -115)).astype(np.float32)
    x = np.abs(rng.standard_normal((4, hidden))) * 2.0 ** -3
    clean, ref, mag = layer(x, q13, s13, q2, s2, np.zeros((4, 1)), 1, dtype)
    check(clean, ref, tol(mag, hidden, ffn, 1, dtype), dtype)
    x[1] *= 2.0 ** 12                                                    # gate times up is past 2^128
    if dtype != torch.float16:
        x[3] *= 2.0 ** 90                                                # gates and up rows are
    got, _, _ = layer(x, q13, s13, q2, s2, np.zeros((4, 1)), 1, dtype)
    gone = [1] if dtype == torch.float16 else [1, 3]
    rest = [t for t in range(4) if t not in gone]
    assert np.all(np.isnan(got[gone])) and np.array_equal(got[rest], clean[rest])


# ------------------------------------------------------------------ bits

def few(terms, dtype):
    """The bound of a sum of products of hidden values, |terms| their absolute values' sum."""
    n = 2
    inner = 3 * (1.28 + 1.0) + 4 + 0.5 if dtype == torch.float32 else 4 + 0.5
    rows = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -17
    return terms * (inner * 2.0 ** -23 + rows + (3 * n + 1) * 2.0 ** -23) * (1 + 2.0 ** -10)


@pytest.mark.parametrize("dtype", TYPES)
def test_every_term_counts(dtype):
    """out = silu(g) (u1 - u2), hidden rows that nearly cancel: u1 = 15 x / 8, u2 = 14 x / 8.  A second term left out would be 2^-9 of
    the hidden rows, 2^-5 of the result; fp32's third 2^-17, 2^-13 of it."""
    rng = np.random.default_rng(7)
    hidden, tokens = 200, 32
    x = np.zeros((tokens, hidden))
    x[np.arange(tokens), rng.integers(0, hidden, tokens)] = rng.uniform(1.0, 8.0, tokens)
    w13 = codes(4, hidden, np.array([[1.0], [1.0], [1.875], [1.75]]), np.s_[:, :hidden])
    rows = rng.choice([-2.0, 0.5, 1.0, 1.5], hidden)
    w2 = codes(hidden, 2, rows[:, None] * np.array([1.0, -1.0]), np.s_[:, :2])
    got, ref, _ = layer(x, w13, ones(4, hidden), w2, ones(hidden, 2), np.zeros((tokens, 1)), 1, dtype)
    value = torch.from_numpy(x).to(dtype).double().numpy().sum(1)
    a = value / (1 + np.exp(-value)) * value
    terms = a[:, None] * (1.875 + 1.75) * np.abs(rows)
    assert np.allclose(ref, a[:, None] * 0.125 * rows, rtol=1e-12)
    check(got, ref, few(terms, dtype), dtype)


def test_every_term_of_an_fp32_row_counts():
    """One gate of 1 (from a column of ones) and an up row of one fp32 number in its 24 bits."""
    rng = np.random.default_rng(8)
    x = np.zeros((32, 2))
    x[:, 0], x[:, 1] = 1.0, rng.uniform(1.0, 2.0, 32).astype(np.float32)
    w13 = codes(2, 2, np.array([[1.0, 0.0], [0.0, 1.0]]), np.s_[:, :2])
    w2 = codes(2, 1, np.array([[1.0], [1.5]]), np.s_[:, :1])
    got, ref, _ = layer(x, w13, ones(2, 2), w2, ones(2, 1), np.zeros((32, 1)), 1, torch.float32)
    check(got, ref, few(np.abs(ref), torch.float32), torch.float32)
    # the ratio of two tokens' results is the ratio of their numbers: silu's error is the same in both
    ratio, want = got[1:, 0] / got[:-1, 0], x[1:, 1] / x[:-1, 1]
    assert np.max(np.abs(ratio / want - 1)) <= 2 * (2 + 0.5 + 1 + 4 + 1) * 2.0 ** -23
