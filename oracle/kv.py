"""Rotary positions, the paged cache of E4M3 codes and its attention, in 64 bits.

A cache is a dict of numpy arrays: k codes [pages, heads, 64, dp], v codes [pages, heads, dp, 64] (uint8),
k_scale and v_scale [pages, heads].  Scales are powers of two.
"""
from __future__ import annotations

import math

import numpy as np

from . import fp8

PAGE = 64


def padded_dim(dim: int) -> int:
    return next(p for p in (32, 64, 96, 128, 192, 256) if p >= dim)


def rope(x, positions, freqs, interleaved: bool = False, mscale: float = 1.0, backward: bool = False):
    """x [tokens, heads, dim] with its first 2 len(freqs) columns turned, in fp64."""
    y = np.array(x, dtype=np.float64)
    r = 2 * len(freqs)
    a = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freqs, dtype=np.float64)
    c, s = mscale * np.cos(a)[:, None], mscale * np.sin(a)[:, None] * (-1.0 if backward else 1.0)
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    x1, x2 = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = x1 * c - x2 * s, x1 * s + x2 * c
    return y


def scale_for(values) -> float:
    """The smallest power of two, 2^-126 at least, with |finite values| <= 448 times it."""
    v = np.abs(np.asarray(values, dtype=np.float64))
    v = v[np.isfinite(v)]
    s = 2.0 ** -126
    while v.size and v.max() > 448.0 * s:
        s *= 2.0
    return s


def encode(values, scale: float):
    v = np.asarray(values, dtype=np.float64)
    ok = np.isfinite(v)
    with np.errstate(invalid="ignore"):
        return np.where(ok, fp8.encode(np.clip(np.where(ok, v, 0.0) / scale, -448.0, 448.0)), np.uint8(0x7F)).astype(np.uint8)


def empty(pages: int, heads: int, dim: int) -> dict:
    dp = padded_dim(dim)
    return {"k": np.zeros((pages, heads, PAGE, dp), np.uint8), "v": np.zeros((pages, heads, dp, PAGE), np.uint8),
            "k_scale": np.zeros((pages, heads)), "v_scale": np.zeros((pages, heads))}


def rows_of(offsets, lens, tokens: int):
    """(sequence, row, position) of every new token whose position is not negative."""
    for s, length in enumerate(lens):
        lo, hi = (s, s + 1) if offsets is None else (min(max(0, offsets[s]), tokens), min(max(0, offsets[s + 1]), tokens))
        for i in range(lo, hi):
            p = max(0, length) - (hi - lo) + i - lo
            if p >= 0:
                yield s, i, p


def append(cache: dict, k, v, pages, lens, offsets=None) -> None:
    """k (turned already) and v [tokens, heads, dim] into their pages."""
    groups: dict = {}
    for s, i, p in rows_of(offsets, lens, k.shape[0]):
        if p // PAGE < pages.shape[1] and 0 <= pages[s, p // PAGE] < cache["k"].shape[0]:
            groups.setdefault((s, p // PAGE), []).append((i, p % PAGE))
    dim = k.shape[2]
    for (s, pi), new in groups.items():
        page, rows, slots = int(pages[s, pi]), [i for i, _ in new], [t for _, t in new]
        held = slots[0]
        for h in range(k.shape[1]):
            for name, x in (("k", k), ("v", v)):
                codes = cache[name][page, h] if name == "k" else cache[name][page, h].T
                old = cache[name + "_scale"][page, h]
                now = scale_for(x[rows, h])
                if held:
                    now = max(now, old)
                    if now != old:
                        codes[:held, :dim] = encode(np.where(codes[:held, :dim] % 128 == 127, np.nan, fp8.decode(codes[:held, :dim]) * old), now)
                codes[slots, :dim] = encode(x[rows, h], now)
                if name == "k":
                    codes[slots, dim:] = 0
                cache[name + "_scale"][page, h] = now


def values(cache: dict, pages, s: int, length: int, h: int, dim: int):
    """Keys and values [length, dim] of a head of sequence s, and which positions are there."""
    k, v, there = np.zeros((length, dim)), np.zeros((length, dim)), np.zeros(length, bool)
    for pi in range(min(-(-length // PAGE), pages.shape[1])):
        page = int(pages[s, pi])
        if 0 <= page < cache["k"].shape[0]:
            n = min(PAGE, length - pi * PAGE)
            at = slice(pi * PAGE, pi * PAGE + n)
            k[at] = fp8.decode(cache["k"][page, h, :n, :dim]) * float(cache["k_scale"][page, h])
            v[at] = fp8.decode(cache["v"][page, h, :dim, :n]).T * float(cache["v_scale"][page, h])
            there[at] = True
    return k, v, there


def attention(q, cache: dict, pages, lens, offsets=None, scale=None, window: int = 0):
    """(out [tokens, heads, dim], sum of p |v|, the largest sum of |scale q k| that a row sees, 2^-40 sum of |v|); rows of
    no sequence are NaN."""
    q = np.asarray(q, dtype=np.float64)
    tokens, heads, dim = q.shape
    rep = heads // cache["k"].shape[1]
    scale = 1.0 / math.sqrt(dim) if scale is None else scale
    out, mag, most = np.full(q.shape, np.nan), np.zeros(q.shape), np.zeros((tokens, heads))
    small = np.zeros(q.shape)
    for s, length in enumerate(lens):
        lo, hi = (s, s + 1) if offsets is None else (min(max(0, offsets[s]), tokens), min(max(0, offsets[s + 1]), tokens))
        length = max(0, int(length))
        for h in range(heads if hi > lo else 0):
            k, v, there = values(cache, pages, s, length, h // rep, dim)
            for i in range(lo, hi):
                p = length - (hi - lo) + i - lo
                j = np.arange(length)
                see = there & (j <= p) & ((j > p - window) if window else True)
                out[i, h] = 0.0
                if not see.any():
                    continue
                x = scale * (k[see] @ q[i, h])
                e = np.exp(x - x.max())
                e /= e.sum()
                out[i, h] = e @ v[see]
                mag[i, h] = e @ np.abs(v[see])
                small[i, h] = 2.0 ** -40 * np.abs(v[see]).sum(0)
                most[i, h] = np.max(abs(scale) * (np.abs(k[see]) @ np.abs(q[i, h])))
    return out, mag, most, small
