"""E4M3 codes with a scale for each block of 128, and the products on them.

The code values come from the format's definition (sign, 4 exponent bits of bias
7, 3 mantissa bits, no infinity, one NaN a sign); rounding picks the nearer of the
two neighbouring values, the even code on a tie.  ``quant_act`` follows the
library's stated fp32 steps bit for bit; the products are fp64 sums.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
MIN_SCALE = np.float32(2.0 ** -126)


def _values() -> np.ndarray:
    out = np.empty(256, dtype=np.float64)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f / 8.0 * 2.0 ** -6 if e == 0 else (1.0 + f / 8.0) * 2.0 ** (e - 7)
        if e == 15 and f == 7:
            v = np.nan
        out[c] = -v if c & 0x80 else v
    return out


VALUES = _values()
_POS = VALUES[:127]                                  # ascending, 0 .. 448


def encode(x) -> np.ndarray:
    """Nearest E4M3 code of values within [-448, 448] (ties to the even code); NaN -> 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = (pick + np.where(np.signbit(x), 128, 0)).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def decode(codes) -> np.ndarray:
    return VALUES[np.asarray(codes, dtype=np.uint8)]


def blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _scale(amax: np.ndarray) -> np.ndarray:
    """fp32 scales of fp32 block maxima."""
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.maximum((amax / np.float32(E4M3_MAX)).astype(np.float32), MIN_SCALE)
    s = np.where(amax > 0, s, np.float32(1.0))
    return np.where(np.isfinite(amax), s, np.float32(np.nan)).astype(np.float32)


def swiglu64(x) -> np.ndarray:
    """silu(gate) * up of rows [gate | up] in fp64."""
    x = np.asarray(x, dtype=np.float64)
    k = x.shape[1] // 2
    with np.errstate(over="ignore"):
        return x[:, :k] / (1.0 + np.exp(-x[:, :k])) * x[:, k:]


def quant_act(v):
    """fp32 v [m, k] -> (codes [m, 128 kb] uint8, scale [kb, m] fp32)."""
    v = np.asarray(v, dtype=np.float32)
    m, k = v.shape
    kb = blocks(k)
    p = np.zeros((m, kb * BLOCK), dtype=np.float32)
    p[:, :k] = v
    p = p.reshape(m, kb, BLOCK)
    s = _scale(np.max(np.abs(p), axis=2))
    with np.errstate(invalid="ignore", over="ignore"):
        r = np.clip((p / s[..., None]).astype(np.float32), -E4M3_MAX, E4M3_MAX)
    return encode(r).reshape(m, kb * BLOCK), np.ascontiguousarray(s.T)


def quant_weight(w):
    """fp32 w [rows, cols] -> (codes [rows, 128 kb] uint8, scale [ceil(rows/128), kb] fp32)."""
    w = np.asarray(w, dtype=np.float32)
    rows, cols = w.shape
    nb, kb = blocks(rows), blocks(cols)
    p = np.zeros((nb * BLOCK, kb * BLOCK), dtype=np.float32)
    p[:rows, :cols] = w
    p = p.reshape(nb, BLOCK, kb, BLOCK)
    s = _scale(np.max(np.abs(p), axis=(1, 3)))
    with np.errstate(invalid="ignore", over="ignore"):
        r = np.clip((p / s[:, None, :, None]).astype(np.float32), -E4M3_MAX, E4M3_MAX)
    return encode(r).reshape(nb * BLOCK, kb * BLOCK)[:rows], s


def act_values(q, scale) -> np.ndarray:
    """fp64 [m, 128 kb] of activation codes and scales [kb, m]."""
    return decode(q) * np.repeat(np.asarray(scale, dtype=np.float64).T, BLOCK, axis=1)


def weight_values(w, scale) -> np.ndarray:
    """fp64 [rows, 128 kb] of weight codes and scales [ceil(rows/128), kb]."""
    s = np.repeat(np.repeat(np.asarray(scale, dtype=np.float64), BLOCK, axis=0), BLOCK, axis=1)
    return decode(w) * s[:w.shape[0]]


def gemm(w, ws, q, qs):
    """(y fp64 [m, rows], magnitude: the sum of the absolute values of its terms)."""
    a, b = act_values(q, qs), weight_values(w, ws)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def gemm_grouped(w, ws, q, qs, offsets, row_ids=None):
    """The grouped product's rows offsets[0] .. offsets[-1] - 1 of y and of its magnitude
    (zeros elsewhere), [slots, rows]."""
    slots = len(row_ids) if row_ids is not None else q.shape[0]
    y = np.zeros((slots, w.shape[1]))
    mag = np.zeros_like(y)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            t = np.arange(lo, hi) if row_ids is None else np.asarray(row_ids)[lo:hi]
            y[lo:hi], mag[lo:hi] = gemm(w[e], ws[e], q[t], qs[:, t])
    return y, mag
