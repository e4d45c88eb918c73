"""GPU parity of the 8-bit float products and the mixture-of-experts calls.

Codes, scales, expert choices and positions are bit-exact with the oracle.  Products:
|y - ref| <= tol x magnitude + half a step of y's type, with tol from the
arithmetic.  A block's 128 products (8 significant bits each) are exact in fp32
and are added with at most 128 roundings of 2^-23 (the matrix cores may truncate
instead of rounding), its scale product and the scaling round once each and the
kb blocks are added with a rounding of 2^-24 each:

    tol = 128 x 2^-23 + (kb + 3) x 2^-24
"""
from __future__ import annotations

import math

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


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.view(dtype)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    t = t.view(torch.uint8) if t.dtype == F8 else t.to(torch.float64) if t.is_floating_point() else t
    return t.cpu().numpy()


def acts(rng, m, k):
    x = rng.standard_normal((m, k)) * np.exp(rng.standard_normal((m, 1)))
    x[:, rng.random(k) < 0.02] *= 30.0
    return x.astype(np.float32)


def gemm_tol(k):
    return 128 * 2.0 ** -23 + (of8.blocks(k) + 3) * 2.0 ** -24


def check_product(y, ref, mag, k, dtype, label):
    got = host(y)
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2     # half a subnormal step
    err = np.abs(got - ref)
    tol = gemm_tol(k) * mag
    bound = tol + half * (np.abs(ref) + tol) + tiny
    assert np.all(np.isfinite(got)), label
    worst = float(np.max(err / np.maximum(bound, 1e-300)))
    assert worst <= 1.0, f"{label}: {worst:.3g} of the bound at {np.unravel_index(np.argmax(err / bound), err.shape)}"


# ------------------------------------------------------------------ quantizers

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,k,gap", [(1, 1, 0), (1, 4096, 0), (3, 127, 0), (15, 129, 1), (16, 128, 0), (17, 312, 8),
                                     (33, 1092, 0), (130, 640, 64), (5, 14336, 0)])
def test_quant_bit_exact(m, k, gap, dtype):
    rng = np.random.default_rng(m * 1000 + k)
    x = torch.from_numpy(acts(rng, m, k + gap)).to(dtype)
    x[m // 2, :] = 0.0
    if m > 2:
        x[1, 0] = 448.0 * 17 / 16                   # a quotient half way between two codes
        x[2, :] *= 2.0 ** -20
    d = x.to(DEV)[:, :k]
    q, s = B.fp8_quant(d)
    assert q.dtype == F8 and q.is_contiguous()
    qr, sr = of8.quant_act(x[:, :k].float().numpy())
    assert np.array_equal(s.cpu().numpy().view(np.uint32), sr.view(np.uint32))
    assert np.array_equal(host(q) & 0x7F, qr & 0x7F)
    nz = (qr & 0x7F) != 0                           # the sign of a zero code carries nothing
    assert np.array_equal(host(q)[nz], qr[nz])


def test_quant_ties_and_extremes():
    v = np.zeros((7, 256), dtype=np.float32)
    mids = ((of8.VALUES[:126] + of8.VALUES[1:127]) / 2).astype(np.float32)
    v[0, :126], v[0, 127] = mids, 448.0
    v[1, :126], v[1, 127] = -mids, -448.0
    v[2, :] = 3.0e38
    v[3, 0], v[3, 130] = 2.0 ** -149, 2.0 ** -127
    v[4, 5], v[4, 6] = np.nan, 1.0
    v[5, 200], v[5, 3] = -np.inf, 2.0
    q, s = B.fp8_quant(dev(v))
    qr, sr = of8.quant_act(v)
    assert np.array_equal(s.cpu().numpy(), sr, equal_nan=True)
    assert np.array_equal(of8.decode(host(q)), of8.decode(qr), equal_nan=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,k", [(1, 64), (3, 127), (17, 312), (40, 1024), (2, 14336)])
def test_quant_swiglu(m, k, dtype):
    """v: exp within 1 unit (2^-23), 1 + e, the division and the product one rounding
    each: 2.5 x 2^-23, on a scale one more rounding.  The code is the nearest to a
    quotient that is off by both: half a step (2^-4, 2^-10 below 2^-6) and 6 x 2^-23."""
    rng = np.random.default_rng(m + k)
    x = torch.from_numpy(acts(rng, m, 2 * k)).to(dtype)
    q, s = B.fp8_quant(x.to(DEV), swiglu=True)
    kb = of8.blocks(k)
    v = np.zeros((m, kb * 128))
    v[:, :k] = of8.swiglu64(x.double().numpy())
    a = np.abs(v).reshape(m, kb, 128).max(2)
    want = np.where(a > 0, np.maximum(a / 448.0, 2.0 ** -126), 1.0).T
    assert np.all(np.abs(host(s) - want) <= 3 * 2.0 ** -23 * want)
    ideal = v / np.repeat(want.T, 128, axis=1)
    slack = 6 * 2.0 ** -23 * np.abs(ideal)
    err = np.abs(of8.decode(host(q)) - ideal)
    assert np.all(err <= (np.maximum(np.abs(ideal), 2.0 ** -6) * 2.0 ** -4) * (1 + 2.0 ** -20) + slack)


def test_quant_swiglu_extremes():
    x = np.zeros((3, 256), dtype=np.float32)
    x[0, 0], x[0, 128] = -200.0, 3.0                # silu of a large negative gate is 0
    x[1, 0], x[1, 128] = 90.0, 2.0
    x[2, 0], x[2, 128] = np.nan, 1.0
    q, s = B.fp8_quant(dev(x), swiglu=True)
    s = s.cpu().numpy()
    assert s[0, 0] <= 2.0 ** -126 or s[0, 0] == 1.0
    assert abs(s[0, 1] - 180.0 / 448.0) < 1e-6 and np.isnan(s[0, 2])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (129, 257), (312, 1092), (3, 130, 200)])
def test_pack_bit_exact(shape, dtype):
    rng = np.random.default_rng(sum(shape))
    w = torch.from_numpy((0.02 * rng.standard_normal(shape)).astype(np.float32)).to(dtype)
    q, s = B.fp8_pack(w.to(DEV))
    lead = w.reshape(-1, *w.shape[-2:]).float().numpy()
    qs = [of8.quant_weight(e) for e in lead]
    assert np.array_equal(s.cpu().numpy().reshape(-1, *qs[0][1].shape), np.stack([b for _, b in qs]))
    assert np.array_equal(of8.decode(host(q)).reshape(-1, *qs[0][0].shape), np.stack([of8.decode(a) for a, _ in qs]))


# ------------------------------------------------------------------ products

def operands(rng, m, n, k, experts=None):
    q, qs = of8.quant_act(acts(rng, m, k))
    ws = [of8.quant_weight((0.02 * rng.standard_normal((n, k))).astype(np.float32)) for _ in range(experts or 1)]
    w, s = np.stack([a for a, _ in ws]), np.stack([b for _, b in ws])
    return q, qs, (w if experts else w[0]), (s if experts else s[0])


GEMM_SIZES = [(1, 1, 1), (1, 16, 128), (1, 312, 312), (1, 4096, 1024), (2, 129, 129), (4, 1000, 4096), (7, 33, 640),
              (16, 256, 256), (17, 1024, 512), (31, 200, 300), (32, 512, 2048), (33, 130, 127), (48, 320, 384),
              (64, 128, 128), (65, 1092, 312), (77, 1092, 312), (100, 255, 1000), (128, 384, 256), (129, 257, 129),
              (200, 640, 896), (256, 256, 1024), (300, 1000, 200), (513, 300, 384), (1, 100, 14336), (9, 70, 14336)]


@pytest.mark.parametrize("m,n,k", GEMM_SIZES)
def test_gemm(m, n, k):
    rng = np.random.default_rng(m + 7 * n + 13 * k)
    q, qs, w, ws = operands(rng, m, n, k)
    ref, mag = of8.gemm(w, ws, q, qs)
    args = (dev(w, F8), dev(ws), k, dev(q, F8), dev(qs))
    for dtype in TYPES:
        check_product(B.fp8_gemm(*args, dtype=dtype), ref, mag, k, dtype, f"{m}x{n}x{k} {dtype}")
    y = torch.full((m, n), math.nan, device=DEV)
    assert B.fp8_gemm(*args, y=y) is y
    check_product(y, ref, mag, k, torch.float32, "y given")


# one size for each kernel that the sizes choose between, with rows shorter and longer than its pipeline
ROUTES = [(3, 5000, 200), (16, 4800, 2300), (30, 4000, 700), (32, 6001, 128), (50, 4096, 300), (64, 4000, 2176),
          (65, 5000, 640), (70, 5001, 100), (129, 4000, 384), (130, 9000, 256), (300, 8000, 130), (200, 12000, 520),
          (1100, 4002, 200), (1025, 4000, 96), (1000, 4224, 1100)]


@pytest.mark.parametrize("m,n,k", ROUTES)
def test_gemm_routes(m, n, k):
    rng = np.random.default_rng(m + n + k)
    q, qs, w, ws = operands(rng, m, n, k)
    ref, mag = of8.gemm(w, ws, q, qs)
    for dtype in (torch.float32, torch.bfloat16):
        y = B.fp8_gemm(dev(w, F8), dev(ws), k, dev(q, F8), dev(qs), dtype=dtype)
        check_product(y, ref, mag, k, dtype, f"{m}x{n}x{k} {dtype}")


@pytest.mark.parametrize("kind", ["dense", "grouped"])
def test_native_sums(kind):
    """Large products with 16-bit results and 32 blocks a row or more.  The 8-bit instructions: of each 8
    neighbouring products the largest keeps its bits and the other 7 lose less than
    2^-13 of it each; an eighth such loss stands for adding the groups.  So a sum is off
    by less than 2^-10 of the largest product, over all groups of 8, and by what
    gemm_tol counts.  The error's norm: 2^-13 of the result's, and the rounding to 16 bits,
    uniform over half a step."""
    rng = np.random.default_rng(11)
    m, n, k = (260, 11000, 4096) if kind == "dense" else (280, 4000, 4100)
    dtype = torch.bfloat16 if kind == "dense" else torch.float16
    rows = np.sort(rng.choice(m, 24, replace=False))              # the rows that are checked
    cols = rng.choice(n, 300, replace=False)
    q, qs = of8.quant_act(acts(rng, m, k))
    w, ws = of8.quant_weight((0.02 * rng.standard_normal((n, k))).astype(np.float32))
    wd, sd, qd, qsd = dev(w, F8), dev(ws), dev(q, F8), dev(qs)
    if kind == "dense":
        y = B.fp8_gemm(wd, sd, k, qd, qsd, dtype=dtype)
        exact = B.fp8_gemm(wd, sd, k, qd, qsd, dtype=torch.float32)
    else:
        off = dev(np.array([0, 130, m], dtype=np.int32))
        two, s2 = torch.stack([wd.view(torch.uint8)] * 2).view(F8), torch.stack([sd] * 2)
        y = B.fp8_gemm_grouped(two, s2, k, qd, qsd, off, dtype=dtype)
        exact = B.fp8_gemm_grouped(two, s2, k, qd, qsd, off, dtype=torch.float32)
    y, exact = host(y), host(exact)
    full, mag = of8.gemm(w, ws, q[rows], qs[:, rows])
    ref, mag = full[:, cols], mag[:, cols]
    wide = np.repeat(ws, 128, axis=0)[:n][cols]                   # a scale row for each chosen weight row
    a = np.abs(of8.act_values(q[rows], qs[:, rows])).reshape(len(rows), -1, 8)
    b = np.abs(of8.decode(w[cols]) * np.repeat(wide.astype(np.float64), 128, axis=1)).reshape(len(cols), -1, 8)
    lost = 2.0 ** -10 * np.stack([(a[t][None] * b).max(2).sum(1) for t in range(len(rows))])
    half = torch.finfo(dtype).eps / 2
    got = y[np.ix_(rows, cols)]
    tol = lost + gemm_tol(k) * mag
    assert np.all(np.abs(got - ref) <= tol + half * (np.abs(ref) + tol) + 2.0 ** -25)
    e32 = exact[np.ix_(rows, cols)]
    assert np.all(np.abs(e32 - ref) <= (gemm_tol(k) + 2.0 ** -24) * mag)      # fp32 results do not take it
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert rel <= 2.0 ** -13 + half / math.sqrt(3)


@pytest.mark.parametrize("m,n,k", [(1, 100, 384), (20, 100, 384), (90, 200, 384), (300, 300, 384)])
def test_gemm_scales_of_any_size_and_nan(m, n, k):
    """Scales from 2^-100 to 2^60, negative and zero ones; a NaN token poisons its row alone."""
    rng = np.random.default_rng(m)
    q, qs, w, ws = operands(rng, m, n, k)
    qs = (qs * np.exp2(rng.integers(-100, 60, qs.shape))).astype(np.float32)
    qs[0, m // 2] = 0.0
    ws[0, 1] *= -1.0
    ref, mag = of8.gemm(w, ws, q, qs)
    y = host(B.fp8_gemm(dev(w, F8), dev(ws), k, dev(q, F8), dev(qs), dtype=torch.float32))
    assert np.all(np.abs(y - ref) <= (gemm_tol(k) + 2.0 ** -24) * mag + 2.0 ** -140)
    q[m - 1, 3] = 0x7F
    y2 = host(B.fp8_gemm(dev(w, F8), dev(ws), k, dev(q, F8), dev(qs), dtype=torch.float32))
    assert np.all(np.isnan(y2[m - 1])) and np.array_equal(y2[:m - 1], y[:m - 1])


GROUPED = [  # sizes of the experts' groups, n, k
    ([1], 64, 128),
    ([0, 0, 3], 130, 312),
    ([1, 1, 0, 1, 1, 0, 0, 1], 256, 256),
    ([5, 0, 17, 1, 0, 0, 40, 2], 1092, 312),
    ([129, 0, 64, 1], 320, 200),
    ([0, 300, 7, 130, 0, 65], 257, 384),
    ([16] * 20, 128, 129),
    ([2, 0, 513], 128, 256),
    ([1, 0, 2, 33, 65, 5] * 12, 520, 300),              # 72 experts, 64 x 128 tiles
    ([130, 0, 290, 257, 1, 128], 6000, 200),            # 128 x 128 tiles, whole and ragged
    ([3] * 70, 300, 513),
]


@pytest.mark.parametrize("sizes,n,k", GROUPED)
@pytest.mark.parametrize("gather", [True, False])
def test_grouped(sizes, n, k, gather):
    rng = np.random.default_rng(sum(sizes) + n + k)
    total = sum(sizes)
    m = max(1, total // 3) if gather else total
    q, qs, w, ws = operands(rng, m, n, k, experts=len(sizes))
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rows = rng.integers(0, m, total).astype(np.int32) if gather else None
    ref, mag = of8.gemm_grouped(w, ws, q, qs, offsets, rows)
    for dtype in TYPES:
        y = B.fp8_gemm_grouped(dev(w, F8), dev(ws), k, dev(q, F8), dev(qs), dev(offsets),
                               row_ids=dev(rows) if gather else None, dtype=dtype)
        check_product(y, ref, mag, k, dtype, f"{sizes} {n}x{k} {dtype}")


@pytest.mark.parametrize("sizes,slots", [([3, 0, 4], 12), ([0, 0], 5), ([70, 9], 200), ([100, 200, 3], 600)])
def test_grouped_leaves_other_rows_alone(sizes, slots):
    """Ranges that start after 0 and end before slots; no expert with any row."""
    rng = np.random.default_rng(slots)
    n, k, m = 100, 200, 9
    q, qs, w, ws = operands(rng, m, n, k, experts=len(sizes))
    offsets = (np.concatenate([[0], np.cumsum(sizes)]) + 1).astype(np.int32)
    rows = rng.integers(0, m, slots).astype(np.int32)
    rows[0] = -1
    rows[offsets[-1]:] = -1
    y = torch.full((slots, n), 7.0, device=DEV)
    B.fp8_gemm_grouped(dev(w, F8), dev(ws), k, dev(q, F8), dev(qs), dev(offsets), row_ids=dev(rows), y=y)
    ref, mag = of8.gemm_grouped(w, ws, q, qs, offsets, rows)
    lo, hi = offsets[0], offsets[-1]
    got = host(y)
    assert np.all(got[:lo] == 7.0) and np.all(got[hi:] == 7.0)
    assert np.all(np.abs(got[lo:hi] - ref[lo:hi]) <= (gemm_tol(k) + 2.0 ** -24) * mag[lo:hi])


def test_native_sums_pass_nan_on():
    """A NaN code in a large 16-bit product makes its token's row NaN and no other."""
    rng = np.random.default_rng(12)
    m, n, k = 300, 16000, 4096
    q, qs = of8.quant_act(acts(rng, m, k))
    w, ws = of8.quant_weight((0.02 * rng.standard_normal((n, k))).astype(np.float32))
    wd, sd, qsd = dev(w, F8), dev(ws), dev(qs)
    y = B.fp8_gemm(wd, sd, k, dev(q, F8), qsd)
    q[77, 4000] = 0xFF
    z = B.fp8_gemm(wd, sd, k, dev(q, F8), qsd)
    assert bool(torch.isnan(z[77]).all()) and bool(torch.isfinite(y).all())
    assert torch.equal(z[:77], y[:77]) and torch.equal(z[78:], y[78:])


# ------------------------------------------------------------------ routing

def check_route(r, x, top, renorm, label):
    ids, w, off, rows, slots = omoe.route(x, top, renorm)
    for name, want in (("ids", ids), ("offsets", off), ("row_ids", rows), ("slots", slots)):
        assert np.array_equal(host(getattr(r, name)), want), f"{label}: {name}"
    # exp: 1 unit each side of the quotient and its argument's rounding (|l - max| 2^-24, where the
    # result is no underflow |l - max| < 104), the sum one rounding an addend, the division one
    n = x.shape[1]
    got = host(r.weights)
    bound = w * (4 * 2.0 ** -23 + (n + 2 + 2 * 104) * 2.0 ** -24) + 2.0 ** -120
    assert np.all(np.abs(got - w) <= bound), f"{label}: weights off by {np.max(np.abs(got - w))}"


@pytest.mark.parametrize("tokens,experts,top", [(1, 1, 1), (1, 64, 8), (4, 64, 8), (3, 12, 3), (63, 7, 7), (64, 65, 4),
                                                (65, 64, 2), (200, 256, 8), (300, 257, 5), (129, 1024, 32),
                                                (1000, 100, 1), (5000, 32, 6), (64, 64, 32), (40000, 9, 2)])
def test_route(tokens, experts, top):
    rng = np.random.default_rng(tokens + experts)
    for dtype in TYPES:
        x = torch.from_numpy(rng.standard_normal((tokens, experts + 3)).astype(np.float32)).to(dtype)
        x = x[:, 1:1 + experts]                      # strided rows, no 16-byte alignment
        for renorm in (True, False):
            check_route(B.moe_route(x.to(DEV), top, renorm=renorm), x.double().numpy(), top, renorm,
                        f"{tokens}x{experts} top {top} {dtype}")


# each number of logits a lane, and chunks of one token a wave, of two, and the last one ragged
@pytest.mark.parametrize("tokens,experts,top", [(16, 512, 10), (17, 512, 10), (4097, 513, 6), (4096, 384, 12), (700, 128, 8),
                                                (700, 129, 8)])
def test_route_many_experts(tokens, experts, top):
    test_route(tokens, experts, top)


@pytest.mark.parametrize("tokens", [6, 130])
def test_route_masks_ties_and_extremes(tokens):
    rng = np.random.default_rng(tokens)
    x = rng.integers(-2, 3, (tokens, 48)).astype(np.float32)       # many equal logits
    x[rng.random(x.shape) < 0.5] = -np.inf
    x[0] = -np.inf                                                 # no expert left
    x[1, 1:] = -np.inf                                             # one left
    x[2] = np.nan
    x[2, 40] = 1.0
    x[3, [5, 9]] = np.inf
    x[4] = -3.4028234663852886e38                                  # the type's lowest value is no mask
    x[5] = [0.0, -0.0] * 24
    for renorm in (True, False):
        check_route(B.moe_route(dev(x), 6, renorm=renorm), x, 6, renorm, f"{tokens} tokens")
    none = np.full((tokens, 48), -np.inf, dtype=np.float32)
    r = B.moe_route(dev(none), 4)
    assert np.all(host(r.ids) == -1) and np.all(host(r.weights) == 0) and np.all(host(r.offsets) == 0)
    assert np.all(host(r.row_ids) == -1) and np.all(host(r.slots) == -1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,top,d", [(1, 1, 1), (1, 8, 2048), (5, 3, 312), (33, 2, 1092), (7, 12, 257), (3, 4, 5000)])
def test_combine(tokens, top, d, dtype):
    rng = np.random.default_rng(tokens + top + d)
    rows = tokens * top + 3
    y = torch.from_numpy(rng.standard_normal((rows, d)).astype(np.float32)).to(dtype)
    slots = rng.permutation(rows)[:tokens * top].reshape(tokens, top).astype(np.int32)
    w = rng.random((tokens, top)).astype(np.float32)
    if tokens > 2:
        slots[1] = -1                                              # nothing to combine: zeros
        slots[2, 0] = -1
        y[slots[2, 1]] = 1e4
    unread = [r for r in range(rows) if r not in set(slots.ravel().tolist())]
    y[unread] = math.nan                                           # rows that no slot names are not read
    ref, mag = omoe.combine(y.double().numpy(), slots, w)
    got = host(B.moe_combine(y.to(DEV), dev(slots), dev(w)))
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    tol = top * 2.0 ** -24 * mag
    assert np.all(np.abs(got - ref) <= tol + half * (np.abs(ref) + tol) + tiny)
    if tokens > 2:
        assert np.all(got[1] == 0)


# ------------------------------------------------------------------ streams, graphs, large offsets

def layer(x, logits, w13, s13, w2, s2, hidden, ffn, top):
    r = B.moe_route(logits, top)
    q, qs = B.fp8_quant(x)
    h = B.fp8_gemm_grouped(w13, s13, hidden, q, qs, r.offsets, row_ids=r.row_ids)
    a, a_s = B.fp8_quant(h, swiglu=True)
    y = B.fp8_gemm_grouped(w2, s2, ffn, a, a_s, r.offsets)
    return B.moe_combine(y, r.slots, r.weights)


@pytest.mark.parametrize("tokens", [1, 5, 300])
def test_layer_on_a_stream_and_in_a_graph(tokens):
    """The five calls as one layer give the same bits eagerly, on another stream and
    in every replay of a graph, with eager work between the replays."""
    g = torch.Generator(device=DEV)
    g.manual_seed(tokens)
    hidden, ffn, experts, top = 256, 200, 16, 4
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    w13, s13 = B.fp8_pack(0.05 * rand(experts, 2 * ffn, hidden))
    w2, s2 = B.fp8_pack(0.05 * rand(experts, hidden, ffn))
    static_x, static_l = rand(tokens, hidden).bfloat16(), rand(tokens, experts)
    args = (w13, s13, w2, s2, hidden, ffn, top)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = layer(static_x, static_l, *args)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(warm, layer(static_x, static_l, *args))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(static_x, static_l, *args)
    for _ in range(4):
        x, lg = rand(tokens, hidden).bfloat16(), rand(tokens, experts)
        want = layer(x, lg, *args)
        static_x.copy_(x)
        static_l.copy_(lg)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_grouped_weights_past_32_bits():
    """Experts whose codes lie past 2^32 bytes: the last of 5 experts of 1 GiB."""
    experts, n, k = 5, 65536, 16384
    w = torch.zeros((experts, n, k), dtype=torch.uint8, device=DEV)
    ws = torch.ones((experts, n // 128, k // 128), device=DEV)
    w[4, n - 3:, k - 5:] = 0x38                                     # ones
    w[4, 0, 0] = 0x40                                               # 2
    q = torch.full((2, k), 0x38, dtype=torch.uint8, device=DEV).view(F8)
    qs = torch.ones((k // 128, 2), device=DEV)
    off = torch.tensor([0, 0, 0, 0, 1, 2], dtype=torch.int32, device=DEV)
    y = host(B.fp8_gemm_grouped(w.view(F8), ws, k, q, qs, off, dtype=torch.float32))
    assert np.all(y[0] == 0) and y[1, 0] == 2 and np.all(y[1, -3:] == 5) and np.all(y[1, 1:-3] == 0)


@pytest.mark.parametrize("tokens", [1, 37])
def test_example_layer(tokens):
    """The example's layer against fp32: three roundings to E4M3 (activations, weights, the inner
    activations; at most 2^-4 each, uniform over a step: about 2^-4 / sqrt(3) in the mean)
    and the two products' two operands each: sqrt(4) x 0.036 = 0.072 at the most."""
    import importlib.util
    import os

    from tests.conftest import ROOT
    spec = importlib.util.spec_from_file_location("fp8_moe_ffn", os.path.join(ROOT, "examples", "fp8_moe_ffn.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    rel, us = example.run(tokens, 256, 192, 8, 2, replays=3)
    assert rel < 0.072 and us > 0
