"""GPU: the E4M3 and mixture-of-experts calls over the whole range that their definitions
allow."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_quantized_matmul_amd import binding as B
from oracle import fp8 as of8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.view(dtype)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    t = t.view(torch.uint8) if t.dtype == F8 else t.to(torch.float64) if t.is_floating_point() else t
    return t.cpu().numpy()


def gemm_tol(k):
    """A block's 128 exact products added with at most 128 roundings of 2^-23, the scales'
    product and the scaling one rounding of 2^-24 each, the kb blocks one each."""
    return 128 * 2.0 ** -23 + (of8.blocks(k) + 3) * 2.0 ** -24


def normal_codes(rng, shape, size):
    """Codes of normal values of the given size, drawn from a pool of 4096."""
    pool = of8.encode(np.clip(size * rng.standard_normal(4096), -448.0, 448.0))
    return pool[rng.integers(0, 4096, shape)]


# ------------------------------------------------------------------ sums

LARGE = [  # rows of each expert (one: a dense product), n, k: 128 x 128 tiles for every compute unit
    ([260], 11000, 4096),
    ([131], 33000, 4100),
    ([130, 0, 300, 97], 9000, 4100),
    ([512, 1], 8193, 7000),
]


@pytest.mark.parametrize("signs", ["both", "one"])
@pytest.mark.parametrize("sizes,n,k", LARGE)
def test_large_products_sum_in_fp32(sizes, n, k, signs):
    """Rows of 32 blocks and more, a few columns 30 times the others, terms of either sign
    and of one: every element of an fp32 result within the bound, and a 16-bit result is
    the fp32 result rounded once, whatever the type."""
    rng = np.random.default_rng(n + k)
    experts, total, kb = len(sizes), sum(sizes), of8.blocks(k)
    m = total
    q = np.zeros((m, kb * 128), dtype=np.uint8)
    w = np.zeros((experts, n, kb * 128), dtype=np.uint8)
    q[:, :k] = np.where(rng.random(k) < 0.02, normal_codes(rng, (m, k), 200.0), normal_codes(rng, (m, k), 7.0))
    w[:, :, :k] = normal_codes(rng, (experts, n, k), 120.0)
    if signs == "one":
        q &= 0x7F
        w &= 0x7F
    qs = np.exp(rng.standard_normal((kb, m))).astype(np.float32)
    ws = np.exp(rng.standard_normal((experts, of8.blocks(n), kb))).astype(np.float32)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    wd, wsd, qd, qsd = dev(w, F8), dev(ws), dev(q, F8), dev(qs)
    for gather in ([None] if experts == 1 else [False, True]):
        rows = rng.integers(0, m, total).astype(np.int32) if gather else np.arange(total, dtype=np.int32)

        def product(dtype):
            if experts == 1:
                return B.fp8_gemm(wd[0], wsd[0], k, qd, qsd, dtype=dtype)
            return B.fp8_gemm_grouped(wd, wsd, k, qd, qsd, dev(offsets), row_ids=dev(rows) if gather else None,
                                      dtype=dtype)

        y = product(torch.float32)
        got = host(y)
        for e in range(experts):
            if sizes[e] == 0:
                continue
            pick = offsets[e] + np.unique(np.r_[0, sizes[e] - 1, rng.integers(0, sizes[e], 12)])
            cols = np.unique(np.r_[0, n - 1, rng.integers(0, n, 200)])
            a = of8.act_values(q[rows[pick]], qs[:, rows[pick]])
            b = of8.decode(w[e][cols]) * np.repeat(ws[e][cols // 128].astype(np.float64), 128, axis=1)
            ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
            assert np.all(np.abs(got[np.ix_(pick, cols)] - ref) <= (gemm_tol(k) + 2.0 ** -24) * mag)
        for dtype in (torch.bfloat16, torch.float16):
            z = product(dtype)
            off = int((z != y.to(dtype)).sum())
            assert off == 0, f"{dtype}, gather {gather}: {off} of {z.numel()} are not the fp32 result rounded"

# ------------------------------------------------------------------ tokens

def test_combine_more_tokens_than_a_launch():
    """2^24 tokens and a few: one workgroup each would be 2^32 threads."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    tokens, d, rows = (1 << 24) + 5, 8, 1000
    y = torch.randn(rows, d, device=DEV, generator=g).bfloat16()
    slots = torch.randint(-1, rows, (tokens, 1), device=DEV, generator=g, dtype=torch.int32)
    weights = torch.rand(tokens, 1, device=DEV, generator=g)
    out = B.moe_combine(y, slots, weights)
    for t0 in range(0, tokens, 1 << 22):
        s, w = slots[t0:t0 + (1 << 22), 0].long(), weights[t0:t0 + (1 << 22)]
        want = torch.where(s[:, None] >= 0, y[s.clamp(min=0)].float() * w, 0.0).bfloat16()
        assert torch.equal(out[t0:t0 + (1 << 22)], want)

# ------------------------------------------------------------------ gates

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_swiglu_of_far_negative_gates(dtype):
    """silu(g) u where exp(-g) leaves fp32's range but the value does not.  exp(g / 2) within a
    unit (2^-23), twice, and three products (2^-24 each): 3.5 x 2^-23, on a scale one more
    rounding; the code as near to the quotient as half a step and both allow."""
    rng = np.random.default_rng(4)
    m, k = 24, 300
    g = np.linspace(-140.0, -60.0, m)[:, None] - rng.random((m, k))
    u = rng.standard_normal((m, k)) * np.exp(np.clip(-g - 60.0, 0.0, 80.0))
    x = torch.from_numpy(np.concatenate([g, u], 1).astype(np.float32)).to(dtype)
    q, s = B.fp8_quant(x.to(DEV), swiglu=True)
    x = x.double().numpy()
    v = np.zeros((m, 3 * 128))
    v[:, :k] = x[:, :k] * np.exp(x[:, :k]) / (1.0 + np.exp(x[:, :k])) * x[:, k:]
    a = np.abs(v).reshape(m, 3, 128).max(2)
    assert a.min() > 2.0 ** -117                    # every block's scale is a normal number
    want = (a / 448.0).T
    assert np.all(np.abs(host(s) - want) <= 4 * 2.0 ** -23 * want)
    ideal = v / np.repeat(want.T, 128, axis=1)
    err = np.abs(of8.decode(host(q)) - ideal)
    assert np.all(err <= np.maximum(np.abs(ideal), 2.0 ** -6) * 2.0 ** -4 * (1 + 2.0 ** -20) + 8 * 2.0 ** -23 * np.abs(ideal))

# ------------------------------------------------------------------ scales

# every kernel that the sizes choose between: 1, 2 and 4 fragments of tokens, 64 x 64, 64 x 128 and
# 128 x 128 tiles; rows shorter and longer than the tiles' pipelines
SCALED = [(3, 300, 384), (20, 300, 1100), (300, 300, 384), (300, 500, 1152), (70, 5001, 384), (70, 5001, 1152),
          (129, 9000, 384), (129, 9000, 700), (1000, 4224, 300), (1000, 4224, 1152)]


@pytest.mark.parametrize("m,n,k", SCALED)
def test_products_of_scales_past_the_range(m, n, k):
    """Scales whose product overflows (2^132) where the block's sum is small or 0, and is
    subnormal (2^-143) where the sum brings the result back: as if the three were
    multiplied exactly.  Beside gemm_tol a rounding more for the scaling in two steps, and
    half a subnormal step for each block."""
    rng = np.random.default_rng(m + n + k)
    kb, nb = of8.blocks(k), of8.blocks(n)
    q, w = np.zeros((m, kb * 128), dtype=np.uint8), np.zeros((n, kb * 128), dtype=np.uint8)
    q[:, :k], w[:, :k] = normal_codes(rng, (m, k), 100.0), normal_codes(rng, (n, k), 100.0)
    # by block modulo 3: scales of tokens (modulo 3) and of weight rows (even and odd blocks of 128)
    ex = np.array([[72, 5, -75], [60, 0, -75], [-2, 3, -75]])[np.arange(kb) % 3][:, np.arange(m) % 3]
    ew = np.array([[60, -60, 0], [-68, -68, -68]])[np.arange(nb) % 2][:, np.arange(kb) % 3]
    # codes of a high block are the type's subnormals, and every other weight row is 0 there
    cols = np.repeat(np.arange(kb) % 3 == 0, 128)
    q[:, cols] &= 0x87
    w[:, cols] &= 0x87
    w[np.ix_(np.arange(n) % 2 == 0, cols)] = 0
    qs = (np.exp2(ex.astype(np.float64)) * rng.uniform(1, 2, ex.shape)).astype(np.float32)
    ws = (np.exp2(ew.astype(np.float64)) * rng.uniform(1, 2, ew.shape) * rng.choice([-1.0, 1.0], ew.shape)).astype(np.float32)
    qs[0, m // 2] = 0.0
    ref, mag = of8.gemm(w, ws, q, qs)
    assert np.abs(ref).max() < 3.4e38
    got = host(B.fp8_gemm(dev(w, F8), dev(ws), k, dev(q, F8), dev(qs), dtype=torch.float32))
    assert np.all(np.isfinite(got)), f"{int((~np.isfinite(got)).sum())} results are not finite"
    bound = (gemm_tol(k) + 2.0 ** -23) * mag + kb * 2.0 ** -149
    worst = np.max(np.abs(got - ref) / bound)
    assert worst <= 1.0, f"{worst:.3g} of the bound"
    # the same rows as two experts' and gathered
    off = dev(np.array([0, m // 3, m], dtype=np.int32))
    two = torch.stack([dev(w)] * 2).view(F8)
    ids = rng.permutation(m).astype(np.int32)
    got = host(B.fp8_gemm_grouped(two, torch.stack([dev(ws)] * 2), k, dev(q, F8), dev(qs), off, row_ids=dev(ids),
                                  dtype=torch.float32))
    assert np.all(np.abs(got - ref[ids]) <= bound[ids])


@pytest.mark.parametrize("m,n", [(2, 130), (300, 300), (70, 5001), (1000, 4224)])
def test_scales_that_are_no_numbers(m, n):
    """An infinite scale makes its token's results infinite or, where the sum is 0, NaN; a NaN
    scale makes them NaN; other tokens are untouched."""
    rng = np.random.default_rng(m)
    k = 256
    q, w = normal_codes(rng, (m, k), 100.0), normal_codes(rng, (n, k), 100.0)
    w[5, :128] = 0
    qs, ws = np.ones((2, m), dtype=np.float32), np.ones((of8.blocks(n), 2), dtype=np.float32)
    args = dev(w, F8), dev(ws), k, dev(q, F8)
    clean = host(B.fp8_gemm(*args, dev(qs), dtype=torch.float32))
    qs[0, 0], qs[1, 1] = np.inf, np.nan
    y = host(B.fp8_gemm(*args, dev(qs), dtype=torch.float32))
    part, _ = of8.gemm(w[:, :128], ws[:, :1], q[:1, :128], np.ones((1, 1)))
    with np.errstate(invalid="ignore"):
        assert np.array_equal(y[0], part[0] * np.inf, equal_nan=True)
    assert np.all(np.isnan(y[1])) and np.array_equal(y[2:], clean[2:])
