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
