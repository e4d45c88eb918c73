"""The E4M3 and routing oracle against independent statements of the same facts (CPU)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import fp8 as of8
from oracle import moe as omoe


def test_code_values_match_the_type():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(of8.VALUES, want, equal_nan=True)


def test_encode_matches_a_conversion_of_fp32():
    rng = np.random.default_rng(5)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 0.01, of8.VALUES[:127],
                        (of8.VALUES[:126] + of8.VALUES[1:127]) / 2, [0.0, -0.0, 448.0, -448.0]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(of8.encode(x), want)
    assert of8.encode([np.nan])[0] == 0x7F


def test_quant_scales():
    v = np.zeros((3, 130), dtype=np.float32)
    v[0, 5] = 896.0
    v[1, 129] = 2.0 ** -149
    v[2, 0] = np.inf
    q, s = of8.quant_act(v)
    assert q.shape == (3, 256) and s.shape == (2, 3)
    assert s[0, 0] == 2.0 and s[1, 0] == 1.0 and s[1, 1] == of8.MIN_SCALE
    assert np.isnan(s[0, 2]) and np.all(q[2, :128] == 0x7F) and s[1, 2] == 1.0
    assert of8.decode(q)[0, 5] == 448.0


def test_gemm_is_the_blockwise_sum():
    rng = np.random.default_rng(6)
    q, qs = of8.quant_act(rng.standard_normal((3, 200)).astype(np.float32))
    w, ws = of8.quant_weight(rng.standard_normal((150, 200)).astype(np.float32))
    y, _ = of8.gemm(w, ws, q, qs)
    for t, r in [(0, 0), (2, 149), (1, 127), (1, 128)]:
        total = 0.0
        for b in range(2):
            part = sum(of8.VALUES[q[t, 128 * b + j]] * of8.VALUES[w[r, 128 * b + j]] for j in range(128))
            total += float(qs[b, t]) * float(ws[r // 128, b]) * part
        assert abs(total - y[t, r]) <= 1e-12 * abs(y).max()


@pytest.mark.parametrize("renorm", [True, False])
def test_route(renorm):
    x = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [np.nan, np.inf, 0.0, -1.0]])
    ids, w, off, rows, slots = omoe.route(x, 3, renorm)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [1, 2, 3]]
    assert off.tolist() == [0, 1, 3, 5, 6]
    assert rows.tolist() == [0, 0, 2, 0, 2, 2, -1, -1, -1]
    assert slots.tolist() == [[1, 3, 0], [-1, -1, -1], [2, 4, 5]]
    assert np.allclose(w.sum(1), [1, 0, 1]) and w[2].tolist() == [1.0, 0.0, 0.0]
