"""Pins of the oracle's rotary positions, cache and attention (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from bit_quantized_matmul_amd import binding as B
from oracle import fp8 as of8
from oracle import kv as okv
from oracle import moe as omoe


def test_rope_turns_pairs():
    x = np.zeros((3, 1, 6))
    x[:, 0, :4] = [1.0, 2.0, 3.0, 4.0]
    x[:, 0, 4:] = [7.0, 8.0]
    f = [np.pi / 2, np.pi]                                        # a quarter and a half turn a position
    half = okv.rope(x, [0, 1, 3], f)
    assert np.allclose(half[0], x[0])
    assert np.allclose(half[1, 0], [-3.0, -2.0, 1.0, -4.0, 7.0, 8.0])
    assert np.allclose(half[2, 0], [3.0, -2.0, -1.0, -4.0, 7.0, 8.0])
    inter = okv.rope(x, [0, 1, 3], f, interleaved=True, mscale=2.0)
    assert np.allclose(inter[1, 0], [-4.0, 2.0, -6.0, -8.0, 7.0, 8.0])
    back = okv.rope(half, [0, 1, 3], f, backward=True)
    assert np.allclose(back, x)


def test_scales_are_the_smallest_powers_of_two():
    assert okv.scale_for([448.0]) == 1.0 and okv.scale_for([-449.0]) == 2.0 and okv.scale_for([224.0, np.inf]) == 0.5
    assert okv.scale_for([0.0]) == 2.0 ** -126 and okv.scale_for([np.nan]) == 2.0 ** -126


def test_append_rescales_what_a_page_holds():
    c = okv.empty(2, 1, 4)
    pages = np.array([[1]])
    v = np.array([[[1.0, -2.0, 3.0, 448.0]], [[896.0, 0.0, 1.0, -5.0]]])
    okv.append(c, v[:1], v[:1], pages, [1])
    assert c["k_scale"][1, 0] == 1.0
    okv.append(c, v[1:], v[1:], pages, [2])
    assert c["k_scale"][1, 0] == 2.0
    k, w, there = okv.values(c, pages, 0, 2, 0, 4)
    assert np.array_equal(k, v[:, 0]) and np.array_equal(w, v[:, 0]) and there.all()   # all are multiples of a step


def test_attention_of_one_key_is_its_value_and_of_none_is_zero():
    rng = np.random.default_rng(0)
    c = okv.empty(3, 2, 8)
    k, v = rng.standard_normal((2, 1, 2, 8))
    pages = np.array([[2]])
    okv.append(c, k, v, pages, [1])
    out, *_ = okv.attention(rng.standard_normal((1, 4, 8)), c, pages, [1])
    want = of8.decode(c["v"][2, :, :8, 0]) * c["v_scale"][2][:, None]
    assert np.allclose(out[0], np.repeat(want, 2, 0))
    out, *_ = okv.attention(rng.standard_normal((1, 4, 8)), c, np.array([[-1]]), [1])
    assert np.array_equal(out, np.zeros((1, 4, 8)))


def test_freqs_of_long_contexts():
    f = B.rope_freqs(8)
    assert np.allclose(f, 10000.0 ** (-np.arange(4) / 4.0))
    assert np.allclose(B.rope_freqs(8, kind="linear", factor=4.0), f / 4.0)
    base = B.rope_freqs(8, kind="base", factor=4.0)
    assert np.isclose(base[0], f[0]) and np.isclose(base[-1], f[-1] / 4.0)
    for kind in ("turns", "pairs"):
        g = B.rope_freqs(128, kind=kind, factor=8.0, context=8192, low=1.0, high=32.0)
        plain = B.rope_freqs(128)
        turns = 8192 * plain / (2 * np.pi)
        assert np.array_equal(g[0], plain[0]) and np.isclose(g[-1], plain[-1] / 8.0)
        assert np.all(np.diff(g / plain) <= 0)
        if kind == "turns":
            mid = (turns > 1) & (turns < 32)
            part = (turns[mid] - 1) / 31
            assert np.allclose(g[mid], plain[mid] * (part + (1 - part) / 8))
            assert np.allclose(g[turns >= 32], plain[turns >= 32])
    for bad in (dict(rotary=7), dict(rotary=8, kind="other"), dict(rotary=8, kind="turns"), dict(rotary=8, factor=0.0)):
        with pytest.raises(ValueError):
            B.rope_freqs(**bad)


def test_expert_layer_of_one_expert():
    rng = np.random.default_rng(1)
    w13, w2 = rng.standard_normal((1, 6, 4)).astype(np.float32), rng.standard_normal((1, 4, 3)).astype(np.float32)
    q13, s13 = of8.quant_weight(w13[0])
    q2, s2 = of8.quant_weight(w2[0])
    x = rng.standard_normal((2, 4))
    out, _ = omoe.ffn(x, q13[None], s13[None], q2[None], s2[None], np.zeros((2, 1)), 1)
    m13, m2 = of8.weight_values(q13, s13)[:, :4], of8.weight_values(q2, s2)[:, :3]
    h = x @ m13.T
    assert np.allclose(out, (h[:, :3] / (1 + np.exp(-h[:, :3])) * h[:, 3:]) @ m2.T)
