"""Tables of frequencies at the ends of their arguments (CPU only)."""
from __future__ import annotations

import numpy as np
import pytest

from bit_quantized_matmul_amd import binding as B


@pytest.mark.parametrize("change", [dict(low=0.0), dict(low=-1.0), dict(theta=1.0), dict(theta=0.5)])
def test_pairs_refuses_what_its_logarithms_do(change):
    with pytest.raises(ValueError, match="pairs needs low above 0 and theta above 1"):
        B.rope_freqs(64, kind="pairs", factor=4.0, context=4096, **change)
    if "low" in change:                                                  # the other kinds need no logarithm
        assert np.all(np.isfinite(B.rope_freqs(64, kind="turns", factor=4.0, context=4096, **change)))


@pytest.mark.parametrize("kind", ["turns", "pairs"])
@pytest.mark.parametrize("rotary", [2, 12, 128])
def test_contexts_in_which_no_pair_turns_often(kind, rotary):
    """All pairs turn fewer than `low` times in the context: all are divided by factor."""
    plain = B.rope_freqs(rotary)
    assert np.allclose(B.rope_freqs(rotary, kind=kind, factor=4.0, context=1, low=1.0, high=32.0), plain / 4.0, rtol=1e-15)


@pytest.mark.parametrize("kind", ["turns", "pairs"])
def test_contexts_in_which_all_pairs_do(kind):
    plain = B.rope_freqs(16, theta=4.0)
    assert np.allclose(B.rope_freqs(16, theta=4.0, kind=kind, factor=4.0, context=1 << 20), plain, rtol=1e-15)
