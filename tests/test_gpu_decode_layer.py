"""The example of a decoder layer: rope, cache, attention and experts as they are used together."""
from __future__ import annotations

import importlib.util
import os

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,context,hidden,heads,kv_heads,ffn,experts,top", [(3, 200, 256, 4, 2, 128, 8, 2), (1, 70, 128, 2, 1, 72, 4, 4)])
def test_example_runs(seqs, context, hidden, heads, kv_heads, ffn, experts, top):
    spec = importlib.util.spec_from_file_location("fp8_decode_layer", os.path.join(ROOT, "examples", "fp8_decode_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    rel, us = module.run(seqs, context, hidden, heads, kv_heads, ffn, experts, top, replays=3)   # raises where a replay differs
    # activations are quantized around the two projections alone: codes off by half a step (2^-4) of random sign
    assert us > 0 and rel < 0.1
