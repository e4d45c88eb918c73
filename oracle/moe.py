"""Routing of tokens to experts and the combination of their rows, token by token."""
from __future__ import annotations

import math

import numpy as np

HUGE = float(np.finfo(np.float32).max)


def route(logits, top: int, renorm: bool):
    """ids, weights (fp64), offsets, row_ids, slots of fp-valued logits [tokens, experts]."""
    x = np.asarray(logits, dtype=np.float64)
    tokens, experts = x.shape
    ids = np.full((tokens, top), -1, dtype=np.int32)
    weights = np.zeros((tokens, top))
    for t in range(tokens):
        row = [(-math.inf if math.isnan(v) else min(v, HUGE)) for v in x[t].tolist()]
        order = sorted(range(experts), key=lambda e: (-row[e], e))
        chosen = [e for e in order[:top] if row[e] > -math.inf]
        if not chosen:
            continue
        first = row[chosen[0]]
        over = chosen if renorm else [e for e in range(experts) if row[e] > -math.inf]
        total = math.fsum(math.exp(row[e] - first) for e in over)
        for j, e in enumerate(chosen):
            ids[t, j] = e
            weights[t, j] = math.exp(row[e] - first) / total
    offsets, row_ids, slots = sort_pairs(ids, experts)
    return ids, weights, offsets, row_ids, slots


def sort_pairs(ids, experts: int):
    tokens, top = ids.shape
    offsets = np.zeros(experts + 1, dtype=np.int32)
    row_ids = np.full(tokens * top, -1, dtype=np.int32)
    slots = np.full((tokens, top), -1, dtype=np.int32)
    n = 0
    for e in range(experts):
        offsets[e] = n
        for t, j in zip(*np.nonzero(ids == e)):
            row_ids[n] = t
            slots[t, j] = n
            n += 1
    offsets[experts] = n
    return offsets, row_ids, slots


def combine(y, slots, weights):
    """(out fp64 [tokens, d], the sum of the absolute values of its terms)."""
    y = np.asarray(y, dtype=np.float64)
    out = np.zeros((slots.shape[0], y.shape[1]))
    mag = np.zeros_like(out)
    for t in range(slots.shape[0]):
        for j in range(slots.shape[1]):
            if 0 <= slots[t, j] < y.shape[0]:
                term = float(weights[t, j]) * y[slots[t, j]]
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag
