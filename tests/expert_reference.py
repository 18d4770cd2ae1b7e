"""Plain references of the expert-routing operators, used by the tests only:
one walk over the pairs in their order, float64 for sums.  Shares no code with
the library."""
from __future__ import annotations

import numpy as np

from tests import op_reference as ref


def rows_of(tokens, top_k, experts, capacity):
    pairs = tokens * top_k
    return experts * capacity if capacity else (pairs + 15 * min(experts, pairs)) // 16 * 16


def plan(ids, experts, capacity=0):
    """(offsets, counts, slots, sources) of ids [tokens, top_k]."""
    tokens, top_k = ids.shape
    kept = [[] for _ in range(experts)]
    for pair, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < experts and (not capacity or len(kept[e]) < capacity):
            kept[e].append(pair)
    slots = np.full(tokens * top_k, -1, np.int32)
    sources = np.full(rows_of(tokens, top_k, experts, capacity), -1, np.int32)
    offsets = [0]
    for pairs in kept:
        at = offsets[-1] + np.arange(len(pairs))
        slots[pairs] = at
        sources[at] = pairs
        offsets.append(offsets[-1] + (capacity or -(-len(pairs) // 16) * 16))
    return (np.array(offsets, np.int32), np.array([len(p) for p in kept], np.int32),
            slots.reshape(tokens, top_k), sources)


def gather(x, sources, top_k, end, weights=None):
    """bf16 bits of the rows before `end`: those of x [tokens, cols] (bits), or of
    their fp32 products with the pairs' weights, rounded."""
    y = np.zeros((end, x.shape[1]), np.uint16)
    live = np.nonzero(sources[:end] >= 0)[0]
    pairs = sources[live]
    y[live] = x[pairs // top_k]
    if weights is not None:
        v = (y[live].astype(np.uint32) << 16).view(np.float32)
        with np.errstate(all="ignore"):
            y[live] = ref.bf16_round(weights.reshape(-1)[pairs].astype(np.float32)[:, None] * v)
    return y


def combine(x, slots, weights=None, base=None):
    """float64 (y, sum of magnitudes) for x [rows, cols] in float64."""
    tokens, top_k = slots.shape
    y = np.zeros((tokens, x.shape[1])) if base is None else base.astype(np.float64).copy()
    size = np.abs(y)
    for k in range(top_k):
        live = np.nonzero(slots[:, k] >= 0)[0]
        term = x[slots[live, k]]
        if weights is not None:
            term = term * weights[live, k].astype(np.float64)[:, None]
        y[live] += term
        size[live] += np.abs(term)
    return y, size


def combine_weight_gradient(dy, x, slots):
    """float64 (dw, sum of magnitudes)."""
    dw, size = np.zeros(slots.shape), np.zeros(slots.shape)
    for k in range(slots.shape[1]):
        live = np.nonzero(slots[:, k] >= 0)[0]
        term = dy[live] * x[slots[live, k]]
        dw[live, k], size[live, k] = term.sum(1), np.abs(term).sum(1)
    return dw, size
