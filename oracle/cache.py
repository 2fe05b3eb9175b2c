"""Rotary positions, the paged key-value cache and one new token's attention over
it, in float64 and from their definitions. TEST INFRASTRUCTURE ONLY (see
oracle/attention.py)."""
from __future__ import annotations

import numpy as np

from .attention import _as_f64, softmax_weights


def rope(x, positions, axis, freq, interleaved: bool, inverse: bool = False):
    """x [T, H, d] with pair i of every head turned by positions[axis[i], t] *
    freq[i] radians (negated for ``inverse``, which is the gradient: the
    rotation's transpose). Pairs: (i, i + n) or (2 i, 2 i + 1)."""
    y = _as_f64(x).copy()
    n = len(freq)
    sign = -1.0 if inverse else 1.0
    for i, (a, f) in enumerate(zip(axis, freq)):
        # whole turns go before cos and sin: float64 angles of far positions
        angle = sign * np.asarray(positions[a], dtype=np.float64) * f
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        u, v = y[:, :, i0].copy(), y[:, :, i1].copy()
        y[:, :, i0] = u * c - v * s
        y[:, :, i1] = u * s + v * c
    return y


def gather(pages, table_row, n):
    """The first n rows [n, H_kv, d] of a sequence: token p in page
    table_row[p // page_size], slot p % page_size."""
    size = pages.shape[1]
    return np.stack([pages[table_row[p // size], p % size] for p in range(n)]) if n else \
        np.zeros((0, *pages.shape[2:]))


def decode(q, keys, values, scale: float):
    """One query token per sequence: q [B, H, d], keys and values lists of
    [n_b, H_kv, d]. Returns (O [B, H, d], lse [B, H]); a sequence without keys
    gives O = 0 and lse = -inf."""
    q = _as_f64(q)
    B, H, _ = q.shape
    o = np.zeros_like(q)
    lse = np.full((B, H), -np.inf)
    for b in range(B):
        k, v = _as_f64(keys[b]), _as_f64(values[b])
        if k.shape[0] == 0:
            continue
        for h in range(H):
            g = h // (H // k.shape[1])
            P, row = softmax_weights(q[b, h][None], k[:, g], scale)
            o[b, h] = (P @ v[:, g])[0]
            lse[b, h] = row[0]
    return o, lse
