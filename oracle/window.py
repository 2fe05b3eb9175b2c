"""Attention within a sliding window and to the first tokens, in float64 and from its
definition. TEST INFRASTRUCTURE ONLY (see oracle/attention.py)."""
from __future__ import annotations

import numpy as np

from .attention import _as_f64


def visible(Lq: int, Lk: int, left, right, sinks: int) -> np.ndarray:
    """[Lq, Lk]: query i, at place p = i + Lk - Lq, sees key j if j <= p + right and
    (j >= p - left or j < sinks); left, right None: no end."""
    p = np.arange(Lq)[:, None] + (Lk - Lq)
    j = np.arange(Lk)[None]
    near = np.ones((Lq, Lk), dtype=bool) if left is None else j >= p - left
    return (near | (j < sinks)) & (np.ones((Lq, Lk), dtype=bool) if right is None else j <= p + right)


def weights(q_h, k_h, seen, scale: float):
    """One head: P, zero where not seen (rows that see nothing too), and lse."""
    S = np.where(seen, scale * (q_h @ k_h.T), -np.inf)
    m = S.max(axis=1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    E = np.exp(S - m)
    total = E.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(total))[:, 0]
    return E / np.where(total > 0, total, 1.0), lse


def forward(q, k, v, left, right, sinks, scale):
    """q [B, H, Lq, d], k, v [B, H_kv, Lk, d]: (O, lse)."""
    q, k, v = _as_f64(q), _as_f64(k), _as_f64(v)
    B, H, Lq, _ = q.shape
    seen = visible(Lq, k.shape[2], left, right, sinks)
    o, lse = np.zeros_like(q), np.zeros((B, H, Lq))
    for b in range(B):
        for h in range(H):
            g = h // (H // k.shape[1])
            P, lse[b, h] = weights(q[b, h], k[b, g], seen, scale)
            o[b, h] = P @ v[b, g]
    return o, lse


def backward(q, k, v, do, left, right, sinks, scale):
    """Gradients of sum(O dO): (dQ, dK, dV)."""
    q, k, v, do = (_as_f64(x) for x in (q, k, v, do))
    B, H, Lq, _ = q.shape
    seen = visible(Lq, k.shape[2], left, right, sinks)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b in range(B):
        for h in range(H):
            g = h // (H // k.shape[1])
            P, _ = weights(q[b, h], k[b, g], seen, scale)
            dP = do[b, h] @ v[b, g].T
            dS = P * (dP - (P * dP).sum(axis=1, keepdims=True))
            dq[b, h] = scale * dS @ k[b, g]
            dk[b, g] += scale * dS.T @ q[b, h]
            dv[b, g] += P.T @ do[b, h]
    return dq, dk, dv
