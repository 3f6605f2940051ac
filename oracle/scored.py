"""Masked, capped and biased attention, and the accepted path of a drafted tree,
by their definitions in float64 (test infrastructure; no code is shared with
the CUDA path)."""
from __future__ import annotations

import numpy as np


def causal_rows(T: int, n: int, window: int = 0, prefix: int = 0, doc_start=None):
    """(at [n], key_at [T], visible [n, T]) of the n newest positions of a sequence of length T."""
    at = np.arange(T - n, T)
    p = np.arange(T)
    see = (p[None, :] <= at[:, None]) | (p[None, :] < prefix)
    if window:
        see &= at[:, None] - p[None, :] < window
    if doc_start is not None:
        see &= p[None, :] >= np.asarray(doc_start)[:, None]
    return at, p, see & (at[:, None] >= 0)


def tree_rows(T: int, masks, window: int = 0):
    """The same for a drafted tree: masks[i] has bit j where node i sees node j."""
    n = len(masks)
    base = T - n
    bits = np.array([[int(m) >> j & 1 for j in range(n)] for m in masks], dtype=bool).reshape(n, n)
    depth = bits.sum(1) - 1
    at, key_at = base + depth, np.concatenate([np.arange(base), base + depth])
    see = np.concatenate([np.ones((n, base), bool), bits], axis=1)
    if window:
        see &= at[:, None] - key_at[None, :] < window
    return at, key_at, see


def scored_attention(q, k, v, at, key_at, see, scale, softcap=0.0, slopes=None):
    """q [n, H, D], k and v [Hkv, T, D] -> (o [n, H, D], lse [n, H]); rows that see nothing: 0, -inf."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, H, D = q.shape
    G = H // k.shape[0]
    o, lse = np.zeros((n, H, D)), np.full((n, H), -np.inf)
    far = np.abs(np.asarray(at)[:, None] - np.asarray(key_at)[None, :]).astype(np.float64)
    for h in range(H):
        x = (q[:, h] @ k[h // G].T) * scale
        if softcap:
            x = softcap * np.tanh(x / softcap)
        if slopes is not None:
            x = x - float(slopes[h]) * far
        for i in range(n):
            s = np.flatnonzero(see[i])
            if len(s):
                top = x[i, s].max()
                e = np.exp(x[i, s] - top)
                o[i, h] = e @ v[h // G][s] / e.sum()
                lse[i, h] = top + np.log(e.sum())
    return o, lse


def accepted_positions(T: int, n: int, path):
    """Position of the old cache that each position of the new one holds (length T; past the new length: itself)."""
    where = np.arange(T)
    base = T - n
    where[base:base + len(path)] = base + np.asarray(path, dtype=np.int64)
    return where
