"""Accumulated key weights and eviction by weight, from the definitions: NumPy, fp64, one sequence
and kv head at a time."""

from __future__ import annotations

import numpy as np


def attend_with_weights(q: np.ndarray, K: np.ndarray, V: np.ndarray, first_pos: int, scale: float):
    """q [n, Hq, D] at positions first_pos .., K and V [L, Hkv, D]: (out [n, Hq, D], weights
    [Hkv, L]: the softmax weight each key received over the queries that see it and the q heads of
    its kv head)."""
    n, hq, d = q.shape
    hkv = K.shape[1]
    group = hq // hkv
    out = np.zeros((n, hq, d))
    weights = np.zeros((hkv, K.shape[0]))
    for h in range(hq):
        for i in range(n):
            p = first_pos + i + 1
            a = scale * (K[:p, h // group] @ q[i, h])
            w = np.exp(a - a.max())
            w /= w.sum()
            out[i, h] = w @ V[:p, h // group]
            weights[h // group, :p] += w
    return out, weights


def choose(w: np.ndarray, L: int, keep: int, recent: int) -> np.ndarray:
    """Positions that stay, ascending: the last min(recent, k) and the k - r of the largest weight
    before them (ties: the lowest position; NaN counts as -infinity), k = min(keep, L)."""
    k = min(keep, L)
    r = min(recent, k)
    key = [(-np.inf if np.isnan(x) else float(x)) for x in w[:L - r]]
    order = sorted(range(L - r), key=lambda j: (-key[j], j))[:k - r]
    return np.array(sorted(order) + list(range(L - r, L)), dtype=np.int64)
