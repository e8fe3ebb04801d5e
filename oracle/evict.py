"""What cached positions have had of attention, and eviction by it, float64 (oracle side; test infrastructure
only).

    weights  w'[j] = (j < L - n ? decay w[j] : 0) + sum over the rows that see j, and the heads of the KV head, of
             exp(q.k_j - lse)
    evict    n = min(keep, L) positions stay: the first `sinks` and the last `recent` first, then by weight (NaN above all
             numbers), of equal ones the lower position
"""
from __future__ import annotations

import numpy as np

from oracle.paged import visible


def add_weights(old, q, lse, k, decay=1.0, causal=True, window=0, sinks=0):
    """old [L, Hkv], q [n, Hq, d], lse [n, Hq], k [L, Hkv, d] -> new [L, Hkv], and for error bounds the largest
    sum_t |q_t k_jt| of a row that sees the key [L, Hkv]."""
    q, lse, k = (np.asarray(x, dtype=np.float64) for x in (q, lse, k))
    n, L = q.shape[0], k.shape[0]
    g = q.shape[1] // k.shape[1]
    see = visible(n, L, causal, window, sinks)
    new = np.zeros((L, k.shape[1]))
    size = np.zeros((L, k.shape[1]))
    if n == 0:
        return np.array(old, dtype=np.float64), size
    base = L - n
    if decay and base > 0:
        new[:base] = decay * np.asarray(old, dtype=np.float64)[:base]
    for h in range(q.shape[1]):
        for t in range(n):
            j = np.nonzero(see[t])[0]
            if lse[t, h] == -np.inf:
                continue
            s = k[j, h // g] @ q[t, h]
            new[j, h // g] += np.exp(s - lse[t, h])
            size[j, h // g] = np.maximum(size[j, h // g], np.abs(k[j, h // g]) @ np.abs(q[t, h]))
    return new, size


def stay(w, keep, sinks=0, recent=0):
    """w [L] -> the positions that stay, ascending."""
    L = len(w)

    def rank(j):
        forced = j < sinks or j >= L - recent
        return (0 if forced else 1, 0 if forced or np.isnan(w[j]) else 1, 0.0 if forced or np.isnan(w[j]) else -float(w[j]), j)

    return sorted(sorted(range(L), key=rank)[:max(0, min(keep, L))])
