"""The paged K/V cache and attention over it, float64 (oracle side; test infrastructure only).

What follows a prompt that the ring has prefilled: K and V are kept, and new tokens attend over
what is kept.  The pages have no counterpart for the storage; the attention is theirs ("Context
& Expert Parallelism", section "Context parallelism: splitting the sequence": token i attends to
every j <= i), for the last rows of a sequence only, with a window of keys where one is given.

    cache     row of (sequence b, position j) = page block_table[b, j // P], row j % P
    e4m3      scale = 2^e, e = max(-120, least e with max|x| <= 448 * 2^e); value = x / scale to the
              nearest number of 4 significant bits that is a multiple of 2^-9, ties to even
    attention row t of n at position i = L - n + t sees j < L with j <= i (causal) and, under a
              window W, j > i - W or j < sinks; a row that sees nothing has out = 0, lse = -inf
"""
from __future__ import annotations

import numpy as np


def quantise(x):
    """Rows x [..., d] -> (values / scale as e4m3 numbers, scales), float64.  A row with an
    infinity or a NaN is zeros with the scale NaN."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    amax = np.abs(x).max(-1)
    m, e = np.frexp(amax)                       # amax = m 2^e, m in [0.5, 1)
    e = np.where(m <= 0.875, e - 9, e - 8)      # 448 = 0.875 * 2^9
    e = np.where(amax == 0, -120, np.maximum(e, -120))
    y = np.ldexp(x, -e[..., None])
    _, ye = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(ye - 4, -9))
    codes = np.rint(y / step) * step
    return codes, np.where(bad, np.nan, np.ldexp(1.0, e))


def visible(n, L, causal=True, window=0, sinks=0):
    """[n, L] booleans: which keys each of the last n rows of a sequence of L sees."""
    i = (L - n + np.arange(n))[:, None]
    j = np.arange(L)[None, :]
    see = np.ones((n, L), dtype=bool)
    if causal:
        see &= j <= i
    if window:
        see &= (j > i - window) | (j < sinks)
    return see


def attention(q, k, v, causal=True, window=0, sinks=0):
    """q [n, Hq, d] over k, v [L, Hkv, d] -> out [n, Hq, d], lse [n, Hq], and for error bounds
    sum_j p_j |v_j| [n, Hq, d] and the largest sum_t |q_t k_jt| of a visible key [n, Hq]."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    n, Hq, d = q.shape
    L = k.shape[0]
    g = Hq // k.shape[1]
    see = visible(n, L, causal, window, sinks)
    some = see.any(1)
    out, mag = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse, size = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    if L == 0 or not some.any():
        return out, lse, mag, size
    for h in range(Hq):
        kh, vh = k[:, h // g], v[:, h // g]
        used = see.any(0)
        kh, vh = np.where(used[:, None], kh, 0.0), np.where(used[:, None], vh, 0.0)
        with np.errstate(invalid="ignore", over="ignore"):
            s = np.where(see, q[:, h] @ kh.T, -np.inf)[some]
            M = s.max(1, keepdims=True)
            p = np.exp(s - M)
            z = p.sum(1, keepdims=True)
            p = p / z
            lse[some, h] = (M + np.log(z))[:, 0]
            # a key that a row does not see has no part in it, whatever its v holds
            for r, row in zip(np.nonzero(some)[0], p) if not np.isfinite(vh).all() else ():
                out[r, h] = row[see[r]] @ vh[see[r]]
            if np.isfinite(vh).all():
                out[some, h] = p @ vh
                mag[some, h] = p @ np.abs(vh)
            size[some, h] = np.where(see[some], np.abs(q[some, h]) @ np.abs(kh).T, 0.0).max(1)
    return out, lse, mag, size
