"""Norm and rotation of query and key rows, and their gradients, float64 (oracle side; test infrastructure
only).

    y = w * x / sqrt(mean(x^2) + eps); pairs (j, j + rot/2), or (2j, 2j + 1), of y's first `rot` elements turned by
    the angle whose cosine and sine are cos_sin[position, j] and cos_sin[position, rot/2 + j]; the whole times `scale`

The rotation is written as a matrix a token, so that its transpose is the gradient's.
"""
from __future__ import annotations

import numpy as np


def turn_matrix(cos_sin, d, interleaved):
    """cos_sin [T, rot] -> [T, d, d]: z = M y."""
    cos_sin = np.asarray(cos_sin, dtype=np.float64)
    T, rot = cos_sin.shape
    m = np.zeros((T, d, d))
    m[:, np.arange(rot, d), np.arange(rot, d)] = 1.0
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        c, s = cos_sin[:, j], cos_sin[:, rot // 2 + j]
        m[:, a, a], m[:, a, b], m[:, b, a], m[:, b, b] = c, -s, s, c
    return m


def forward(x, w, cos_sin, interleaved=False, eps=1e-6, scale=1.0):
    """x [T, H, d], w [d] or None, cos_sin [T, rot] -> z [T, H, d] and the sum of its terms' absolute values."""
    x = np.asarray(x, dtype=np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, dtype=np.float64)
    y = w * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * scale
    m = turn_matrix(cos_sin, x.shape[-1], interleaved)
    return np.einsum("tij,thj->thi", m, y), np.einsum("tij,thj->thi", np.abs(m), np.abs(y))


def backward(x, w, cos_sin, dz, interleaved=False, eps=1e-6, scale=1.0):
    """-> dx, dw, and the sums of absolute values of the terms that dx [T, H, d] and dw [d] add up."""
    x, dz = np.asarray(x, dtype=np.float64), np.asarray(dz, dtype=np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, dtype=np.float64)
    m = turn_matrix(cos_sin, x.shape[-1], interleaved)
    g = np.einsum("tji,thj->thi", m, dz) * scale
    g_abs = np.einsum("tji,thj->thi", np.abs(m), np.abs(dz)) * abs(scale)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u, u_abs = w * g, np.abs(w) * g_abs
    dx = r * (u - x * r * r * (u * x).mean(-1, keepdims=True))
    dx_abs = r * (u_abs + np.abs(x) * r * r * (u_abs * np.abs(x)).mean(-1, keepdims=True))
    return dx, (g * x * r).sum((0, 1)), dx_abs, (g_abs * np.abs(x) * r).sum((0, 1))
