"""Rotary positions over a token grid, and the per-head norm with that rotation,
in fp64 (oracle; test infrastructure).

Token n of a (T, H, W) grid in raster order has positions (t, h, w).  The first
rd = dt + dh + dw elements of a row form rd/2 pairs; pair i of an axis with dim
m turns by pos * theta**(-2i/m).  Tokens past the grid take no rotation.

The functions work on rows in source (raster) order; perm is applied by the
caller (gather of the result, scatter of a gradient).
"""
from __future__ import annotations

import numpy as np


def rope_angles(grid, dims, n: int, theta: float = 10000.0, start=(0.0, 0.0, 0.0)):
    """Angles [n, rd/2] of the first n tokens."""
    T, H, W = grid
    out = np.zeros((n, sum(dims) // 2))
    for tok in range(min(n, T * H * W)):
        pos = (tok // (H * W) + start[0], (tok // W) % H + start[1], tok % W + start[2])
        p = 0
        for x, m in zip(pos, dims):
            for i in range(m // 2):
                out[tok, p] = x * theta ** (-2.0 * i / m)
                p += 1
    return out


def _pairs(rd: int, layout: str):
    i = np.arange(rd // 2)
    return (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rd // 2)


def rotate(x, angles, layout: str = "interleaved", inverse: bool = False):
    """x [..., n, d] with every row's pairs turned by angles [n, rd/2]."""
    x = np.asarray(x, dtype=np.float64)
    a, b = _pairs(2 * angles.shape[1], layout)
    c, s = np.cos(angles), np.sin(angles) * (-1.0 if inverse else 1.0)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def _rows(w, x):
    """A weight [d] or [H, d] beside x [B, H, n, d]."""
    w = np.asarray(w, dtype=np.float64)
    return w if w.ndim == 1 else w[:, None, :]


def norm(x, w, eps: float = 1e-6):
    """(x / sqrt(mean(x^2) + eps), and that times w) for x [B, H, n, d]."""
    x = np.asarray(x, dtype=np.float64)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return n, n * _rows(w, x)


def norm_rope(x, w, angles=None, layout: str = "interleaved", eps: float = 1e-6):
    u = norm(x, w, eps)[1]
    return u if angles is None else rotate(u, angles, layout)


def norm_rope_grad(dy, x, w, angles=None, layout: str = "interleaved", eps: float = 1e-6):
    """(dx, dw) of norm_rope; dw has w's shape."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    du = dy if angles is None else rotate(dy, angles, layout, inverse=True)
    n = norm(x, w, eps)[0]
    dw = (du * n).sum(axis=(0, 2))
    dw = dw.sum(0) if np.ndim(w) == 1 else dw
    dn = du * _rows(w, x)
    dx = (dn - n * (dn * n).mean(-1, keepdims=True)) / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return dx, dw
