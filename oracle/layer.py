"""What stands around an attention layer's products, in numpy float64, from the definitions: the norm
and rotation of the heads of Q and K with its gradient."""
from __future__ import annotations

import numpy as np


def rotate(x, positions, inv_freq, interleaved, back=False):
    """x [total, heads, d] with its first 2 len(inv_freq) values turned by position."""
    y = np.array(x, np.float64)
    n = len(inv_freq)
    ang = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang), np.sin(-ang if back else ang)
    ia = np.arange(0, 2 * n, 2) if interleaved else np.arange(n)
    ib = ia + (1 if interleaved else n)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def norm_rope(x, weight, positions, inv_freq, eps, interleaved):
    x = np.asarray(x, np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(x * r * weight, positions, inv_freq, interleaved)


def norm_rope_bwd(x, dy, weight, positions, inv_freq, eps, interleaved):
    """(dx, dweight)."""
    x = np.asarray(x, np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = rotate(dy, positions, inv_freq, interleaved, back=True)
    h = g * weight
    hat = x * r
    return r * (h - hat * (h * hat).mean(-1, keepdims=True)), (g * hat).sum((0, 1))
