"""What stands around an attention layer's products, in numpy float64, from the definitions: the norm
and rotation of the heads of Q and K, attention with a sliding window and sinks, and their gradients."""
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


def window_seen(n, L, window, sinks):
    """Whether query i of the n last of L keys sees key j: bool [n, L]."""
    p, j = np.arange(n)[:, None] + L - n, np.arange(L)
    return (j <= p) & ((j > p - window) | (j < sinks))


def window_attention(q, k, v, window, sinks, scale):
    """One sequence: q [n, H, d], k and v [L, kv_heads, d] -> (O [n, H, d], lse [H, n])."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, H, d = q.shape
    G = H // k.shape[1]
    seen = window_seen(n, len(k), window, sinks)
    O, lse = np.zeros((n, H, d)), np.full((H, n), -np.inf)
    for h in range(H if len(k) else 0):
        s = np.where(seen, q[:, h] @ k[:, h // G].T * scale, -np.inf)
        m = s.max(1)
        m[m == -np.inf] = 0
        e = np.exp(s - m[:, None])
        z = e.sum(1)
        O[:, h] = e @ v[:, h // G] / np.where(z > 0, z, 1)[:, None]
        with np.errstate(divide="ignore"):
            lse[h] = m + np.log(z)
    return O, lse


def window_attention_bwd(q, k, v, do, window, sinks, scale):
    """Gradients of sum(dO * O) for one sequence: (dq, dk, dv)."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    O, lse = window_attention(q, k, v, window, sinks, scale)
    H, G = q.shape[1], q.shape[1] // k.shape[1]
    seen = window_seen(len(q), len(k), window, sinks)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for h in range(H if len(k) else 0):
        kh, vh = k[:, h // G], v[:, h // G]
        s = q[:, h] @ kh.T * scale
        p = np.where(seen, np.exp(np.where(seen, s - np.where(lse[h] > -np.inf, lse[h], 0)[:, None], -np.inf)), 0)
        ds = p * (do[:, h] @ vh.T - (do[:, h] * O[:, h]).sum(1, keepdims=True)) * scale
        dq[:, h] = ds @ kh
        dk[:, h // G] += ds.T @ q[:, h]
        dv[:, h // G] += p.T @ do[:, h]
    return dq, dk, dv
