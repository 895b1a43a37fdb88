"""4-bit paged key/value cache, reference side (TEST INFRASTRUCTURE ONLY).

The format of include/fa.h, value by value, and attention on the values held,
in float64 on the CPU.  The code of a value is decided in float32 by the
definition; here each of its operations is done in float64 and rounded to
float32 once.  Nothing is shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np

CELL = 16


def f32(x) -> np.ndarray:
    """Rounded to float32 once, kept in float64."""
    return np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64)


def bf16(x) -> np.ndarray:
    """float64 values rounded to bf16 in one step (nearest, ties to even)."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    ok = np.isfinite(x) & (x != 0)
    e = np.maximum(np.frexp(x[ok])[1] - 1, -126)
    step = np.ldexp(1.0, e - 7)
    y = np.rint(x[ok] / step) * step
    y[np.abs(y) >= 2.0 ** 128] *= np.inf
    out[ok] = y
    return out


def quantise(x, group: int):
    """(codes uint8 [..., d], scale, min float64 [..., d / group]) of bf16 values x."""
    with np.errstate(invalid="ignore", over="ignore"):
        g = np.asarray(x, dtype=np.float64).reshape(*np.shape(x)[:-1], np.shape(x)[-1] // group, group)
        lo, hi = g.min(-1), g.max(-1)
        scale = bf16(f32(f32(hi / 2 - lo / 2) * float(np.float32(2.0 / 15.0))))
        scale = np.where(scale < 2.0 ** -126, 0.0, scale)
        inv = np.where(scale > 0, f32(1.0 / np.where(scale > 0, scale / 2, 1.0)), 0.0)
        t = f32(g / 2 - lo[..., None] / 2)
        code = np.clip(np.rint(f32(t * inv[..., None])), 0, 15)
        bad = ~np.isfinite(g).all(-1)
        code = np.where(bad[..., None], 0, np.nan_to_num(code)).astype(np.uint8)
    return (code.reshape(np.shape(x)), np.where(bad, np.nan, scale), np.where(bad, np.nan, lo))


def values(code, scale, lo) -> np.ndarray:
    """min + scale * code in float64."""
    g = code.astype(np.float64).reshape(*scale.shape, code.shape[-1] // scale.shape[-1])
    return (lo[..., None] + scale[..., None] * g).reshape(code.shape)


def cell_bytes(d: int, group: int) -> int:
    return CELL * d + 2 * CELL * (d // group) * 4


def code_place(d: int, is_v: bool, t: int, i: int):
    """(byte in the cell, shift) of value i of token t."""
    if not is_v:
        w = i // 8
        j, c = divmod(w, 4)
        return t * (d // 2) + 4 * (c * (d // 32) + j) + (i % 8) // 2, 4 * (i % 2)
    q, g = divmod(i // 4, 8)
    a = t * (d // 2) + 2 * (g * (d // 32) + q) + (i % 4) // 2
    s, r = divmod(a, 32)
    return CELL * (d // 2) + ((s & ~3) | ((s + (s >> 2)) & 3)) * 32 + r, 4 * (i % 2)


def par_place(d: int, group: int, is_v: bool, t: int, g: int) -> int:
    return CELL * d + (CELL * (d // group) * 4 if is_v else 0) + (t * (d // group) + g) * 4


def _places(d, group):
    code = np.array([[[code_place(d, v, t, i) for i in range(d)] for t in range(CELL)]
                     for v in (False, True)])
    par = np.array([[[par_place(d, group, v, t, g) for g in range(d // group)]
                     for t in range(CELL)] for v in (False, True)])
    return code[..., 0], code[..., 1], par


def _bf16_bits(x) -> np.ndarray:
    """Bit patterns of float64 values that bf16 holds exactly (NaN: 0x7fc0)."""
    bits = (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7fc0), bits)


def write(cache, table, pos, k, v, page_size: int, group: int) -> None:
    """Rows k, v [T, Hkv, d] of one sequence at positions pos [T], into cache
    (uint8 [pages, Hkv, bytes], changed in place) by its row of the page table."""
    T, H, d = k.shape
    byte, shift, par = _places(d, group)
    cells = cache.reshape(cache.shape[0], H, page_size // CELL, cell_bytes(d, group))
    for is_v, x in ((0, k), (1, v)):
        code, scale, lo = quantise(x, group)
        pair = np.stack((_bf16_bits(scale), _bf16_bits(lo)), -1)
        for r in range(T):
            page, off = int(table[pos[r] // page_size]), int(pos[r] % page_size)
            t = off % CELL
            for h in range(H):
                c = cells[page, h, off // CELL]
                c[byte[is_v, t]] = 0               # a byte holds two values of one row
                np.bitwise_or.at(c, byte[is_v, t], code[r, h] << shift[is_v, t].astype(np.uint8))
                for g in range(d // group):
                    c[par[is_v, t, g]:par[is_v, t, g] + 4] = pair[r, h, g].view(np.uint8)


def read(cache, table, length: int, page_size: int, d: int, group: int):
    """The values (K, V) float64 [length, Hkv, d] of one sequence's tokens."""
    byte, shift, par = _places(d, group)
    H = cache.shape[1]
    cells = cache.reshape(cache.shape[0], H, page_size // CELL, cell_bytes(d, group))
    out = np.zeros((2, length, H, d))
    for r in range(length):
        off = r % page_size
        t = off % CELL
        c = cells[int(table[r // page_size]), :, off // CELL]
        for is_v in (0, 1):
            code = (c[:, byte[is_v, t]] >> shift[is_v, t].astype(np.uint8)) & 15
            p = par[is_v, t][:, None] + np.arange(4)
            bits = np.ascontiguousarray(c[:, p]).view(np.uint16).astype(np.uint32) << 16
            pair = bits.view(np.float32).astype(np.float64)          # [H, groups, 2]
            out[is_v, r] = values(code, pair[..., 0], pair[..., 1])
    return out[0], out[1]


def attention(q, K, V, scale: float, causal: bool):
    """(O [Nq, H, d], lse [H, Nq]) of queries q [Nq, H, d] on K, V [L, Hkv, d] in
    float64; causal: query i sees keys j <= i + L - Nq.  A row without a key:
    O = 0, lse = -inf."""
    Nq, H, d = q.shape
    L, Hkv, _ = K.shape
    O, lse = np.zeros((Nq, H, d)), np.full((H, Nq), -np.inf)
    seen = np.ones((Nq, L), bool)
    if causal:
        seen = np.arange(L)[None, :] <= np.arange(Nq)[:, None] + (L - Nq)
    rows = seen.any(1)
    if not rows.any():
        return O, lse
    for h in range(H):
        s = scale * (q[rows, h].astype(np.float64) @ K[:, h // (H // Hkv)].T)
        s = np.where(seen[rows], s, -np.inf)
        m = s.max(1, keepdims=True)
        p = np.where(seen[rows], np.exp(s - m), 0.0)
        z = p.sum(1, keepdims=True)
        with np.errstate(invalid="ignore"):
            # a value behind the mask never counts, whatever it is
            pv = np.stack([pr[sr] @ V[sr, h // (H // Hkv)] for pr, sr in zip(p, seen[rows])])
        O[rows, h] = pv / z
        lse[h, rows] = (m + np.log(z))[:, 0]
    return O, lse
