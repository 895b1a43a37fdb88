"""Window attention test cases: sequences on the CPU, their three layouts, and derived tolerances.

Tolerances.  A probability is rounded to bf16, off by half a step, 2^-8 of it at most; so is the
output, and the sum that divides it is corrected by the largest one's rounding: 2^-8 of mean_p |v|,
and 2^-7 of |O|.  Scores are fp32 sums of d exact products: off by ds <= d 2^-24 sum |q k| scale,
which moves a probability by 2 ds (its own and the sum's) and the logsumexp by ds, each with some
2^-20 for exp2, log2 and the conversion of the scale.
"""
from __future__ import annotations

import numpy as np
import torch

import online_softmax_06_gb300 as fa
from oracle import layer


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


class Batch:
    """Sequences of n queries and L keys in one of the layouts: "dense" (all alike, all rows keys),
    "cache" (rows with room for more keys), "packed"; "fused": packed, with rows further apart."""

    def __init__(self, n, L, H, Hkv, d, form, seed=0, room=None, spare=5):
        rng = np.random.default_rng(seed)
        self.n, self.L, self.H, self.Hkv, self.d, self.form = list(n), list(L), H, Hkv, d, form
        make = lambda m, h: bf16(rng.standard_normal((m, h, d)))  # noqa: E731
        self.q = [make(m, H) for m in n]
        off = rng.standard_normal((Hkv, d))                     # keys with an offset of their own
        self.k = [bf16(rng.standard_normal((m, Hkv, d)) + off) for m in L]
        self.v = [make(m, Hkv) for m in L]
        self.kw = {}
        nan = lambda m, h: torch.full((m, h, d), float("nan"), dtype=torch.bfloat16)  # noqa: E731
        if form in ("dense", "cache"):
            room = max(list(L) + [1]) + (3 if form == "cache" else 0) if room is None else room
            stack = lambda x, m, h: torch.stack([torch.cat((y, nan(m - len(y), h))) for y in x])  # noqa: E731
            self.gq = torch.stack(self.q).cuda()
            self.gk, self.gv = stack(self.k, room, Hkv).cuda(), stack(self.v, room, Hkv).cuda()
            if form == "cache":
                self.kw["seqlens_k"] = torch.tensor(L, dtype=torch.int32, device="cuda")
            return
        cat = lambda x, h: torch.cat(list(x) + [nan(spare, h)])  # noqa: E731
        gq, gk, gv = (cat(x, h).cuda() for x, h in ((self.q, H), (self.k, Hkv), (self.v, Hkv)))
        if form == "fused":
            def apart(x):
                rows = torch.full((len(x), x.shape[1] + 2, d), float("nan"), dtype=x.dtype, device="cuda")
                rows[:, 1:-1] = x
                return rows[:, 1:-1]
            gq, gk, gv = apart(gq), apart(gk), apart(gv)
        self.gq, self.gk, self.gv = gq, gk, gv
        cu = lambda x: torch.tensor(np.concatenate(([0], np.cumsum(x))), dtype=torch.int32, device="cuda")  # noqa: E731
        self.kw.update(cu_seqlens_q=cu(n), cu_seqlens_k=cu(L), max_q=max(n), max_k=max(L))

    def split(self, o, lse):
        """(O, lse [H, n]) of each sequence, as float64."""
        o, lse = f64(o), f64(lse)
        if self.form in ("dense", "cache"):
            return list(zip(o, lse))
        at = np.concatenate(([0], np.cumsum(self.n)))
        return [(o[i:j], lse[:, i:j]) for i, j in zip(at[:-1], at[1:])]


def score_error(q, k, scale, d):
    """ds above for each query and head [n, H, 1]."""
    G = q.shape[1] // k.shape[1]
    if len(k) == 0:
        return np.zeros(q.shape[:2] + (1,))
    top = np.abs(k).max(0).repeat(G, 0)                          # [H, d]
    return d * 2.0 ** -24 * scale * (np.abs(q) * top).sum(-1, keepdims=True) + 2.0 ** -20


def check_forward(batch, o, lse, window, sinks, scale=None):
    scale = batch.d ** -0.5 if scale is None else scale
    for b, (go, gl) in enumerate(batch.split(o, lse)):
        q, k, v = f64(batch.q[b]), f64(batch.k[b]), f64(batch.v[b])
        if len(q) == 0:
            continue
        ro, rl = layer.window_attention(q, k, v, window, sinks, scale)
        spread = layer.window_attention(q, k, np.abs(v), window, sinks, scale)[0]
        ds = score_error(q, k, scale, batch.d)
        tol = (2.0 ** -8 + 2 * ds) * spread + 2.0 ** -7 * np.abs(ro)
        assert np.all(np.abs(go - ro) <= tol), ("O", b, np.nanmax(np.abs(go - ro) - tol))
        none = rl == -np.inf
        assert np.array_equal(gl == -np.inf, none)
        err = np.abs(np.where(none, 0, gl) - np.where(none, 0, rl))
        tol = ds[..., 0].T + 2.0 ** -20 * (1 + np.abs(np.where(none, 0, rl)))
        assert np.all(err <= tol), ("lse", b, (err / tol).max())


def check_gradients(batch, do, grads, window, sinks, scale=None):
    """dS is rounded to bf16 (2^-8), as is P; D = dO . O has O's rounding (2^-7 of |dO| |O| and what
    P's does to it); the gradients are rounded at the end.  do: float64 [n, H, d] per sequence."""
    scale = batch.d ** -0.5 if scale is None else scale
    at = np.concatenate(([0], np.cumsum(batch.n)))
    for b in range(len(batch.n)):
        q, k, v, g = f64(batch.q[b]), f64(batch.k[b]), f64(batch.v[b]), do[b]
        if len(q) == 0:
            continue
        n, H, d = q.shape
        G = H // k.shape[1]
        ref = layer.window_attention_bwd(q, k, v, g, window, sinks, scale)
        O, lse = layer.window_attention(q, k, v, window, sinks, scale)
        spread = layer.window_attention(q, k, np.abs(v), window, sinks, scale)[0]
        ds_err = score_error(q, k, scale, d)                      # relative error of P
        seen = layer.window_seen(n, len(k), window, sinks)
        tol = [np.zeros_like(x) for x in ref]
        for h in range(H):
            kh, vh = k[:, h // G], v[:, h // G]
            p = np.where(seen, np.exp(np.where(seen, q[:, h] @ kh.T * scale - lse[h][:, None], -np.inf)), 0)
            dp = g[:, h] @ vh.T
            mass = np.abs(g[:, h]) @ np.abs(vh).T                 # what dP sums
            D = (g[:, h] * O[:, h]).sum(1, keepdims=True)
            # D's error: O's in each value, times dO; sums of d products in fp32
            eo = (2.0 ** -8 + 2 * ds_err[:, h]) * spread[:, h] + 2.0 ** -7 * np.abs(O[:, h])
            eD = (np.abs(g[:, h]) * eo).sum(1, keepdims=True)
            e = p * (eD + d * 2.0 ** -24 * mass) + (2 * ds_err[:, h] + 2.0 ** -20) * p * np.abs(dp - D)
            # dQ has the sum of these errors times a mean of the keys taken off, at most the largest key:
            # sum_j e_j (K_j - mean) in place of sum_j e_j K_j
            tol[0][:, h] = e.sum(1, keepdims=True) * np.abs(kh).max(0) * scale
            e = e + 2.0 ** -8 * p * np.abs(dp - D)
            tol[0][:, h] += e @ np.abs(kh) * scale
            tol[1][:, h // G] += e.T @ np.abs(q[:, h]) * scale
            tol[2][:, h // G] += ((2.0 ** -8 + 2 * ds_err[:, h] + 2.0 ** -20) * p).T @ np.abs(g[:, h])
        for name, got, r, t in zip("qkv", grads, ref, tol):
            got = f64(got)
            got = got[b] if batch.form == "dense" else got[at[b]:at[b + 1]]
            t = t + 2.0 ** -8 * (np.abs(r) + t) + 1e-12
            err = np.abs(got - r)
            assert np.all(err <= t), ("d" + name, b, np.unravel_index(np.argmax(err / t), err.shape), (err / t).max())


__all__ = ["Batch", "bf16", "check_forward", "check_gradients", "f64", "fa", "layer", "score_error"]
