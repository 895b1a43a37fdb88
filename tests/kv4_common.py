"""Paged 4-bit cache test cases: pools of pages, tables and rows, made on the CPU."""
from __future__ import annotations

import numpy as np
import torch

import online_softmax_06_gb300 as fa
from oracle import kv4


class Pool:
    """A pool of pages in random order for sequences of the given lengths.

    Bytes that no token occupies are 0xff: codes 15 and NaN parameters, which
    show up in any result that they reach.  Table entries behind a sequence's
    last page are -1.
    """

    def __init__(self, lengths, Hkv, d, group, page_size, seed=0, spare_pages=3, extra_cols=2):
        rng = np.random.default_rng(seed)
        self.lengths, self.Hkv, self.d, self.group = list(lengths), Hkv, d, group
        self.page_size = page_size
        per = [-(-L // page_size) for L in lengths]
        self.num_pages = sum(per) + spare_pages
        order = rng.permutation(self.num_pages).astype(np.int32)
        self.table = np.full((len(per), max(per, default=0) + extra_cols), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        nbytes = page_size // kv4.CELL * kv4.cell_bytes(d, group)
        self.bytes = np.full((self.num_pages, Hkv, nbytes), 0xff, np.uint8)

    def fill(self, k_rows, v_rows, first=None):
        """The oracle writes sequence b's rows from position first[b] (default 0) on."""
        for b, (k, v) in enumerate(zip(k_rows, v_rows)):
            p0 = 0 if first is None else first[b]
            kv4.write(self.bytes, self.table[b], np.arange(p0, p0 + len(k)), k, v, self.page_size,
                      self.group)

    def rows(self, b, length=None):
        L = self.lengths[b] if length is None else length
        return kv4.read(self.bytes, self.table[b], L, self.page_size, self.d, self.group)


def bf16_rows(rng, n, Hkv, d, std=1.0, offset=0.0):
    """float64 [n, Hkv, d], every value a bf16 number."""
    x = rng.standard_normal((n, Hkv, d)) * std + offset
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


def gpu_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).cuda()


def gpu_i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def same_cache(got, want, d, group):
    """Equal byte for byte, but for the sign of a zero minimum."""
    if np.array_equal(got, want):
        return True
    cell = kv4.cell_bytes(d, group)
    g, w = got.reshape(-1, cell), want.reshape(-1, cell)
    if not np.array_equal(g[:, :16 * d], w[:, :16 * d]):
        return False
    zero = lambda x: np.where(x == 0x8000, 0, x)  # noqa: E731
    gp, wp = (np.ascontiguousarray(x[:, 16 * d:]).view(np.uint16) for x in (g, w))
    return np.array_equal(zero(gp), zero(wp))


__all__ = ["Pool", "bf16_rows", "gpu_bf16", "gpu_i32", "same_cache", "fa", "kv4"]
