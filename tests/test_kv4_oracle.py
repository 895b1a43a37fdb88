"""The 4-bit cache's oracle, pinned on the CPU, and the entry points' refusals
that return before any CUDA call."""
import numpy as np
import pytest
import torch

import online_softmax_06_gb300 as fa
from kv4_common import Pool, bf16_rows
from oracle import kv4

FORMATS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa.build()
    return fa.lib()


def test_bf16_rounding_is_torchs_and_single():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(4000), rng.standard_normal(500) * 1e30,
                        rng.standard_normal(500) * 1e-39, [0.0, np.inf, -np.inf, 3.4e38, -3.4e38]])
    x32 = x.astype(np.float32)
    want = torch.from_numpy(x32).to(torch.bfloat16).double().numpy()
    assert np.array_equal(kv4.bf16(x32.astype(np.float64)), want)
    # just above a half-way point: one rounding goes up, two go to the even neighbour
    assert kv4.bf16(1 + 2.0 ** -8 + 2.0 ** -40) == 1 + 2.0 ** -7
    assert kv4.bf16(1 + 2.0 ** -8) == 1.0


@pytest.mark.parametrize("d,group", FORMATS)
def test_places_cover_the_cell_once(d, group):
    seen = np.zeros((kv4.cell_bytes(d, group), 2), int)
    for v in (False, True):
        for t in range(16):
            for i in range(d):
                b, s = kv4.code_place(d, v, t, i)
                seen[b, s // 4] += 1
            for g in range(d // group):
                p = kv4.par_place(d, group, v, t, g)
                seen[p:p + 4] += 1
    assert (seen == 1).all()
    assert fa.fa_kv4_page_bytes(48, d, group) == 3 * kv4.cell_bytes(d, group)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantise_against_a_search(group):
    rng = np.random.default_rng(2)
    x = bf16_rows(rng, 7, 2, 128, std=1.7, offset=0.4)
    code, scale, lo = kv4.quantise(x, group)
    val = kv4.values(code, scale, lo)
    g = x.reshape(7, 2, -1, group)
    # the least value is held exactly; every other within half a step of its
    # value (and the top one within the scale's own rounding, 15 * 2^-8 steps)
    assert np.array_equal(val.reshape(g.shape).min(-1), g.min(-1))
    step = scale[..., None]
    assert (np.abs(val.reshape(g.shape) - g) <= step * (0.5 + 2.0 ** -20)).all()
    # no other code is nearer
    alt = lo[..., None, None] + step[..., None] * np.arange(16)
    best = np.abs(alt - g[..., None]).min(-1)
    assert (np.abs(val.reshape(g.shape) - g) <= best + step * 1e-6).all()


def test_quantise_special_groups():
    x = np.zeros((5, 1, 64))
    x[0] = 2.5                                  # constant: scale 0, held exactly
    x[1, 0, 3] = np.nan
    x[2, 0, 40] = np.inf                        # second group only (group 32)
    big = float(torch.finfo(torch.bfloat16).max)
    x[3, 0, :2] = (big, -big)                   # max - min is beyond float32
    x[4, 0, 0] = 2.0 ** -133                    # range below the least normal scale
    code, scale, lo = kv4.quantise(x, 32)
    val = kv4.values(code, scale, lo)
    assert (val[0] == 2.5).all() and (code[0] == 0).all()
    assert np.isnan(val[1, 0, :32]).all() and (val[1, 0, 32:] == 0).all()
    assert (val[2, 0, :32] == 0).all() and np.isnan(val[2, 0, 32:]).all()
    assert np.isfinite(scale[3]).all() and code[3, 0, 0] == 15 and code[3, 0, 1] == 0
    assert abs(val[3, 0, 2]) <= scale[3, 0, 0] / 2 * (1 + 2.0 ** -8)
    assert (val[4] == 0).all()


@pytest.mark.parametrize("d,group", FORMATS)
def test_write_then_read(d, group):
    rng = np.random.default_rng(3)
    pool = Pool([37, 0, 1], 2, d, group, 32, seed=4)
    k = [bf16_rows(rng, n, 2, d) for n in pool.lengths]
    v = [bf16_rows(rng, n, 2, d) for n in pool.lengths]
    pool.fill(k, v)
    for b in range(3):
        K, V = pool.rows(b)
        for x, y in ((k[b], K), (v[b], V)):
            assert np.array_equal(kv4.values(*kv4.quantise(x, group)), y)
    # a second write of some rows changes those alone
    before = pool.bytes.copy()
    k2, v2 = bf16_rows(rng, 5, 2, d), bf16_rows(rng, 5, 2, d)
    kv4.write(pool.bytes, pool.table[0], np.arange(10, 15), k2, v2, 32, group)
    K, V = pool.rows(0)
    assert np.array_equal(K[10:15], kv4.values(*kv4.quantise(k2, group)))
    pool.bytes, after = before, pool.bytes
    K0, V0 = pool.rows(0)
    keep = np.r_[0:10, 15:37]
    assert np.array_equal(K[keep], K0[keep]) and np.array_equal(V[keep], V0[keep])
    assert not np.array_equal(before, after)


@pytest.mark.parametrize("causal", [False, True])
def test_attention_oracle_against_torch(causal):
    rng = np.random.default_rng(5)
    Nq, L, H, Hkv, d = 6, 19, 6, 2, 64
    q, K, V = rng.standard_normal((Nq, H, d)), rng.standard_normal((L, Hkv, d)), \
        rng.standard_normal((L, Hkv, d))
    O, lse = kv4.attention(q, K, V, 0.2, causal)
    t = lambda x: torch.from_numpy(x).transpose(0, 1)  # noqa: E731
    k, v = (t(x).repeat_interleave(H // Hkv, 0) for x in (K, V))
    mask = torch.ones(Nq, L, dtype=torch.bool).tril(L - Nq) if causal else None
    want = torch.nn.functional.scaled_dot_product_attention(t(q), k, v, attn_mask=mask, scale=0.2)
    assert np.abs(O - want.transpose(0, 1).numpy()).max() < 1e-13
    s = 0.2 * t(q) @ k.transpose(1, 2)
    if causal:
        s = s.masked_fill(~mask, -np.inf)
    assert np.abs(lse - torch.logsumexp(s, -1).numpy()).max() < 1e-13
    # fewer keys than queries: the first rows see none
    O, lse = kv4.attention(q, K[:4], V[:4], 0.2, True)
    assert (O[:2] == 0).all() and (lse[:, :2] == -np.inf).all() and np.isfinite(lse[:, 2:]).all()
    # a NaN behind the mask does not reach the rows that do not see it
    V2 = V.copy()
    V2[-1] = np.nan
    O2, _ = kv4.attention(q, K, V2, 0.2, True)
    O1, _ = kv4.attention(q, K, V, 0.2, True)
    assert np.array_equal(O2[:-1], O1[:-1]) and np.isnan(O2[-1]).all()


def test_refusals_without_gpu():
    pb = fa.fa_kv4_page_bytes
    assert pb(16, 128, 64) == 16 * (128 + 16)
    assert pb(0, 128, 64) == fa.FA_ERR_UNSUPPORTED
    assert pb(24, 128, 64) == fa.FA_ERR_UNSUPPORTED
    assert pb(16, 96, 32) == fa.FA_ERR_UNSUPPORTED
    assert pb(16, 64, 128) == fa.FA_ERR_UNSUPPORTED
    assert pb(16, 128, 16) == fa.FA_ERR_UNSUPPORTED
    for call in (fa.fa_kv4_append, fa.fa_kv4_read):
        def go(k=16, v=16, ks=256, vs=256, cache=16, pages=4, ps=16, table=16, mp=2, lens=16,
               cu=None, B=1, N=1, total=1, Hkv=2, d=128, group=64):
            return call(k, v, ks, vs, cache, pages, ps, table, mp, lens, cu, B, N, total, Hkv, d,
                        group)
        assert go(B=-1) == fa.FA_ERR_BAD_SIZE
        assert go(N=-1) == fa.FA_ERR_BAD_SIZE
        assert go(pages=-1) == fa.FA_ERR_BAD_SIZE
        assert go(total=2) == fa.FA_ERR_BAD_SIZE           # dense: total = B N
        assert go(ks=255 + 1 - 8) == fa.FA_ERR_BAD_SIZE    # a row does not hold its heads
        assert go(vs=260) == fa.FA_ERR_MISALIGNED
        assert go(k=8) == fa.FA_ERR_MISALIGNED
        assert go(cache=8) == fa.FA_ERR_MISALIGNED
        assert go(lens=2) == fa.FA_ERR_MISALIGNED
        assert go(v=None) == fa.FA_ERR_NULL_POINTER
        assert go(lens=None) == fa.FA_ERR_NULL_POINTER
        assert go(d=80) == fa.FA_ERR_UNSUPPORTED
        assert go(ps=8) == fa.FA_ERR_UNSUPPORTED
        assert go(ps=1 << 20, mp=1 << 12) == fa.FA_ERR_TOO_LARGE
        assert go(B=0, total=0) == fa.FA_OK
        assert go(N=0, total=0, k=None) == fa.FA_OK
        assert go(Hkv=0, k=None) == fa.FA_OK


def test_helper_refusals_without_gpu():
    with pytest.raises(fa.FaError):
        fa.kv4_cache(2, 1, 24, 128, device="cpu")
    cache = fa.kv4_cache(2, 1, 16, 128, device="cpu")
    assert cache.shape == (2, 1, 16 * 144) and cache.dtype == torch.uint8
    k = torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.kv4_append(k, k, cache, table, lens)            # no CUDA tensors
    with pytest.raises(ValueError):
        fa.kv4_append(k.float(), k.float(), cache, table, lens)


def test_attention_refusals_without_gpu():
    wb = fa.fa_attention_kv4_workspace_bytes
    assert wb(1, -1, 1, 5000, 8, 2, 128) == fa.FA_ERR_BAD_SIZE
    assert wb(1, 1, 1, 5000, 9, 2, 128) == fa.FA_ERR_BAD_SIZE
    assert wb(1, 1, 1, 5000, 8, 0, 128) == fa.FA_ERR_BAD_SIZE
    assert wb(1, 1, 1, 5000, 8, 2, 96) == fa.FA_ERR_UNSUPPORTED
    # a descriptor and two parts a range, of 4 or 8 rows (456 ranges) or 16 (304)
    for Nq, rows in ((1, 4), (2, 8), (3, 16), (4, 16), (5, 16), (500, 16)):
        assert wb(1, Nq, Nq, 1025, 8, 2, 128) == (304 if rows == 16 else 456) * (32 + 2 * rows * (8 + 512))

    assert wb(1, 1, 1, 1024, 8, 2, 128) == 0                     # whole heads: no parts
    assert wb(1, 1, 1, -1, 8, 2, 128) == fa.FA_ERR_BAD_SIZE

    # many rows: fp16 Q [total, H, d], K and V [B, Hkv, tiles of 128, d], the factors
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    assert wb(3, 900, 2000, 1000, 32, 8, 128) == (
        up(2000 * 32 * 256) + 2 * 3 * 8 * 1024 * 256 + up(2000 * 32 * 4) + up(3 * 8 * 8 * 8))
    assert wb(64, 1, 64, 1000, 32, 8, 128) == 0

    def go(q=256, qs=1024, cache=256, pages=4, ps=16, table=256, mp=80, lens=256, cu=None, o=256,
           lse=256, B=1, Nq=1, total=1, Nk=1100, H=8, Hkv=2, d=128, group=64, ws=256, wsb=1 << 30):
        return fa.fa_attention_kv4(q, qs, cache, pages, ps, table, mp, lens, cu, o, lse, B, Nq,
                                   total, Nk, H, Hkv, d, group, 1.0, 1, ws, wsb)
    assert go(B=-1) == fa.FA_ERR_BAD_SIZE
    assert go(Nk=1281) == fa.FA_ERR_BAD_SIZE                 # more keys than the table holds
    assert go(H=7) == fa.FA_ERR_BAD_SIZE
    assert go(Hkv=0) == fa.FA_ERR_BAD_SIZE
    assert go(total=2) == fa.FA_ERR_BAD_SIZE
    assert go(qs=1016) == fa.FA_ERR_BAD_SIZE
    assert go(wsb=1000) == fa.FA_ERR_BAD_SIZE
    assert go(qs=1028) == fa.FA_ERR_MISALIGNED
    assert go(ws=16) == fa.FA_ERR_MISALIGNED
    assert go(o=8) == fa.FA_ERR_MISALIGNED
    assert go(d=96) == fa.FA_ERR_UNSUPPORTED
    assert go(group=16) == fa.FA_ERR_UNSUPPORTED
    assert go(q=None) == fa.FA_ERR_NULL_POINTER
    assert go(cache=None) == fa.FA_ERR_NULL_POINTER
    assert go(ws=None) == fa.FA_ERR_NULL_POINTER
    assert go(B=1025, total=1025) == fa.FA_ERR_TOO_LARGE
    assert go(B=1024, total=1024 << 14, Nq=1 << 14, mp=1 << 20, Nk=1 << 24) == fa.FA_ERR_TOO_LARGE
    assert go(B=0, total=0) == fa.FA_OK
    assert go(Nq=0, total=0) == fa.FA_OK
    assert go(H=0, Hkv=0) == fa.FA_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are none: no device may take the call")
def test_loose_bounds_of_packed_queries_are_no_refusal():
    """A call's size goes by its rows: the queries of one sequence, however many may be
    allowed, do not count for each sequence."""
    def go(B, Nq, total, Nk, H, Hkv=8, d=128, cu=256):
        return fa.fa_attention_kv4(256, H * d, 256, 4, 256, 256, 1 << 20, 256, cu, 256, 256, B, Nq,
                                   total, Nk, H, Hkv, d, 64, 1.0, 1, 256, 1 << 40)
    # one query each of 1024 sequences, most = all: 16-row tiles on up to 131072 keys
    assert go(1024, 1024, 1024, 131072, 64) == fa.FA_ERR_NO_DEVICE
    assert go(1024, 2 ** 31 - 1, 1024, 131072, 64) == fa.FA_ERR_NO_DEVICE
    # 256 queries each of 256 sequences, in the form for many rows, which has no such count
    assert go(256, 65536, 65536, 4096, 64) == fa.FA_ERR_NO_DEVICE
    # what does not fit 32 bits is refused: (2^25 / 16 * 8 + 1024) * 2052 * 8 blocks
    assert go(1024, 1 << 25, 1 << 25, 1 << 18, 64) == fa.FA_ERR_TOO_LARGE
    assert go(1024, 1 << 16, 1 << 26, 1 << 18, 64, cu=None) == fa.FA_ERR_TOO_LARGE
