"""Attention over the 4-bit paged cache against the float64 oracle.

Tolerances, from the arithmetic (half a step is finfo.eps / 2 of the value: u16 =
2^-11 for fp16 with its 10 fraction bits, ub = 2^-8 for bf16 with its 7):
  * a score is a sum of d products of exact factors; the tensor core rounds it
    once per 16 of them and the groups' sums add a few fp32 roundings more,
    12 steps of 2^-23 at most of the sum of magnitudes:
        eS = scale * max_j sum_k |q_k| (15 s_jk + |m_jk|) * 2^-19;
  * |lse - ref| <= 2 eS + 2^-20 (exp2's error) + 2^-22 |lse|;
  * P s is rounded to fp16 and multiplies codes up to 15; below 2^-14 of a
    row's largest P s the step is fixed, which L <= 2^13 keys can add up to the
    same again; errors of S act on P twice (weight and sum); O is rounded:
        |O - ref| <= 2 u16 * 15 max_j s_j + 4 eS max |v| + ub |ref|;
  * with many query rows K, V and P are rounded to fp16, K and V once each with
    their tile's power of two: eS grows by scale * max_j sum_k |q_k k_jk| u16, and
    |O - ref| by 2 u16 max |v| in the place of the first term (V's rounding and P's).
"""
import math

import numpy as np
import pytest
import torch

from gpu_common import device_error_clear, require_gpu
from kv4_common import Pool, bf16_rows, fa, gpu_bf16, gpu_i32, kv4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def dev():
    d = require_gpu()
    fa.fa_get_device_error()
    return d


def params(pool, b):
    """(largest 15 s + |m| of K, largest s of V, largest |value| of V) over the sequence."""
    K, V = pool.rows(b)
    g = pool.group
    span = lambda x: (x.reshape(*x.shape[:2], -1, g).max(-1) -  # noqa: E731
                      x.reshape(*x.shape[:2], -1, g).min(-1))
    if not len(K):
        return np.zeros((0, pool.Hkv, pool.d)), 0.0, 0.0
    # a group's largest code is 15 (or its scale 0): 15 s is the span
    k_abs = np.repeat(span(K), g, -1) + np.abs(K)
    return (k_abs, float(np.nanmax(span(V), initial=0)) / 15,
            float(np.nanmax(np.abs(V), initial=0)))


def check(pool, q_rows, O, lse, scale, causal, many=False):
    """O [total, H, d], lse [H, total] against the oracle, sequence by sequence."""
    at = 0
    for b, q in enumerate(q_rows):
        n, H, d = q.shape
        K, V = pool.rows(b)
        Or, lr = kv4.attention(q, K, V, scale, causal)
        o, l = O[at:at + n].double().cpu().numpy(), lse[:, at:at + n].double().cpu().numpy()
        at += n
        k_abs, s_v, v_max = params(pool, b)
        eS = 0.0
        if len(K) and n:
            for h in range(H):
                eS0 = abs(scale) * float(np.nanmax(np.abs(q[:, h]) @ k_abs[:, h // (H // pool.Hkv)].T)) \
                    * 2.0 ** -19
                eS = max(eS, eS0)
                if many:
                    eS = max(eS, abs(scale) * float(np.nanmax(
                        np.abs(q[:, h]) @ np.abs(K[:, h // (H // pool.Hkv)]).T)) * 2.0 ** -11 + eS0)
        assert np.array_equal(np.isneginf(l), np.isneginf(lr)), b
        assert np.array_equal(np.isnan(l), np.isnan(lr)), b
        fin = np.isfinite(lr)
        err_l = np.abs(l[fin] - lr[fin])
        assert (err_l <= 2 * eS + 2.0 ** -20 + 2.0 ** -22 * np.abs(lr[fin])).all(), (b, err_l.max(), eS)
        assert np.array_equal(np.isnan(o), np.isnan(Or)), b
        ok = ~np.isnan(Or)
        err = np.abs(o[ok] - Or[ok])
        tol = 4 * eS * v_max + 2.0 ** -8 * np.abs(Or[ok]) + \
            (2.0 ** -10 * v_max if many else 2.0 ** -10 * 15 * s_v)
        assert (err <= tol).all(), (b, (err - tol).max(), err.max())


def make(lens, Nq, H, Hkv, d, group, page, seed, k_off=1.0, q_std=1.5, v_std=1.0, **kw):
    """(pool, q rows of each sequence); Nq: one count, or one for each sequence."""
    rng = np.random.default_rng(seed)
    nq = [Nq] * len(lens) if np.isscalar(Nq) else Nq
    pool = Pool(lens, Hkv, d, group, page, seed=seed + 1, **kw)
    off = rng.standard_normal((Hkv, d)) * k_off
    k = [bf16_rows(rng, n, Hkv, d, offset=off) for n in lens]
    v = [bf16_rows(rng, n, Hkv, d, std=v_std) for n in lens]
    pool.fill(k, v)
    return pool, [bf16_rows(rng, n, H, d, std=q_std) for n in nq]


def run(pool, q_rows, causal, packed, scale=None, pad=0, lens=None, **kw):
    """(O [total, H, d], lse [H, total]) through the helper, dense or packed."""
    cache = torch.from_numpy(pool.bytes).cuda()
    table, sl = gpu_i32(pool.table), gpu_i32(pool.lengths if lens is None else lens)
    kw = dict(group=pool.group, causal=causal, scale=scale, **kw)
    if packed:
        n = [len(q) for q in q_rows]
        x = np.concatenate(q_rows + [np.ones((pad, *q_rows[0].shape[1:]))])
        o, l = fa.attention_kv4(gpu_bf16(x), cache, table, sl,
                                cu_seqlens=gpu_i32(np.concatenate([[0], np.cumsum(n)])),
                                max_q=max(n), **kw)
        return o, l
    o, l = fa.attention_kv4(gpu_bf16(np.stack(q_rows)), cache, table, sl, **kw)
    B, Nq, H, d = o.shape
    return o.reshape(-1, H, d), l.transpose(0, 1).reshape(H, -1)


CASES = [
    # lens, Nq, H, Hkv, d, group, page, causal, packed
    ([1], 1, 1, 1, 128, 128, 16, True, False),
    ([15, 16, 17, 0, 130], 1, 8, 2, 128, 64, 16, True, False),
    ([127, 128, 129, 1000], 1, 4, 4, 128, 32, 48, True, False),
    ([300, 77], 1, 16, 1, 64, 64, 32, False, False),
    ([257, 31, 2], 1, 24, 2, 64, 32, 16, True, False),           # 12 heads a kv head: two tiles of 8
    ([4000], 1, 8, 1, 128, 64, 64, True, False),                 # split over many CTAs
    ([2100, 5, 900], 4, 8, 2, 128, 128, 128, True, False),       # 16 rows
    ([150, 3, 0, 64], 5, 14, 2, 128, 64, 16, True, False),       # 35 rows: two tiles; rows without a key
    ([150, 3, 0, 64], 5, 14, 2, 64, 64, 16, False, False),
    ([600, 70, 129], [100, 1, 129], 8, 2, 128, 32, 32, True, True),
    ([600, 70, 0], [33, 0, 2], 2, 2, 64, 32, 64, True, True),
    ([40, 300], [64, 7], 3, 1, 128, 128, 256, False, True),      # more queries than keys
    ([130, 4100, 9], 1, 3, 1, 128, 64, 32, True, False),         # 3 rows
    ([2100, 1, 33], 2, 4, 2, 128, 32, 64, True, False),          # 2 queries x 2 heads
    ([1500, 2, 260], 3, 2, 2, 64, 32, 16, True, False),          # 3 queries; rows without a key
    ([3000, 700], [4, 1], 1, 1, 128, 128, 128, False, True),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_against_the_oracle(case):
    lens, Nq, H, Hkv, d, group, page, causal, packed = case
    pool, q = make(lens, Nq, H, Hkv, d, group, page, seed=100)
    scale = 1 / math.sqrt(d)
    O, lse = run(pool, q, causal, packed)
    check(pool, q, O, lse, scale, causal)
    device_error_clear()


@pytest.mark.parametrize("B", [300, 1024])
def test_many_sequences(B):
    rng = np.random.default_rng(110)
    lens = [int(x) for x in rng.integers(0, 40, B)]
    pool, q = make(lens, 1, 2, 1, 64, 64, 16, seed=111)
    O, lse = run(pool, q, True, False)
    check(pool, q, O, lse, 1 / 8, True)
    device_error_clear()


def test_scores_that_grow_with_the_position():
    """Every key outscores all earlier ones by far: the reference moves on every tile."""
    d, L = 128, 700
    rng = np.random.default_rng(120)
    pool = Pool([L], 1, d, 32, 64, seed=121)
    k = bf16_rows(rng, L, 1, d, std=0.05) + np.linspace(0, 8, L)[:, None, None]
    pool.fill([kv4.bf16(k)], [bf16_rows(rng, L, 1, d)])
    q = [np.abs(bf16_rows(rng, 1, 8, d, std=1.0))]
    for sign in (1, -1):
        O, lse = run(pool, [sign * q[0]], True, False, scale=0.5)
        check(pool, [sign * q[0]], O, lse, 0.5, True)


def test_values_of_far_apart_scales():
    """P s goes into fp16 relative to the row's largest P s, not to its largest P."""
    d, L = 128, 400
    rng = np.random.default_rng(130)
    for lo, hi in ((1e-6, 1.0), (1e-30, 1e-30), (1e30, 1e30), (1.0, 1e-5)):
        pool = Pool([L], 1, d, 64, 16, seed=131)
        v = bf16_rows(rng, L, 1, d)
        v[:200] *= lo
        v[200:] *= hi
        k = bf16_rows(rng, L, 1, d, std=0.3)
        k[200:] -= 2.0                       # the second half scores far below the first
        pool.fill([kv4.bf16(k)], [kv4.bf16(v)])
        q = [np.abs(bf16_rows(rng, 1, 4, d))]
        O, lse = run(pool, q, True, False, scale=0.15)
        K, V = pool.rows(0)
        Or, lr = kv4.attention(q[0], K, V, 0.15, True)
        o = O.double().cpu().numpy()
        # the bound of the module's head, but with each key's own weight: the sum
        # over the keys of P 15 s, and a fixed step of 2^-24 of the largest P s
        s = 0.15 * q[0][0] @ K[:, 0].T
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        sv = (V[:, 0].reshape(L, 2, 64).max(-1) - V[:, 0].reshape(L, 2, 64).min(-1)).max(-1) / 15
        eS = 0.15 * (np.abs(q[0][0]) @ (np.abs(K[:, 0]) + 15).T).max() * 2.0 ** -19
        tol = (p * sv).sum(1) * (15 * 2.0 ** -11 + 4 * eS) + L * 15 * 2.0 ** -24 * (p * sv).max(1)
        assert (np.abs(o[0] - Or[0]) <= tol[:, None] + 2.0 ** -8 * np.abs(Or[0])).all(), (lo, hi)
    device_error_clear()


def test_constant_values_and_keys():
    """Groups of one value have scale 0: the minimum alone carries them."""
    d, L = 64, 90
    pool = Pool([L], 2, d, 32, 16, seed=140)
    v = np.zeros((L, 2, d))
    v[:, 0, :32], v[:, 0, 32:], v[:, 1] = 3.0, -0.5, 1e4
    k = np.full((L, 2, d), 0.25)
    pool.fill([k], [v])
    rng = np.random.default_rng(141)
    q = [bf16_rows(rng, 1, 4, d)]
    O, lse = run(pool, q, True, False)
    want = np.repeat(v[0][None], 1, 0)
    o = O.double().cpu().numpy()
    # equal scores: P is 1 / L up to the sums' roundings, L * 2^-24 relative
    assert (np.abs(o[0, :2] - want[0, 0]) <= (2.0 ** -8 + L * 2.0 ** -23) * np.abs(want[0, 0])).all()
    assert (np.abs(o[0, 2:] - want[0, 1]) <= (2.0 ** -8 + L * 2.0 ** -23) * np.abs(want[0, 1])).all()


def test_nan_at_keys_that_a_query_does_not_see():
    d, L, Nq = 128, 200, 4
    pool, q = make([L], Nq, 8, 2, d, 64, 16, seed=150)
    rng = np.random.default_rng(151)
    bad = bf16_rows(rng, 2, 2, d)
    bad[:, 0, 5] = np.nan
    bad[:, 1, 70] = np.inf
    kv4.write(pool.bytes, pool.table[0], np.array([L - 2, L - 1]), bad, bad, 16, 64)
    O, lse = run(pool, q, True, False)
    o = O.double().cpu().numpy()
    assert np.isfinite(o[:2]).all() and np.isfinite(lse[:, :2].cpu().numpy()).all()
    clean, _ = make([L], Nq, 8, 2, d, 64, 16, seed=150)
    # queries 0 and 1 see keys up to L - 3: as if the last two were not there
    O1, l1 = run(clean, q, True, False)
    assert torch.equal(O[:2], O1[:2]) and torch.equal(lse[:, :2], l1[:, :2])
    assert np.isnan(o[2:]).all() and torch.isnan(lse[:, 2:]).all()


def test_nan_values_stay_in_their_group():
    """A NaN in V reaches its own group of the head dimension alone; lse not at all."""
    d, L = 128, 60
    pool, q = make([L], 1, 4, 1, d, 32, 16, seed=155)
    rng = np.random.default_rng(156)
    k, v = bf16_rows(rng, 1, 1, d), bf16_rows(rng, 1, 1, d)
    v[0, 0, 40] = np.nan
    kv4.write(pool.bytes, pool.table[0], np.array([30]), k, v, 16, 32)
    O, lse = run(pool, q, True, False)
    o = O.cpu().float().numpy()
    assert np.isnan(o[..., 32:64]).all()
    assert np.isfinite(o[..., :32]).all() and np.isfinite(o[..., 64:]).all()
    assert np.isfinite(lse.cpu().numpy()).all()


def test_zero_and_huge_queries():
    d = 64
    pool, q = make([77], 1, 3, 1, d, 64, 16, seed=160)
    q[0][0, 0] = 0.0                                # uniform weights
    q[0][0, 1] *= 2.0 ** 60                         # one key takes all
    q[0][0, 2] *= 2.0 ** -120
    O, lse = run(pool, q, True, False)
    K, V = pool.rows(0)
    Or, lr = kv4.attention(q[0], K, V, 1 / 8, True)
    o, l = O.double().cpu().numpy(), lse.double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(Or) + 2.0 ** -7        # s < 0.5: 2 u16 15 s, the head's bound
    assert (np.abs(o - Or) <= tol).all()
    assert np.abs(l[[0, 2]] - lr[[0, 2]]).max() < 2.0 ** -17
    assert abs(l[1, 0] / lr[1, 0] - 1) < 2.0 ** -19


def test_fused_query_rows_and_given_buffers():
    pool, q = make([100, 40], 3, 4, 2, 128, 64, 32, seed=170)
    O, lse = run(pool, q, True, False)
    fused = torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, :, :4] = gpu_bf16(np.stack(q))
    fused[:, :, 4:] = float("nan")
    cache, table, sl = torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table), gpu_i32([100, 40])
    out = torch.empty(2, 3, 4, 128, dtype=torch.bfloat16, device="cuda")
    l = torch.empty(2, 4, 3, device="cuda")
    o2, l2 = fa.attention_kv4(fused[:, :, :4], cache, table, sl, out=out, lse=l, max_seqlen=100)
    assert o2 is out and l2 is l
    assert torch.equal(out.reshape(-1, 4, 128), O)
    assert torch.equal(l.transpose(0, 1).reshape(4, -1), lse)
    # a workspace full of anything
    pool, q = make([3000, 40], 3, 4, 2, 128, 64, 32, seed=171)
    O, lse = run(pool, q, True, False)
    check(pool, q, O, lse, 1 / math.sqrt(128), True)
    ws = torch.full((fa.fa_attention_kv4_workspace_bytes(2, 3, 6, 3000, 4, 2, 128),), 0xff,
                    dtype=torch.uint8, device="cuda")
    o2, l2 = fa.attention_kv4(gpu_bf16(np.stack(q)), torch.from_numpy(pool.bytes).cuda(),
                              gpu_i32(pool.table), gpu_i32([3000, 40]), workspace=ws,
                              max_seqlen=3000)
    assert torch.equal(o2.reshape(O.shape), O)


def test_rows_behind_the_last_sequence_stay():
    pool, q = make([50, 20], [3, 2], 4, 2, 64, 64, 16, seed=180)
    x = np.concatenate(q + [np.ones((4, 4, 64))])
    out = torch.full((9, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((4, 9), 9.0, device="cuda")
    fa.attention_kv4(gpu_bf16(x), torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table),
                     gpu_i32([50, 20]), cu_seqlens=gpu_i32([0, 3, 5]), max_q=3, out=out, lse=l)
    check(pool, q, out[:5], l[:, :5], 1 / 8, True)
    assert (out[5:] == 9).all() and (l[:, 5:] == 9).all()


def test_bad_lengths_and_pages():
    pool, q = make([50, 60, 70], 1, 4, 2, 64, 64, 16, seed=190)
    # lengths above the bound, and below 0: those sequences are left out
    out = torch.full((3, 1, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    cache, table = torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table)
    for bad in (61, -1):
        out.fill_(9.0)
        o, l = fa.attention_kv4(gpu_bf16(np.stack(q)), cache, table, gpu_i32([50, 60, bad]), out=out,
                                max_seqlen=60)
        assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_SEQLENS
        sub = Pool.__new__(Pool)
        sub.__dict__.update(pool.__dict__, lengths=[50, 60])
        check(sub, q[:2], o.reshape(3, 4, 64)[:2], l.transpose(0, 1).reshape(4, -1)[:, :2], 1 / 8, True)
        assert (o[2] == 9).all()
    # a page outside the cache: its tokens are left out, the others stay right
    t2 = pool.table.copy()
    t2[1, 1], t2[2, 0] = pool.num_pages, -5
    o, l = fa.attention_kv4(gpu_bf16(np.stack(q)), cache, gpu_i32(t2), gpu_i32([50, 60, 70]))
    assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_PAGE
    assert torch.isfinite(o).all()
    sub.__dict__.update(pool.__dict__, lengths=[50])
    check(sub, q[:1], o.reshape(3, 4, 64)[:1], l.transpose(0, 1).reshape(4, -1)[:, :1], 1 / 8, True)
    # packed: more queries than max_q, a run that leaves the rows
    x = gpu_bf16(np.concatenate(q))
    for cu in ([0, 2, 3, 3], [0, 1, 2, 9]):
        fa.attention_kv4(x, cache, table, gpu_i32([50, 60, 70]), cu_seqlens=gpu_i32(cu), max_q=1)
        assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_SEQLENS


def test_cache_beyond_32_bits():
    """Pages whose bytes lie beyond 4 GiB of the cache."""
    pool, q = make([150], 1, 8, 8, 128, 64, 64, seed=200)
    per = pool.bytes[0].size
    pages = (1 << 32) // per + 20
    cache = torch.empty((pages, *pool.bytes.shape[1:]), dtype=torch.uint8, device="cuda")
    shift = pages - pool.num_pages
    cache[shift:] = torch.from_numpy(pool.bytes).cuda()
    table = np.where(pool.table >= 0, pool.table + shift, -1)
    sl = gpu_i32([150])
    o, l = fa.attention_kv4(gpu_bf16(np.stack(q)), cache, gpu_i32(table), sl)
    check(pool, q, o[0], l[0], 1 / math.sqrt(128), True)
    k, v = fa.kv4_read(cache, gpu_i32(table), sl, d=128, n=150)
    assert np.array_equal(k[0].double().cpu().numpy(), kv4.bf16(pool.rows(0)[0]))
    low = cache[:shift].clone() if shift < 64 else None
    assert low is None
    fa.kv4_append(-k, -v, cache, gpu_i32(table), sl)
    k2, _ = fa.kv4_read(cache, gpu_i32(table), sl, d=128, n=150)
    assert torch.equal(torch.sign(k2.float().mean()), torch.sign(-k.float().mean()))
    device_error_clear()


def test_decode_steps_follow_the_prompt():
    """As a program uses them together: a prompt is written, then tokens one at a
    time, each step's queries attending to what the cache holds."""
    rng = np.random.default_rng(210)
    H, Hkv, d, group, page = 8, 2, 128, 64, 16
    prompt, steps = [40, 0, 17], 9
    B = len(prompt)
    pool = Pool([n + steps for n in prompt], Hkv, d, group, page, seed=211)
    cache, table = torch.from_numpy(pool.bytes.copy()).cuda(), gpu_i32(pool.table)
    k = [bf16_rows(rng, n, Hkv, d) for n in prompt]
    v = [bf16_rows(rng, n, Hkv, d) for n in prompt]
    pool.fill(k, v)
    cu = gpu_i32(np.concatenate([[0], np.cumsum(prompt)]))
    fa.kv4_append(gpu_bf16(np.concatenate(k)), gpu_bf16(np.concatenate(v)), cache, table,
                  gpu_i32(prompt), cu_seqlens=cu, group=group)
    for t in range(steps):
        lens = [n + t + 1 for n in prompt]
        kn, vn = bf16_rows(rng, B, Hkv, d), bf16_rows(rng, B, Hkv, d)
        q = bf16_rows(rng, B, H, d)
        sl = gpu_i32(lens)
        fa.kv4_append(gpu_bf16(kn[:, None]), gpu_bf16(vn[:, None]), cache, table, sl, group=group)
        O, lse = fa.attention_kv4(gpu_bf16(q[:, None]), cache, table, sl, group=group)
        for b in range(B):
            kv4.write(pool.bytes, pool.table[b], np.array([lens[b] - 1]), kn[b:b + 1], vn[b:b + 1],
                      page, group)
        now = Pool.__new__(Pool)
        now.__dict__.update(pool.__dict__, lengths=lens)
        check(now, [q[b:b + 1] for b in range(B)], O[:, 0], lse[:, :, 0].T.contiguous(),
              1 / math.sqrt(d), True)
    device_error_clear()


def test_agrees_with_split_kv_on_what_is_read_back():
    """The cache read back as bf16 and attended to by the framework's own split-KV
    forward: the values differ by their rounding to bf16 alone."""
    lens, H, d = [500, 130], 4, 128
    pool, q = make(lens, 6, H, H, d, 64, 32, seed=220, k_off=0.0, q_std=1.0)
    cache, table, sl = torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table), gpu_i32(lens)
    cu_k, cu_q = gpu_i32([0, 500, 630]), gpu_i32([0, 6, 12])
    k, v = fa.kv4_read(cache, table, sl, total=630, d=d, cu_seqlens=cu_k)
    x = gpu_bf16(np.concatenate(q))
    O1, l1 = fa.attention_fwd_splitkv_varlen(x, k, v, cu_q, cu_k, 6, 500, causal=True)
    O2, l2 = fa.attention_kv4(x, cache, table, sl, cu_seqlens=cu_q, max_q=6)
    # K rounded to bf16 moves a score by sum |q k| 2^-8 / sqrt(d) at most and O by
    # twice that times |v|; V, P and O rounded to bf16 by 2^-8 of |v| each
    qk = max(float((np.abs(q[b]).transpose(1, 0, 2) @ np.abs(pool.rows(b)[0]).transpose(1, 2, 0)).max())
             for b in range(2)) / math.sqrt(d) * 2.0 ** -8
    vm = max(float(np.abs(pool.rows(b)[1]).max()) for b in range(2))
    assert (l1 - l2).abs().max() <= qk + 1e-3
    assert (O1.float() - O2.float()).abs().max() <= 2 * qk * vm + 2.0 ** -6 * vm


def test_same_bits_every_time_and_in_a_graph_on_a_stream():
    pool, q = make([3000, 10, 700], 1, 8, 2, 128, 64, 64, seed=230)
    O, lse = run(pool, q, True, False)
    for _ in range(3):
        O1, l1 = run(pool, q, True, False)
        assert torch.equal(O, O1) and torch.equal(lse, l1)
    cache, table, sl = torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table), gpu_i32([3000, 10, 700])
    x = gpu_bf16(np.stack(q))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, l = fa.attention_kv4(x, cache, table, sl)
    s.synchronize()
    assert torch.equal(o.reshape(O.shape), O)
    # two graphs, each with its own workspace, replayed on two streams at once
    graphs = []
    for _ in range(2):
        xx, ss = x.clone(), sl.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            og, lg = fa.attention_kv4(xx, cache, table, ss, max_seqlen=3000)
        graphs.append((g, xx, ss, og, lg))
    graphs[1][1].neg_()
    graphs[1][2].copy_(gpu_i32([2000, 0, 701 - 1]))
    torch.cuda.synchronize()
    t = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s):
            graphs[0][0].replay()
        with torch.cuda.stream(t):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][3].reshape(O.shape), O)
    # the replayed call went by the new lengths and queries
    sub = Pool.__new__(Pool)
    sub.__dict__.update(pool.__dict__, lengths=[2000, 0, 700])
    og, lg = graphs[1][3], graphs[1][4]
    check(sub, [-x for x in q], og.reshape(O.shape), lg.transpose(0, 1).reshape(8, -1), 1 / math.sqrt(128),
          True)
    device_error_clear()


def test_helper_refusals():
    cache = fa.kv4_cache(4, 2, 16, 128)
    table, sl = gpu_i32([[0, 1]]), gpu_i32([20])
    q = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    ok = dict(q=q, cache=cache, page_table=table, seqlens=sl)
    fa.attention_kv4(**ok)
    bad = [dict(q=q.float()), dict(q=q[0]), dict(q=q[:, :, :3]), dict(q=q.cpu()),
           dict(q=torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16, device="cuda")),
           dict(max_seqlen=33), dict(group=128), dict(group=48), dict(seqlens=sl.float()),
           dict(cu_seqlens=gpu_i32([0, 1])), dict(out=q.float()), dict(lse=torch.zeros(1, device="cuda")),
           dict(page_table=gpu_i32([[0], [1]]))]
    for change in bad:
        with pytest.raises((ValueError, fa.FaError)):
            fa.attention_kv4(**{**ok, **change})
    wide = torch.zeros(1, 80, dtype=torch.int32, device="cuda")
    with pytest.raises(fa.FaError):        # too small a workspace
        fa.attention_kv4(**{**ok, "page_table": wide},
                         workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    B = 1025
    with pytest.raises(fa.FaError):
        fa.attention_kv4(torch.zeros(B, 1, 4, 128, dtype=torch.bfloat16, device="cuda"), cache,
                         torch.zeros(B, 2, dtype=torch.int32, device="cuda"),
                         torch.zeros(B, dtype=torch.int32, device="cuda"))
    device_error_clear()


# ---- many query rows: the cache's values through fp16 and the tcgen05 kernel --------

def takes_many(pool, q_rows, bound):
    B, total = len(q_rows), sum(len(q) for q in q_rows)
    H, d = q_rows[0].shape[1:]
    L = fa.fa_attention_kv4_workspace_bytes(B, max(len(q) for q in q_rows), total, bound, H, pool.Hkv, d)
    return L > total * H * d * 2 + 4 * B * pool.Hkv * bound * d


MANY = [
    # lens, queries, H, Hkv, d, group, page, causal, packed
    ([700, 513, 64], [700, 600, 64], 16, 16, 64, 64, 48, True, True),
    ([900, 300], [500, 160], 32, 8, 128, 32, 64, True, True),
    ([260, 700], [700, 160], 24, 8, 128, 128, 16, True, True),   # more queries than keys
    ([260, 700], [700, 160], 24, 8, 128, 64, 128, False, True),
    ([129, 640], 640, 16, 16, 64, 32, 32, True, False),
    ([0, 1, 1300], [300, 300, 700], 16, 16, 128, 64, 16, True, True),
    ([4500, 130, 2300], [700, 200, 400], 16, 16, 64, 64, 64, True, True),   # several ranges of keys
    ([2200, 2049], [2500, 100], 8, 8, 128, 128, 128, True, True),           # and rows that see none
]


@pytest.mark.parametrize("case", MANY, ids=[str(i) for i in range(len(MANY))])
def test_many_rows_against_the_oracle(case):
    lens, Nq, H, Hkv, d, group, page, causal, packed = case
    pool, q = make(lens, Nq, H, Hkv, d, group, page, seed=300)
    assert takes_many(pool, q, pool.table.shape[1] * page)
    O, lse = run(pool, q, causal, packed)
    check(pool, q, O, lse, 1 / math.sqrt(d), causal, many=True)
    O1, l1 = run(pool, q, causal, packed)
    assert torch.equal(O, O1) and torch.equal(lse, l1)
    device_error_clear()


@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_many_rows_other_scales(scale):
    pool, q = make([400, 200], [400, 240], 32, 8, 64, 64, 32, seed=310)
    O, lse = run(pool, q, True, True, scale=scale)
    check(pool, q, O, lse, scale, True, many=True)
    small, q1 = make([90], 2, 4, 2, 64, 64, 32, seed=311)         # and the few rows' form
    O, lse = run(small, q1, True, False, scale=scale)
    check(small, q1, O, lse, scale, True)
    device_error_clear()


def test_many_rows_scales_of_the_inputs():
    """Rows of Q, and tiles of K and V, of magnitudes far from 1 and from one another."""
    d, L, n = 128, 400, 160
    rng = np.random.default_rng(320)
    pool = Pool([L], 16, d, 64, 16, seed=321)
    k, v = bf16_rows(rng, L, 16, d), bf16_rows(rng, L, 16, d)
    k[:128] *= 2.0 ** -30
    k[128:256] *= 2.0 ** 20
    v[:128] *= 2.0 ** 40
    v[256:] *= 2.0 ** -20
    q = bf16_rows(rng, n * 9, 16, d)
    q[::3] *= 2.0 ** -25
    q[1::3] *= 2.0 ** -40
    q[2::3] *= 2.0 ** -60
    pool.fill([k], [v])
    O, lse = run(pool, [q], False, True, scale=0.1)
    assert takes_many(pool, [q], pool.table.shape[1] * 16)
    check(pool, [q], O, lse, 0.1, False, many=True)


def test_many_rows_nan_behind_the_mask():
    d, L, n = 64, 300, 160
    pool, q = make([L, 200], [n * 6, n * 4], 8, 8, d, 64, 16, seed=330)
    q = [x[:, :8] for x in q]
    clean, _ = make([L, 200], [n * 6, n * 4], 8, 8, d, 64, 16, seed=330)
    rng = np.random.default_rng(331)
    bad = bf16_rows(rng, 2, 8, d)
    bad[:, :, 5] = np.nan
    kv4.write(pool.bytes, pool.table[0], np.array([L - 2, L - 1]), bf16_rows(rng, 2, 8, d), bad, 16, 64)
    x = [np.repeat(a, 2, 1) for a in q]                             # 16 heads on 8
    assert takes_many(pool, x, pool.table.shape[1] * 16)
    O, lse = run(pool, x, True, True)
    O1, l1 = run(clean, x, True, True)
    n0 = len(x[0])
    # sequence 0's queries but the last two, and all of sequence 1, do not see them
    keep = torch.ones(O.shape[0], dtype=torch.bool)
    keep[n0 - 2:n0] = False
    assert torch.equal(O[keep], O1[keep]) and torch.equal(lse[:, keep], l1[:, keep])
    assert torch.isnan(O[n0 - 2:n0]).all()
    device_error_clear()


def test_many_rows_bad_lengths_and_pages_and_the_rest_stays():
    pool, q = make([300, 200, 256], [300, 200, 256], 32, 8, 64, 64, 16, seed=340)
    x = np.concatenate(q + [np.ones((5, 32, 64))])
    cache, table = torch.from_numpy(pool.bytes).cuda(), pool.table.copy()
    cu = [0, 300, 500, 756]
    out = torch.full((761, 32, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((32, 761), 9.0, device="cuda")

    def call(lens, tab, cu=cu):
        out.fill_(9.0)
        lse.fill_(9.0)
        fa.attention_kv4(gpu_bf16(x), cache, gpu_i32(tab), gpu_i32(lens), cu_seqlens=gpu_i32(cu),
                         max_q=300, max_seqlen=300, out=out, lse=lse)
        return fa.fa_get_device_error()

    def first(n):
        sub = Pool.__new__(Pool)
        sub.__dict__.update(pool.__dict__, lengths=pool.lengths[:n])
        m = cu[n]
        check(sub, q[:n], out[:m], lse[:, :m], 1 / 8, True, many=True)

    assert call([300, 200, 256], table) == 0
    first(3)
    assert (out[756:] == 9).all() and (lse[:, 756:] == 9).all()
    for bad in (301, -1):
        assert call([300, 200, bad], table) == fa.FA_DEVERR_BAD_SEQLENS
        first(2)
        assert (out[500:] == 9).all() and (lse[:, 500:] == 9).all()
    table[2, 3] = pool.num_pages
    assert call([300, 200, 256], table) == fa.FA_DEVERR_BAD_PAGE
    first(2)
    assert torch.isfinite(out[500:756]).all()
    assert call([300, 200, 256], pool.table, [0, 301, 500, 756]) == fa.FA_DEVERR_BAD_SEQLENS


def test_many_rows_in_a_graph_on_a_stream():
    pool, q = make([300, 640], [300, 1000], 16, 16, 64, 64, 16, seed=350)
    assert takes_many(pool, q, 640)
    O, lse = run(pool, q, True, True)
    cache, table, sl = torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table), gpu_i32([300, 640])
    x, cu = gpu_bf16(np.concatenate(q)), gpu_i32([0, 300, 1300])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fa.attention_kv4(x, cache, table, sl, cu_seqlens=cu, max_q=1000)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        og, lg = fa.attention_kv4(x, cache, table, sl, cu_seqlens=cu, max_q=1000)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(og, O) and torch.equal(lg, lse)
    x.neg_()
    sl.copy_(gpu_i32([123, 640]))
    g.replay()
    torch.cuda.synchronize()
    sub = Pool.__new__(Pool)
    sub.__dict__.update(pool.__dict__, lengths=[123, 640])
    check(sub, [-y for y in q], og, lg, 1 / 8, True, many=True)
    device_error_clear()


FORMS = [  # the few rows' form and the many rows', keys in several ranges
    ([5000, 40], 2, 8, 2, 128, 64, 32),
    ([4500, 130, 2300], [700, 200, 400], 16, 16, 64, 64, 64),
]


@pytest.mark.parametrize("form", FORMS, ids=["few", "many"])
def test_nan_query_rows_stay_alone(form):
    lens, Nq, H, Hkv, d, group, page = form
    pool, q = make(lens, Nq, H, Hkv, d, group, page, seed=360)
    O, lse = run(pool, q, True, True)
    q[0][1, 3, 7] = np.nan
    q[0][-1, 0] = np.inf
    O1, l1 = run(pool, q, True, True)
    for i, h in ((1, 3), (len(q[0]) - 1, 0)):
        assert torch.isnan(O1[i, h]).all() and torch.isnan(l1[h, i])
        O1[i, h], l1[h, i] = O[i, h], lse[h, i]
    assert torch.equal(O, O1) and torch.equal(lse, l1)
    device_error_clear()


@pytest.mark.parametrize("form", FORMS, ids=["few", "many"])
def test_sequences_that_share_pages(form):
    _, Nq, H, Hkv, d, group, page = form
    nq = Nq if np.isscalar(Nq) else Nq[:2]
    pool, q = make([2310, 2300], nq, H, Hkv, d, group, page, seed=370)
    pool.table[1] = pool.table[0]
    O, lse = run(pool, q, True, True)
    check(pool, q, O, lse, 1 / math.sqrt(d), True, many=not np.isscalar(Nq))
    device_error_clear()


def test_calls_at_once_on_two_streams():
    sets = []
    for i, (lens, Nq, H, Hkv, d, group, page) in enumerate(FORMS):
        pool, q = make(lens, Nq, H, Hkv, d, group, page, seed=380 + i)
        n = [len(x) for x in q]
        sets.append(dict(q=gpu_bf16(np.concatenate(q)), cache=torch.from_numpy(pool.bytes).cuda(),
                         page_table=gpu_i32(pool.table), seqlens=gpu_i32(lens), group=group,
                         cu_seqlens=gpu_i32(np.concatenate([[0], np.cumsum(n)])), max_q=max(n)))
    want = [fa.attention_kv4(**s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i % 2, fa.attention_kv4(**sets[i % 2])))
    torch.cuda.synchronize()
    for i, (O, lse) in got:
        assert torch.equal(O, want[i][0]) and torch.equal(lse, want[i][1])
    device_error_clear()


def test_no_keys_and_no_pages():
    cache = fa.kv4_cache(0, 2, 16, 64)
    q = torch.ones(3, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    O, lse = fa.attention_kv4(q, cache, torch.empty(3, 0, dtype=torch.int32, device="cuda"),
                              gpu_i32([0, 0, 0]))
    assert (O == 0).all() and torch.isneginf(lse).all()
    k = torch.empty(3, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    fa.kv4_append(k, k, cache, torch.empty(3, 0, dtype=torch.int32, device="cuda"), gpu_i32([0, 0, 0]))
    device_error_clear()


def test_many_rows_factors_that_overflow_together():
    """Q's and K's largest values in different places: their factors' product is not finite."""
    pool, q = make([400, 200], [400, 240], 32, 8, 128, 64, 32, seed=390)
    rng = np.random.default_rng(391)
    k, v = bf16_rows(rng, 400, 8, 128), bf16_rows(rng, 400, 8, 128)
    k[..., 64:] = 0
    k[..., 100] = 2.0 ** 70
    q[0][7, :, 1] = 2.0 ** 100
    q[0][7, :, 64:] = 0
    pool.fill([k], [v])
    assert takes_many(pool, q, pool.table.shape[1] * 32)
    O, lse = run(pool, q, False, True)
    assert torch.isfinite(O).all() and torch.isfinite(lse).all()
    device_error_clear()


@pytest.mark.parametrize("form", FORMS, ids=["few", "many"])
def test_inputs_written_by_the_kernels_just_before(form):
    """Kernels start while those before them end: queries, new rows, lengths and the table's
    pages come from the launches directly ahead, again and again in the same places."""
    lens, Nq, H, Hkv, d, group, page = form
    pool, q = make(lens, Nq, H, Hkv, d, group, page, seed=400)
    cache, table = torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table)
    n = [len(x) for x in q]
    cu, x = gpu_i32(np.concatenate([[0], np.cumsum(n)])), gpu_bf16(np.concatenate(q))
    steps = 12
    g = torch.Generator(device="cuda").manual_seed(7)
    new = [torch.randn(2, len(lens), 1, Hkv, d, device="cuda", generator=g).bfloat16()
           for _ in range(steps)]
    length = [gpu_i32([L - i for L in lens]) for i in range(steps)]
    place, sl = torch.empty_like(x), torch.empty_like(length[0])
    rows = torch.empty_like(new[0])

    def step(i, wait):
        for a, b in ((sl, length[i]), (rows, new[i]), (place, x * (1 + i % 3))):
            a.copy_(b)
            wait()
        fa.kv4_append(rows[0], rows[1], cache, table, sl, group=group)
        wait()
        out = fa.attention_kv4(place, cache, table, sl, cu_seqlens=cu, max_q=max(n),
                               max_seqlen=max(lens), group=group)
        wait()
        return out

    fresh = cache.clone()
    want = [step(i, torch.cuda.synchronize) for i in range(steps)]
    cache.copy_(fresh)                     # the steps write into it
    got = [step(i, lambda: None) for i in range(steps)]
    torch.cuda.synchronize()
    for (O, lse), (O1, l1) in zip(want, got):
        assert torch.equal(O, O1) and torch.equal(lse, l1)
    device_error_clear()


@pytest.mark.parametrize("form", FORMS, ids=["few", "many"])
def test_captured_behind_several_streams(form):
    """In a graph: behind kernels of two streams, a copy, a fill, and at its very start."""
    lens, Nq, H, Hkv, d, group, page = form
    pool, q = make(lens, Nq, H, Hkv, d, group, page, seed=410)
    O, lse = run(pool, q, True, True)
    cache, table = torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table)
    n = [len(x) for x in q]
    cu, x, sl = gpu_i32(np.concatenate([[0], np.cumsum(n)])), gpu_bf16(np.concatenate(q)), gpu_i32(lens)
    place, lengths, junk = torch.zeros_like(x), torch.zeros_like(sl), torch.empty(1000, device="cuda")
    kw = dict(cu_seqlens=cu, max_q=max(n), group=group)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        first = fa.attention_kv4(x, cache, table, sl, **kw)          # the graph's first nodes
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.mul(x, 1, out=place)                               # a kernel
            junk.zero_()
        lengths.copy_(sl)                                            # a copy
        main.wait_stream(side)
        second = fa.attention_kv4(place, cache, table, lengths, **kw)
        lengths.zero_()                                              # a fill
        third = fa.attention_kv4(place, cache, table, lengths, **kw)
    for _ in range(3):
        place.zero_()
        g.replay()
    torch.cuda.synchronize()
    for o, l in (first, second):
        assert torch.equal(o, O) and torch.equal(l, lse)
    assert (third[0] == 0).all() and torch.isneginf(third[1]).all()
    device_error_clear()


@pytest.mark.parametrize("lens", [[600, 1000, 33], [9000, 40]], ids=["whole", "ranges"])
def test_steps_straight_after_one_another(lens):
    """Writing into the pages that the attention launched just before still reads."""
    steps, B, Hkv, d = 24, len(lens), 4, 128
    pool, q = make(lens, 1, 16, Hkv, d, 64, 16, seed=420)
    cache, table = torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table)
    x, sl = gpu_bf16(np.stack(q)), gpu_i32(lens)
    g = torch.Generator(device="cuda").manual_seed(8)
    new = [torch.randn(2, B, 30, Hkv, d, device="cuda", generator=g).bfloat16()
           for _ in range(steps)]

    def run_all(wait):
        out = []
        for k, v in new:                   # the last 30 tokens again and again
            fa.kv4_append(k, v, cache, table, sl)
            wait()
            out.append(fa.attention_kv4(x, cache, table, sl, max_seqlen=max(lens)))
            wait()
        torch.cuda.synchronize()
        return out

    for (O, lse), (O1, l1) in zip(run_all(torch.cuda.synchronize), run_all(lambda: None)):
        assert torch.equal(O, O1) and torch.equal(lse, l1)
    device_error_clear()


@pytest.mark.parametrize("d,group,page", [(64, 64, 16), (128, 64, 32)])
def test_many_sequences_in_ranges_time_after_time(d, group, page):
    """The layout of 1024 sequences and the first copies of the keys are apart in shared
    memory, whichever comes first."""
    rng = np.random.default_rng(430)
    lens = [int(x) for x in rng.integers(0, 60, 1024)]
    lens[0], lens[500], lens[1023] = 1500, 1100, 2000
    pool, q = make(lens, 1, 2, 1, d, group, page, seed=431)
    args = (gpu_bf16(np.stack(q)), torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table),
            gpu_i32(lens))
    O, lse = fa.attention_kv4(*args, group=group, max_seqlen=2000)
    check(pool, q, O.reshape(-1, 2, d), lse.transpose(0, 1).reshape(2, -1), 1 / math.sqrt(d), True)
    for _ in range(50):
        O1, l1 = fa.attention_kv4(*args, group=group, max_seqlen=2000)
        assert torch.equal(O, O1) and torch.equal(lse, l1)
    device_error_clear()


def group_params(pool, b):
    """(scale, |min|) of V, float64 [L, Hkv, d / group], from the values held (a group's
    largest code is 15, its least 0)."""
    V = pool.rows(b)[1]
    g = V.reshape(*V.shape[:2], -1, pool.group)
    return (g.max(-1) - g.min(-1)) / 15, np.abs(g.min(-1))


@pytest.mark.parametrize("H,Nq", [(4, 1), (8, 1), (4, 4)], ids=["4 rows", "8 rows", "16 rows"])
@pytest.mark.parametrize("d,group", [(128, 64), (128, 32), (64, 32)])
@pytest.mark.parametrize("k", [8, 12, 16, 20, 40])
def test_groups_of_far_apart_scales(H, Nq, d, group, k):
    """A group of V keeps its accuracy beside groups of scales 2^k times its own, in every
    key, or in every other one.

    Few rows: P s goes to fp16 after a power of two of its (row, group), so 2^-11 of
    each key's P 15 s, and a fixed step of 2^-25 where the largest P s of the group is
    2^7 at least: 2^-32 of it a key, 2^-20 for 4000 keys.  Errors of S (eS) act twice,
    on the weights and their sum, and on codes and minimum alike; the fp32 sums of at
    most 2^8 terms a lane add 2^-16 of the sum of the magnitudes.  The bound goes by the
    row's and the group's own P, s and m:
        2 u16 sum_j P 15 s + (4 eS + 2^-16) sum_j P (15 s + |m|) + ub |ref|.
    """
    L = 4000
    rng = np.random.default_rng(440 + k)
    pool = Pool([L], 1, d, group, 64, seed=441)
    v = bf16_rows(rng, L, 1, d)
    v[:, :, :group] *= 2.0 ** -k
    v[::2, :, -group:] *= 2.0 ** -k                # the last group's in every other key
    pool.fill([bf16_rows(rng, L, 1, d, std=1.3)], [v])
    q = bf16_rows(rng, Nq, H, d, std=1.3)
    scale = 1 / math.sqrt(d)
    O, lse = run(pool, [q], True, False, scale=scale)
    K, V = pool.rows(0)
    Or, lr = kv4.attention(q, K, V, scale, True)
    s, m = (np.repeat(x[:, 0], group, -1) for x in group_params(pool, 0))
    k_abs = params(pool, 0)[0]
    eS = scale * float(np.max(np.abs(q).reshape(-1, d) @ k_abs[:, 0].T)) * 2.0 ** -19
    o = O.double().cpu().numpy().reshape(Nq, H, d)
    for i in range(Nq):
        S = scale * q[i] @ K[:, 0].T
        S[:, L - Nq + i + 1:] = -np.inf
        P = np.exp(S - S.max(1, keepdims=True))
        P /= P.sum(1, keepdims=True)
        tol = 2.0 ** -10 * 15 * P @ s + (4 * eS + 2.0 ** -16) * (P @ (15 * s + m)) + \
            2.0 ** -8 * np.abs(Or[i])
        err = np.abs(o[i] - Or[i])
        assert (err <= tol).all(), (i, (err / tol).max())
    assert np.abs(lse.cpu().numpy() - lr).max() <= 2 * eS + 2.0 ** -20 + 2.0 ** -22 * np.abs(lr).max()
    device_error_clear()


@pytest.mark.parametrize("H,n", [(4, 1), (8, 800)], ids=["few", "many"])
def test_scores_of_huge_magnitude_below_zero(H, n):
    """Scores near -2^114 and -2^115 for every key: the first half of them counts alike."""
    d, L = 128, 1300
    rng = np.random.default_rng(450)
    pool = Pool([L], 4, d, 64, 16, seed=451)
    k, v = np.full((L, 4, d), -2.0 ** 55), bf16_rows(rng, L, 4, d)
    k[L // 2:] *= 2
    q = np.full((n, H, d), 2.0 ** 55)
    pool.fill([k], [v])
    assert takes_many(pool, [q], pool.table.shape[1] * 16) == (n > 1)
    O, lse = run(pool, [q], False, True, scale=0.1)
    V = pool.rows(0)[1]
    want = np.repeat(V[:L // 2].mean(0), H // 4, 0)
    o, l = O.double().cpu().numpy(), lse.double().cpu().numpy()
    if n == 1:
        # the weights are equal: the head's bounds with eS = 0
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * np.abs(V).max()
        assert (np.abs(o - want) <= tol).all()
    else:
        # With many rows the reference is the largest S log2e + f, f the exponent of the
        # tile's V, rounded to 2^-24 of 2^114: f is lost, and tiles of other exponents weigh
        # powers of two more or less (eS is of that size).  But the weights are positive, sum
        # to 1, and are 0 for the second half, 2^114 below: each value lies within the range
        # of the first half's, up to the roundings of V, P and O.
        lo, hi = (np.repeat(f(V[:L // 2], 0), H // 4, 0) for f in (np.min, np.max))
        tol = 2.0 ** -8 * np.maximum(np.abs(lo), np.abs(hi)) + 2.0 ** -10 * np.abs(V).max()
        assert (o >= lo - tol).all() and (o <= hi + tol).all()
    # -0.1 d 2^110, which log L / 2 does not show beside; a few roundings of the factors
    assert (np.abs(l / (-0.1 * d * 2.0 ** 110) - 1) <= 2.0 ** -20).all()
    device_error_clear()


@pytest.mark.parametrize("H,n", [(4, 1), (16, 1), (8, 800)], ids=["few", "16 rows", "many"])
@pytest.mark.parametrize("e", [-122, -105, 105])
def test_queries_and_keys_of_opposite_magnitudes(H, n, e):
    """Q times 2^e and K times 2^-e give the scores of Q and K: nothing of a row is lost
    to fp16's range, however small or large its values are."""
    d, L = 128, 1300
    rng = np.random.default_rng(460 + e)
    pool = Pool([L], 4, d, 64, 16, seed=461)
    pool.fill([bf16_rows(rng, L, 4, d) * 2.0 ** -e], [bf16_rows(rng, L, 4, d)])
    q = bf16_rows(rng, n, H, d) * 2.0 ** e
    q = np.where(np.abs(q) < 2.0 ** -126, 0, q)            # bf16's normal numbers
    assert takes_many(pool, [q], pool.table.shape[1] * 16) == (n > 1)
    O, lse = run(pool, [q], True, True, scale=0.1)
    check(pool, [q], O, lse, 0.1, True, many=n > 1)
    device_error_clear()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("lens,nq", [([900, 700], 3), ([900, 300], 500), ([5000], 1100)],
                         ids=["few", "many", "many, ranges"])
def test_nan_values_reach_their_columns(lens, nq, group):
    """A NaN in V reaches the columns of its group in the rows that see it, and nothing
    else, with few query rows and with many."""
    H, Hkv, d, page = 16, 8, 128, 32
    pool, q = make(lens, nq, H, Hkv, d, group, page, seed=470)
    assert takes_many(pool, q, pool.table.shape[1] * page) == (nq > 3)
    rng = np.random.default_rng(471)
    L = lens[0]
    for pos, h, i in ((L - nq // 2 - 1, 0, 5), (L - 2, 0, 100), (L - nq - 1, 2, 64), (L - 1, 3, 127),
                      (100, 4, 40)):
        k, v = bf16_rows(rng, 1, Hkv, d), bf16_rows(rng, 1, Hkv, d)
        v[0, h, i] = np.inf if i == 40 else np.nan
        kv4.write(pool.bytes, pool.table[0], np.array([pos]), k, v, page, group)
    O, lse = run(pool, q, True, True)
    assert not torch.isnan(lse).any()
    check(pool, q, O, lse, 1 / math.sqrt(d), True, many=nq > 3)
    device_error_clear()


@pytest.mark.parametrize("k", [10, 24, 28])
def test_many_rows_beside_one_huge_value(k):
    """One value of V 2^k times the others, in a tile of its own: the other tiles' keys
    still count in the other columns.

    With T_j the largest value of key j's tile, P V^ takes P T relative to the row's
    largest, as fp16: 2^-11 of each P, or a step of 2^-25 beside at least 2^7, so
    2^-32 max_i (P_i T_i) |V_j| / T_j; T is known to a factor of 2 (a power of two).  V
    is rounded likewise: 2^-11 of itself, or 2^-25 beside 2^13: 2^-38 T_j P_j.
    """
    d, L, n, H = 128, 1300, 900, 8
    rng = np.random.default_rng(480)
    pool = Pool([L], H, d, 64, 16, seed=481)
    v = bf16_rows(rng, L, H, d)
    v[700, :, 3] = 2.0 ** k
    pool.fill([bf16_rows(rng, L, H, d)], [v])
    q = bf16_rows(rng, n, H, d)
    assert takes_many(pool, [q], pool.table.shape[1] * 16)
    O, lse = run(pool, [q], False, True, scale=0.1)
    K, V = pool.rows(0)
    Or, lr = kv4.attention(q, K, V, 0.1, False)
    o = O.double().cpu().numpy()
    for h in range(H):
        S = 0.1 * q[:, h] @ K[:, h].T
        P = np.exp(S - S.max(1, keepdims=True))
        P /= P.sum(1, keepdims=True)
        eS = 0.1 * (np.abs(q[:, h]) @ np.abs(K[:, h]).T).max() * (2.0 ** -11 + 2.0 ** -15)
        A = np.abs(V[:, h])
        T = np.repeat([A[j:j + 128].max() for j in range(0, L, 128)], 128)[:L]
        step = 2 * (P * T).max(1)[:, None] * 2.0 ** -32 * (A / T[:, None]).sum(0) + \
            2.0 ** -37 * (P @ T)[:, None]
        tol = (2.0 ** -10 + 4 * eS) * (P @ A) + step + 2.0 ** -8 * np.abs(Or[:, h])
        err = np.abs(o[:, h] - Or[:, h])
        assert (err <= tol).all(), (h, (err / tol).max())
    device_error_clear()


def test_one_query_each_with_loose_bounds():
    """A packed decode step of 1024 sequences without max_q, on a table for 131072 keys."""
    rng = np.random.default_rng(490)
    B, H, Hkv, d, page = 1024, 64, 8, 64, 256
    lens = [int(x) for x in rng.integers(0, 40, B)]
    pool, q = make(lens, 1, H, Hkv, d, 64, page, seed=491, extra_cols=511)
    x = gpu_bf16(np.concatenate(q))
    args = (torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table), gpu_i32(lens))
    O, lse = fa.attention_kv4(x, *args, cu_seqlens=gpu_i32(np.arange(B + 1)), group=64)
    check(pool, q, O, lse, 1 / 8, True)
    device_error_clear()


def test_decreasing_cu_seqlens_are_told():
    """Runs that overlap because cu_seqlens falls in between: nothing is computed."""
    pool, q = make([50, 60, 70], 2, 4, 2, 64, 64, 16, seed=495)
    out = torch.full((6, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 6), 9.0, device="cuda")
    for cu in ([0, 6, 0, 6], [0, 2, 1, 4], [4, 2, 2, 2]):
        fa.attention_kv4(gpu_bf16(np.concatenate(q)), torch.from_numpy(pool.bytes).cuda(),
                         gpu_i32(pool.table), gpu_i32([50, 60, 70]), cu_seqlens=gpu_i32(cu), max_q=6,
                         out=out, lse=lse)
        assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_SEQLENS
        assert (out == 9).all() and (lse == 9).all()
    device_error_clear()
