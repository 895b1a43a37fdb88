"""Writing to and reading from the 4-bit paged cache, against the oracle.

The code of a value is defined operation by operation in float32, so the bytes
that the kernel writes are compared with the oracle's bytes exactly; a value
read back is min + scale * code rounded once to bf16, also compared exactly.
"""
import numpy as np
import pytest
import torch

from gpu_common import device_error_clear, require_gpu
from kv4_common import Pool, bf16_rows, fa, gpu_bf16, gpu_i32, kv4, same_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def dev():
    d = require_gpu()
    fa.fa_get_device_error()
    return d


def read_back(x):
    return x.double().cpu().numpy()


@pytest.mark.parametrize("d,group,Hkv,page,new,behind", [
    (128, 64, 2, 64, [1, 1, 1], [0, 63, 130]),          # a decode step, page borders
    (128, 32, 3, 16, [5, 0, 33, 1], [0, 7, 15, 16]),    # odd heads, an empty run, cells crossed
    (128, 128, 8, 128, [200, 129], [0, 55]),
    (64, 32, 1, 48, [1, 50, 16], [47, 3, 16]),
    (64, 64, 5, 32, [31, 70], [1, 0]),
])
def test_packed_write_then_read(d, group, Hkv, page, new, behind):
    rng = np.random.default_rng(10)
    lens = [a + b for a, b in zip(new, behind)]
    pool = Pool(lens, Hkv, d, group, page, seed=11)
    cache = torch.from_numpy(pool.bytes.copy()).cuda()
    k = [bf16_rows(rng, n, Hkv, d, offset=0.5) for n in new]
    v = [bf16_rows(rng, n, Hkv, d, std=2.0) for n in new]
    pool.fill(k, v, first=behind)
    cu = np.concatenate([[0], np.cumsum(new)])
    pad = 3                                               # rows behind the last sequence
    junk = np.full((pad, Hkv, d), 7.0)
    kt, vt = (gpu_bf16(np.concatenate(x + [junk])) for x in (k, v))
    table, sl, cut = gpu_i32(pool.table), gpu_i32(lens), gpu_i32(cu)
    fa.kv4_append(kt, vt, cache, table, sl, cu_seqlens=cut, max_new=max(new), group=group)
    assert same_cache(cache.cpu().numpy(), pool.bytes, d, group)
    ko, vo = torch.full_like(kt, 3.0), torch.full_like(vt, 3.0)
    fa.kv4_read(cache, table, sl, d=d, cu_seqlens=cut, max_new=max(new), group=group, k=ko, v=vo)
    for out, rows in ((ko, k), (vo, v)):
        out = read_back(out)
        want = np.concatenate([kv4.bf16(kv4.values(*kv4.quantise(x, group))) for x in rows])
        assert np.array_equal(out[:cu[-1]], want)
        assert (out[cu[-1]:] == 3.0).all()
    device_error_clear()


@pytest.mark.parametrize("N", [1, 4])
def test_dense_rows_of_a_fused_projection(N):
    B, H, Hkv, d, group, page = 5, 4, 2, 128, 64, 16
    rng = np.random.default_rng(12)
    lens = [N + 3 * b for b in range(B)]
    pool = Pool(lens, Hkv, d, group, page, seed=13)
    cache = torch.from_numpy(pool.bytes.copy()).cuda()
    fused = torch.from_numpy(rng.standard_normal((B, N, H + 2 * Hkv, d))).to(torch.bfloat16)
    x = fused.double().numpy()
    pool.fill(list(x[:, :, H:H + Hkv]), list(x[:, :, H + Hkv:]), first=[n - N for n in lens])
    f = fused.cuda()
    table, sl = gpu_i32(pool.table), gpu_i32(lens)
    fa.kv4_append(f[:, :, H:H + Hkv], f[:, :, H + Hkv:], cache, table, sl, group=group)
    assert same_cache(cache.cpu().numpy(), pool.bytes, d, group)
    ko, vo = fa.kv4_read(cache, table, sl, d=d, n=N, group=group)
    assert ko.shape == (B, N, Hkv, d)
    want = kv4.bf16(kv4.values(*kv4.quantise(x[:, :, H:H + Hkv], group)))
    assert np.array_equal(read_back(ko), want)
    # read into the fused rows: the other heads' values stay
    g = torch.zeros_like(f)
    fa.kv4_read(cache, table, sl, d=d, group=group, k=g[:, :, H:H + Hkv], v=g[:, :, H + Hkv:])
    assert torch.equal(g[:, :, H:H + Hkv], ko) and torch.equal(g[:, :, H + Hkv:], vo)
    assert (g[:, :, :H] == 0).all()
    device_error_clear()


def test_special_values():
    d, group, page = 128, 32, 16
    big = float(torch.finfo(torch.bfloat16).max)
    x = np.zeros((6, 1, d))
    x[0] = -1.5                                           # constant groups
    x[1, 0, 3], x[1, 0, 40], x[1, 0, 70] = np.nan, np.inf, -np.inf
    x[2, 0, :2], x[2, 0, 2] = (big, -big), big / 3        # range beyond float32
    x[3, 0, 0] = 2.0 ** -133                              # range below the least scale
    x[4, 0, :16] = np.arange(16)                          # scale 1: exact
    x[4, 0, 16:32] = np.arange(16) - 0.0
    x[5, 0, :32] = np.linspace(0, 15, 61)[:32]            # ties
    x = kv4.bf16(x)
    pool = Pool([6], 1, d, group, page, seed=14)
    cache = torch.from_numpy(pool.bytes.copy()).cuda()
    pool.fill([x], [-x])
    table, sl = gpu_i32(pool.table), gpu_i32([6])
    fa.kv4_append(gpu_bf16(x[None]), gpu_bf16(-x[None]), cache, table, sl, group=group)
    assert same_cache(cache.cpu().numpy(), pool.bytes, d, group)
    ko, vo = fa.kv4_read(cache, table, sl, d=d, n=6, group=group)
    for out, want in ((ko, pool.rows(0)[0]), (vo, pool.rows(0)[1])):
        assert np.array_equal(read_back(out)[0], kv4.bf16(want), equal_nan=True)
    assert np.array_equal(read_back(ko)[0, 4], x[4])
    device_error_clear()


def test_ragged_prompts_and_whole_sequences():
    """Thousands of rows, many blocks: every byte, and the whole sequences read."""
    d, group, Hkv, page = 128, 64, 4, 64
    rng = np.random.default_rng(15)
    lens = [700, 1, 0, 513]
    pool = Pool(lens, Hkv, d, group, page, seed=16)
    cache = torch.from_numpy(pool.bytes.copy()).cuda()
    k = [bf16_rows(rng, n, Hkv, d) for n in lens]
    v = [bf16_rows(rng, n, Hkv, d) for n in lens]
    pool.fill(k, v)
    cu = gpu_i32(np.concatenate([[0], np.cumsum(lens)]))
    table, sl = gpu_i32(pool.table), gpu_i32(lens)
    fa.kv4_append(gpu_bf16(np.concatenate(k)), gpu_bf16(np.concatenate(v)), cache, table, sl,
                  cu_seqlens=cu, group=group)
    assert same_cache(cache.cpu().numpy(), pool.bytes, d, group)
    ko, vo = fa.kv4_read(cache, table, sl, total=sum(lens), d=d, cu_seqlens=cu, group=group)
    want = [np.concatenate([pool.rows(b)[i] for b in range(4)]) for i in (0, 1)]
    assert np.array_equal(read_back(ko), kv4.bf16(want[0]))
    assert np.array_equal(read_back(vo), kv4.bf16(want[1]))
    device_error_clear()


def test_bad_counts_and_pages_are_left_out():
    d, group, Hkv, page = 64, 64, 2, 16
    rng = np.random.default_rng(17)
    pool = Pool([20, 20, 20, 20], Hkv, d, group, page, seed=18)
    cache = torch.from_numpy(pool.bytes.copy()).cuda()
    k = [bf16_rows(rng, 2, Hkv, d) for _ in range(4)]
    good = Pool([20, 20, 20, 20], Hkv, d, group, page, seed=18)
    table = pool.table.copy()
    table[1, 1] = pool.num_pages                          # the page of the new tokens
    table[2, 1] = -1
    for b in (0,):
        kv4.write(good.bytes, good.table[b], np.arange(18, 20), k[b], k[b], page, group)
    kt = gpu_bf16(np.stack(k))
    # sequence 3 claims fewer tokens than it gets
    fa.kv4_append(kt, kt, cache, gpu_i32(table), gpu_i32([20, 20, 20, 1]), group=group)
    assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_PAGE | fa.FA_DEVERR_BAD_SEQLENS
    assert same_cache(cache.cpu().numpy(), good.bytes, d, group)
    out = torch.full((4, 2, Hkv, d), 5.0, dtype=torch.bfloat16, device="cuda")
    fa.kv4_read(cache, gpu_i32(table), gpu_i32([20, 20, 20, 10 ** 6]), d=d, group=group, k=out,
                v=out.clone())
    assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_PAGE | fa.FA_DEVERR_BAD_SEQLENS
    want = kv4.bf16(kv4.values(*kv4.quantise(k[0], group)))
    assert np.array_equal(read_back(out[0]), want) and (out[1:] == 5.0).all()
    # a packed run longer than max_new
    fa.kv4_append(kt[:, 0], kt[:, 0], cache, gpu_i32(pool.table), gpu_i32([20] * 4),
                  cu_seqlens=gpu_i32([0, 3, 4, 4, 4]), max_new=2, group=group)
    assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_SEQLENS


def test_helper_refusals():
    cache = fa.kv4_cache(4, 2, 16, 128)
    table, sl = gpu_i32([[0]]), gpu_i32([1])
    k = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
    bad = [dict(k=k[..., :64]), dict(k=k.half()), dict(k=k[:, :, :1]), dict(group=32),
           dict(table=table.long()), dict(table=gpu_i32([[0], [0]])), dict(sl=gpu_i32([1, 1])),
           dict(table=table.cpu()), dict(cache=cache[:, :, :100]), dict(k=k.transpose(2, 3)),
           dict(cu=gpu_i32([0, 1])), dict(k=torch.zeros(1, 1, 2, 256, dtype=torch.bfloat16,
                                                        device="cuda")[..., ::2])]
    for change in bad:
        a = dict(k=k, cache=cache, table=table, sl=sl, group=64, cu=None)
        a.update(change)
        with pytest.raises((ValueError, fa.FaError)):
            fa.kv4_append(a["k"], a["k"], a["cache"], a["table"], a["sl"], cu_seqlens=a["cu"],
                          group=a["group"])
    with pytest.raises(ValueError):
        fa.kv4_read(cache, table, sl, cu_seqlens=gpu_i32([0, 1]))
    device_error_clear()


def test_on_a_stream_and_in_a_graph():
    d, group, Hkv, page = 128, 64, 2, 16
    rng = np.random.default_rng(19)
    pool = Pool([9], Hkv, d, group, page, seed=20)
    k, v = bf16_rows(rng, 9, Hkv, d), bf16_rows(rng, 9, Hkv, d)
    empty = torch.from_numpy(pool.bytes).cuda()
    cache = empty.clone()
    pool.fill([k], [v])
    kt, vt = gpu_bf16(k[None]), gpu_bf16(v[None])
    ko, vo = torch.empty_like(kt), torch.empty_like(vt)
    table, sl = gpu_i32(pool.table), gpu_i32([9])

    def step():
        fa.kv4_append(kt, vt, cache, table, sl, group=group)
        fa.kv4_read(cache, table, sl, d=d, group=group, k=ko, v=vo)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert same_cache(cache.cpu().numpy(), pool.bytes, d, group)
    first = ko.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    kt.neg_()
    cache.copy_(empty)
    g.replay()
    torch.cuda.synchronize()
    # the replayed call quantised the new rows
    want = kv4.bf16(kv4.values(*kv4.quantise(-k, group)))
    assert np.array_equal(read_back(ko)[0], want)
    assert not torch.equal(ko, first)
    device_error_clear()


@pytest.mark.parametrize("cu,lens,good", [
    ([0, 2, 4, 9], [20, 20, 20], [0, 1]),        # the last run leaves the rows
    ([-2, 2, 4, 6], [20, 20, 20], [1, 2]),       # the first begins before them
    ([0, 2, 1, 1], [20, 20, 20], [0]),           # a run of fewer than no rows
    ([0, 3, 3, 6], [20, -1, 20], [0, 2]),        # no new rows, but no length
    ([0, 3, 3, 6], [20, 33, 20], [0, 2]),        # nor one that the table holds
])
def test_bad_packed_counts_are_told_and_left_out(cu, lens, good):
    d, group, Hkv, page = 128, 64, 3, 16
    rng = np.random.default_rng(21)
    pool = Pool([20, 20, 20], Hkv, d, group, page, seed=22, extra_cols=0)
    cache = torch.from_numpy(pool.bytes.copy()).cuda()
    x = bf16_rows(rng, 6, Hkv, d)
    table, sl, cut = gpu_i32(pool.table), gpu_i32(lens), gpu_i32(cu)
    kt = gpu_bf16(x)
    for b in good:
        n = cu[b + 1] - cu[b]
        kv4.write(pool.bytes, pool.table[b], np.arange(20 - n, 20), x[cu[b]:cu[b + 1]],
                  x[cu[b]:cu[b + 1]], page, group)
    fa.kv4_append(kt, kt, cache, table, sl, cu_seqlens=cut, max_new=6, group=group)
    assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_SEQLENS
    assert same_cache(cache.cpu().numpy(), pool.bytes, d, group)
    out = torch.full_like(kt, 5.0)
    fa.kv4_read(cache, table, sl, d=d, cu_seqlens=cut, max_new=6, group=group, k=out, v=out.clone())
    assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_SEQLENS
    rows = np.zeros(6, bool)
    for b in good:
        rows[cu[b]:cu[b + 1]] = True
    want = np.where(rows[:, None, None], kv4.bf16(kv4.values(*kv4.quantise(x, group))), 5.0)
    assert np.array_equal(read_back(out), want)
