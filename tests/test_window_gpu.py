"""Attention with a sliding window and sinks, forward, against the fp64 oracle (GB300)."""
import numpy as np
import pytest
import torch

import online_softmax_06_gb300 as fa
from gpu_common import device_error_clear, require_gpu
from window_common import Batch, check_forward, f64, layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def run(n, L, H, Hkv, d, form, window, sinks, seed=0, scale=None, **kw):
    batch = Batch(n, L, H, Hkv, d, form, seed, **kw)
    o, lse = fa.attention_window_fwd(batch.gq, batch.gk, batch.gv, window, sinks, scale=scale,
                                     **batch.kw)
    device_error_clear()
    check_forward(batch, o, lse, window, sinks, scale)
    return batch, o, lse


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (2, 0), (31, 4), (64, 33), (127, 1), (128, 0),
                                          (129, 32), (300, 4), (300, 0), (200, 130), (5000, 4),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (100, 300)])
@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 128), (8, 2, 64)])
def test_dense_windows(window, sinks, H, Hkv, d):
    run([700, 700], [700, 700], H, Hkv, d, "dense", window, sinks)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 8, 16, 60, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_heads_that_share(G, d):
    run([257], [257], 2 * G, 2, d, "dense", 100, 5, seed=G)


@pytest.mark.parametrize("form", ["packed", "fused"])
@pytest.mark.parametrize("H,Hkv,d", [(3, 3, 64), (12, 4, 128), (7, 1, 128)])
def test_packed_ragged(form, H, Hkv, d):
    n = [130, 0, 1, 129, 600, 128, 3, 0]
    batch, o, lse = run(n, [n_ + e for n_, e in zip(n, (0, 70, 500, 3, 1000, 0, 129, 0))], H, Hkv, d,
                        form, 150, 4)


@pytest.mark.parametrize("window", [60, 700])
def test_many_sequences(window):
    """More sequences than a warp looks up at once, most of them short or empty."""
    rng = np.random.default_rng(9)
    n = [int(x) for x in rng.integers(0, 90, 1200)]
    n[700], n[1199] = 1500, 800
    run(n, n, 2, 1, 64, "packed", window, 3)


@pytest.mark.parametrize("n,L,window", [([200, 60], [300, 60], 64), ([200, 60], [300, 60], 290), ([3, 1, 0, 5], [300, 60, 9, 5], 64),
                                        ([100, 90], [4000, 3900], 3800)])
def test_rows_behind_the_last_sequence_stay(n, L, window):
    """One tile a CTA, two, few queries, clusters."""
    batch = Batch(n, L, 4, 2, 128, "packed", spare=90)
    o = torch.full(batch.gq.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, len(batch.gq)), 7.0, device="cuda")
    fa.attention_window_fwd(batch.gq, batch.gk, batch.gv, window, 4, out=o, lse=lse, **batch.kw)
    device_error_clear()
    assert (o[sum(n):] == 7).all() and (lse[:, sum(n):] == 7).all()
    check_forward(batch, o, lse, window, 4)


@pytest.mark.parametrize("nq", [1, 300])
def test_no_keys_at_all(nq):
    q = torch.randn(2, nq, 4, 64, device="cuda").bfloat16()
    k = torch.empty(2, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.attention_window_fwd(q, k, k, 10, 2)
    device_error_clear()
    assert (o == 0).all() and (lse == float("-inf")).all()


def test_no_queries():
    q = torch.empty(2, 0, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 9, 2, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.attention_window_fwd(q, k, k, 10, 2)
    assert o.shape == q.shape and lse.shape == (2, 4, 0)
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    o, lse = fa.attention_window_fwd(e, e, e, 10, 2, cu_seqlens_q=cu, cu_seqlens_k=cu)
    assert o.shape == e.shape and lse.shape == (4, 0)
    assert [g.shape for g in fa.attention_window_bwd(e, e, e, e, e, lse, 10, 2, cu_seqlens=cu)] == [e.shape] * 3


@pytest.mark.parametrize("nq", [1, 300])
def test_rows_far_into_a_long_cache(nq):
    """K and V rows behind 2^31 elements, and rows of K and V unlike distances apart."""
    H, Hkv, d, room, L = 4, 2, 128, 4_300_000, 4_299_990
    rng = np.random.default_rng(8)
    k = torch.empty(2, room, 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")[:, :, :Hkv]     # 2.2e9 elements a sequence
    v = torch.empty(2, room, Hkv, d, dtype=torch.bfloat16, device="cuda")
    q = torch.from_numpy(rng.standard_normal((2, nq, H, d))).bfloat16().cuda()
    seen = slice(L - nq - 200, L)
    for x in (k, v):
        x[1, seen] = torch.from_numpy(rng.standard_normal((nq + 200, Hkv, d))).bfloat16().cuda()
        x[1, :4] = torch.from_numpy(rng.standard_normal((4, Hkv, d))).bfloat16().cuda()
    o, lse = fa.attention_window_fwd(q, k, v, 200, 4, seqlens_k=torch.tensor([0, L], dtype=torch.int32, device="cuda"))
    device_error_clear()
    assert (o[0] == 0).all()
    part = Batch([nq], [nq + 204], H, Hkv, d, "dense")
    part.q = [q[1].cpu()]
    part.k, part.v = ([torch.cat((x[1, :4], x[1, seen])).cpu()] for x in (k, v))
    check_forward(part, o[1:], lse[1:], 200, 4)


@pytest.mark.parametrize("nq", [1, 2, 5, 40, 300])
@pytest.mark.parametrize("H,Hkv,d", [(16, 2, 64), (8, 8, 128), (12, 4, 128)])
def test_cache_with_room(nq, H, Hkv, d):
    """Sequences of no key, of fewer keys than queries (rows that see nothing), of many; the room
    behind the keys holds NaN."""
    run([nq] * 6, [0, 1, nq // 2, nq, 1000, 513], H, Hkv, d, "cache", 130, 4)


@pytest.mark.parametrize("nq,sinks,window", [(1, 0, 1), (1, 200, 40), (4, 31, 3000), (1, 4, 2900),
                                             (260, 4, 2900), (3, 0, 64)])
def test_cache_long(nq, sinks, window):
    run([nq] * 3, [3000, 2999, 2901], 8, 2, 128, "cache", window, sinks)


@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (6, 2, 128), (7, 1, 64), (16, 2, 128)])
@pytest.mark.parametrize("window,sinks", [(3000, 4), (2 ** 30, 0), (2500, 200)])
def test_few_items_long_windows(H, Hkv, d, window, sinks):
    """Items so few that clusters share their steps: whole and cut tiles, queries without a key."""
    run([200, 200, 200], [4000, 100, 0], H, Hkv, d, "cache", window, sinks)
    run([90, 1, 0, 257], [3900, 3001, 50, 257], H, Hkv, d, "packed", window, sinks)


@pytest.mark.parametrize("nq", [1, 200])
def test_large_scores_and_scales(nq):
    """A scale that makes single keys dominate; one that makes all keys alike."""
    for scale in (4.0, 1e-4):
        run([nq], [700], 4, 2, 64, "dense", 300, 2, scale=scale)


@pytest.mark.parametrize("nq", [1, 300])
def test_lowest_values_and_infinities(nq):
    """Keys whose scores are -inf or the type's lowest value have no weight beside others; K of any
    value at keys that a query does not see does not reach it."""
    batch = Batch([nq], [600], 4, 2, 64, "dense", seed=3)
    o0, l0 = fa.attention_window_fwd(batch.gq, batch.gk, batch.gv, 64, 2)
    k = batch.gk.clone()
    k[:, 2:600 - nq - 64 + 1] = float("nan")                    # behind every window
    o1, l1 = fa.attention_window_fwd(batch.gq, k, batch.gv, 64, 2)
    assert torch.equal(o0, o1) and torch.equal(l0, l1)
    q = torch.ones(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, 80, 2, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 60:70] = -torch.finfo(torch.bfloat16).max              # scores -inf
    o, lse = fa.attention_window_fwd(q, k, batch.gv[:, :80].contiguous(), 40, 0)
    v = f64(batch.gv[0, :80])
    want = v[np.r_[40:60, 70:80]].mean(0).repeat(2, 0)
    spread = np.abs(v[np.r_[40:60, 70:80]]).mean(0).repeat(2, 0)
    assert np.all(np.abs(f64(o[0, 0]) - want) <= 2.0 ** -8 * spread + 2.0 ** -7 * np.abs(want))
    assert np.abs(f64(lse) - np.log(30)).max() <= 2.0 ** -18


@pytest.mark.parametrize("nq", [1, 300])
def test_nan_stays_in_its_rows(nq):
    """A NaN of Q makes its own row NaN, one of K the rows that see the key."""
    batch = Batch([nq], [500], 4, 2, 128, "dense", seed=4)
    q, k = batch.gq.clone(), batch.gk.clone()
    q[0, nq - 1, 1, 5] = float("nan")
    k[0, 499, 1, 7] = float("nan")                              # seen by the last query alone
    o, lse = fa.attention_window_fwd(q, k, batch.gv, 90, 3)
    bad = torch.isnan(lse[0])
    want = torch.zeros_like(bad)
    want[1, nq - 1] = want[2:, nq - 1] = True
    assert torch.equal(bad, want)
    assert torch.equal(torch.isnan(o[0]).all(-1), want.t()) and torch.equal(torch.isnan(o[0]).any(-1), want.t())


def test_a_wide_window_is_causal_attention():
    """With window >= keys and one kv head a query head: fa_attention_fwd's masking."""
    batch = Batch([900, 900], [900, 900], 4, 4, 128, "dense", seed=6)
    o, lse = fa.attention_window_fwd(batch.gq, batch.gk, batch.gv, 900, 0)
    ro, rl = fa.attention_fwd(batch.gq, batch.gk, batch.gv, causal=True)
    assert (lse - rl).abs().max() <= 2.0 ** -18 * (1 + rl.abs().max())
    assert ((o.float() - ro.float()).abs() <= 2.0 ** -6 * (1 + ro.float().abs())).all()


def test_bad_counts_are_flagged_and_left_out():
    for what in ("long_q", "long_k", "negative", "decreasing", "beyond"):
        batch = Batch([60, 50], [100, 200], 4, 2, 64, "packed")
        o = torch.full(batch.gq.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, len(batch.gq)), 7.0, device="cuda")
        kw = dict(batch.kw)
        if what == "long_q":
            kw["max_q"] = 59
        elif what == "long_k":
            kw["max_k"] = 199
        elif what == "negative":
            kw["seqlens_k"] = torch.tensor([100, -1], dtype=torch.int32, device="cuda")
        elif what == "decreasing":
            kw["cu_seqlens_q"] = torch.tensor([0, 60, 50], dtype=torch.int32, device="cuda")
        else:
            kw["cu_seqlens_k"] = torch.tensor([0, 100, 10 ** 6], dtype=torch.int32, device="cuda")
        fa.attention_window_fwd(batch.gq, batch.gk, batch.gv, 64, 4, out=o, lse=lse, **kw)
        assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_SEQLENS
        bad = slice(0, 60) if what == "long_q" else slice(60, 110)
        assert (o[bad] == 7).all() and (lse[:, bad] == 7).all()
        good = slice(60, 110) if what == "long_q" else slice(0, 60)
        assert not (o[good] == 7).all(-1).any()


@pytest.mark.parametrize("nq", [1, 300])
def test_replayed_graph_and_other_stream(nq):
    batch = Batch([nq] * 2, [700, 650], 8, 2, 128, "cache", seed=7)
    call = lambda: fa.attention_window_fwd(batch.gq, batch.gk, batch.gv, 300, 4, **batch.kw)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    batch.gq.copy_(torch.randn(batch.gq.shape))
    batch.kw["seqlens_k"].copy_(torch.tensor([300, 700], dtype=torch.int32))
    batch.gk.nan_to_num_(0)
    batch.gv.nan_to_num_(0)
    for _ in range(2):
        g.replay()
    want = call()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert not torch.equal(out[0], side[0])
    device_error_clear()


@pytest.mark.parametrize("n,L,window", [(300, 300, 100), (300, 300, 280), (200, 4000, 3900)])
def test_timed_out_wait(n, L, window):
    """A wait that runs out (one tile a CTA, two, a cluster's) leaves the rows unwritten, flags it, and
    the next call is right."""
    batch = Batch([n], [L], 4, 2, 128, "dense")
    o = torch.full(batch.gq.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, 4, n), 7.0, device="cuda")
    fa.fa_debug_expire_next_wait(1_000_000)
    fa.attention_window_fwd(batch.gq, batch.gk, batch.gv, window, 4, out=o, lse=lse)
    assert fa.fa_get_device_error() == fa.FA_DEVERR_WAIT_TIMEOUT
    assert (o == 7).all() and (lse == 7).all()
    o, lse = fa.attention_window_fwd(batch.gq, batch.gk, batch.gv, window, 4)
    device_error_clear()
    check_forward(batch, o, lse, window, 4)


def test_tensor_refusals():
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 9, 2, 64, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for bad in (dict(q=q.float()), dict(k=k[:1], v=k[:1]), dict(v=k[:, :8]), dict(k=k[:, :, :1].repeat(1, 1, 3, 1)),
                dict(seqlens_k=i32(1)), dict(seqlens_k=i32(1, 1).long()), dict(cu_seqlens_q=i32(0, 3, 6)),
                dict(q=q.cpu()), dict(q=q.transpose(1, 2)), dict(k=k[..., :32], v=k[..., :32]),
                dict(lse=torch.zeros(2, 4, 4, device="cuda")), dict(out=q[:, :, ::2])):
        args = dict(q=q, k=k, v=k, window=4)
        args.update(bad)
        with pytest.raises(ValueError):
            fa.attention_window_fwd(**args)
    for bad in (dict(window=0), dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan"))):
        with pytest.raises(fa.FaError):
            fa.attention_window_fwd(**{**dict(q=q, k=k, v=k, window=4), **bad})
