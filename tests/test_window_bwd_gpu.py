"""Gradients of the window attention against the fp64 oracle (GB300)."""
import numpy as np
import pytest
import torch

import online_softmax_06_gb300 as fa
from gpu_common import device_error_clear, require_gpu
from window_common import Batch, bf16, check_gradients, f64, layer, score_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def upstream(batch, seed=100):
    """dO on the device, laid out as O, NaN behind the last sequence; and of each sequence."""
    rng = np.random.default_rng(seed)
    do = [bf16(rng.standard_normal(x.shape)) for x in batch.q]
    if batch.form == "dense":
        return torch.stack(do).cuda(), [f64(x) for x in do]
    spare = len(batch.gq) - sum(batch.n)
    rest = torch.full((spare, batch.H, batch.d), float("nan"), dtype=torch.bfloat16)
    return torch.cat(do + [rest]).cuda(), [f64(x) for x in do]


def run(n, H, Hkv, d, form, window, sinks, seed=0, scale=None, **kw):
    batch = Batch(n, n, H, Hkv, d, form, seed, **kw)
    o, lse = fa.attention_window_fwd(batch.gq, batch.gk, batch.gv, window, sinks, scale=scale, **batch.kw)
    do, parts = upstream(batch, seed + 100)
    how = {} if form == "dense" else dict(cu_seqlens=batch.kw["cu_seqlens_q"], max_seqlen=batch.kw["max_q"])
    grads = fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, window, sinks, scale=scale, **how)
    device_error_clear()
    check_gradients(batch, parts, grads, window, sinks, scale)
    return batch, o, lse, do, how, grads


@pytest.mark.parametrize("window,sinks", [(1, 3), (2, 0), (31, 4), (64, 33), (127, 1), (128, 0), (129, 32), (300, 4),
                                          (200, 130), (5000, 4), (2 ** 31 - 1, 0), (100, 300), (50, 10 ** 6)])
@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 128), (8, 2, 64)])
def test_dense_windows(window, sinks, H, Hkv, d):
    run([700, 700], H, Hkv, d, "dense", window, sinks)


@pytest.mark.parametrize("G", [1, 3, 6, 7, 16, 60, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_heads_that_share(G, d):
    run([257], 2 * G, 2, d, "dense", 100, 5, seed=G)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 129])
def test_short(n):
    run([n] * 3, 4, 2, 64, "dense", 40, 2)


@pytest.mark.parametrize("n", [1, 2, 4, 7, 16, 17, 90])
@pytest.mark.parametrize("H,Hkv,d", [(4, 4, 64), (6, 2, 128)])
def test_few_keys_without_the_rounding_of_o(n, H, Hkv, d):
    """Queries whose keys fit one step: dQ is off by dS's rounding to bf16 (2^-9 of each), the correction by
    the sum of those roundings times a mean of keys, and its own rounding; D has no part of O's rounding."""
    batch, o, lse, do, how, grads = run([n] * 3, H, Hkv, d, "dense", 40, 3)
    scale, parts = d ** -0.5, [f64(x) for x in do]
    for b in range(3):
        q, k, v, g, got = f64(batch.q[b]), f64(batch.k[b]), f64(batch.v[b]), parts[b], f64(grads[0][b])
        want = layer.window_attention_bwd(q, k, v, g, 40, 3, scale)[0]
        O, stat = layer.window_attention(q, k, v, 40, 3, scale)
        slop = 4 * score_error(q, k, scale, d).max() + 2.0 ** -18
        for h in range(H):
            kh, vh = k[:, h // (H // Hkv)], v[:, h // (H // Hkv)]
            s = np.where(layer.window_seen(n, n, 40, 3), q[:, h] @ kh.T * scale - stat[h][:, None], -np.inf)
            P, dP, D = np.exp(s), g[:, h] @ vh.T, (g[:, h] * O[:, h]).sum(1, keepdims=True)
            dS = np.abs(P * (dP - D))
            top = np.abs(kh).max(0)
            tol = scale * 2.0 ** -9 * (dS @ (np.abs(kh) + top)) + 2.0 ** -8 * np.abs(want[:, h])
            tol += scale * slop * ((P * (np.abs(dP) + np.abs(dP).max(1, keepdims=True) + np.abs(D))) @ (np.abs(kh) + top))
            assert np.all(np.abs(got[:, h] - want[:, h]) <= tol), (np.abs(got[:, h] - want[:, h]) / tol).max()


@pytest.mark.parametrize("H,Hkv,d", [(1, 1, 64), (4, 2, 128)])
@pytest.mark.parametrize("window,sinks", [(64, 4), (300, 140), (1000, 1)])
def test_far_pieces(H, Hkv, d, window, sinks):
    """Sequences long enough for several pieces of queries behind the sinks' windows."""
    run([3000, 3000], H, Hkv, d, "dense", window, sinks)


@pytest.mark.parametrize("form", ["packed", "fused"])
@pytest.mark.parametrize("H,Hkv,d", [(3, 3, 64), (12, 4, 128), (7, 1, 128)])
@pytest.mark.parametrize("sinks", [0, 4])
def test_packed_ragged(form, H, Hkv, d, sinks):
    run([130, 0, 1, 129, 2400, 128, 3, 0], H, Hkv, d, form, 150, sinks)


@pytest.mark.parametrize("window,sinks", [(64, 4), (300, 200), (1000, 1)])
def test_unlike_sequences(window, sinks):
    """Many short sequences and a few long ones: the places of the sinks' parts go by the rows."""
    run([3000, 1, 0, 40] + [17] * 60 + [900, 129] + [128] * 5 + [2300, 3], 2, 1, 64, "packed", window, sinks)


@pytest.mark.parametrize("n,H,Hkv,d,form,window,sinks", [
    ([900] * 3, 14, 14, 64, "dense", 200, 4),                   # three steps each, both d's operands
    ([1500] * 2, 16, 8, 128, "dense", 700, 0),                  # half a dozen
    ([1700] * 2, 12, 6, 64, "dense", 1600, 3),                  # one step to fourteen
    ([int(x) for x in np.random.default_rng(1).integers(0, 70, 220)], 4, 2, 64, "packed", 20, 3),       # one step
    ([int(x) for x in np.random.default_rng(2).integers(0, 300, 90)], 6, 3, 128, "packed", 150, 3)])    # one to three
def test_items_one_behind_the_other(n, H, Hkv, d, form, window, sinks):
    """More tiles of rows than SMs, which take them as they come: the same bits again."""
    batch, o, lse, do, how, grads = run(n, H, Hkv, d, form, window, sinks)
    for _ in range(3):
        again = fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, window, sinks, **how)
        assert all(torch.equal(x[:sum(n)], y[:sum(n)]) for x, y in zip(grads, again))
    device_error_clear()


def test_bad_counts_among_many():
    n = [40] * 300
    batch, o, lse, do, how, grads = run(n, 4, 2, 64, "packed", 20, 3)
    n[100], n[101], n[250] = 70, 10, 43                          # above the bound; the others' rows stay theirs
    n[251] = 37
    cu = torch.tensor(np.concatenate(([0], np.cumsum(n))), dtype=torch.int32, device="cuda")
    out = [torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in grads]
    fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, 20, 3, cu_seqlens=cu, max_seqlen=40,
                            dq=out[0], dk=out[1], dv=out[2])
    assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_SEQLENS
    for x, y in zip(out, grads):
        assert (x[4000:4070] == 7).all() and (x[10000:10043] == 7).all()
        for i, j in ((0, 4000), (4080, 10000), (10080, 12000)):
            assert torch.equal(x[i:j], y[i:j])


@pytest.mark.parametrize("d", [64, 128])
def test_timed_out_wait_with_more_tiles_than_sms(d):
    """Each CTA gives up, whatever it has taken on; the next call is not concerned."""
    batch, o, lse, do, how, grads = run([1000] * 2, 20, 20, d, "dense", 130, 4)
    dq = torch.full_like(grads[0], 7.0)
    fa.fa_debug_expire_next_wait(100_000)
    fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, 130, 4, dq=dq)
    assert fa.fa_get_device_error() == fa.FA_DEVERR_WAIT_TIMEOUT
    assert (dq == 7).all()
    again = fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, 130, 4)
    device_error_clear()
    assert all(torch.equal(x, y) for x, y in zip(grads, again))


def test_rows_behind_the_last_sequence_stay():
    batch, o, lse, do, how, want = run([200, 61], 4, 2, 128, "packed", 64, 4, spare=90)
    out = [torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in want]
    fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, 64, 4, dq=out[0], dk=out[1], dv=out[2], **how)
    for x, y in zip(out, want):
        assert (x[261:] == 7).all() and torch.equal(x[:261], y[:261])


def test_into_a_fused_gradient():
    batch, o, lse, do, how, want = run([150, 300], 6, 2, 64, "packed", 100, 4)
    rows = torch.full((len(batch.gq), 10, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, 100, 4, dq=rows[:, :6], dk=rows[:, 6:8],
                            dv=rows[:, 8:], **how)
    assert torch.equal(rows[:450], torch.cat(want, 1)[:450]) and (rows[450:] == 7).all()


def test_scales():
    for scale in (1.0, 1e-3):
        run([300], 4, 2, 64, "dense", 100, 2, scale=scale)


def test_against_differences():
    """Differences of the kernels' own forward along each gradient, summed in fp64: steps of 0.05 a value
    (third-order terms far below 5 %), and the outputs' roundings, a random walk over 400 * 256 values of
    magnitude 1 at most with steps of 2^-8 and dO about 1."""
    batch, o, lse, do, how, grads = run([400], 4, 2, 64, "dense", 90, 4)
    for x, grad in zip((batch.gq, batch.gk, batch.gv), grads):
        e = grad.float() * (0.05 / grad.float().square().mean().sqrt())
        up, down = (x.float() + e).bfloat16(), (x.float() - e).bfloat16()
        out = []
        for y in (up, down):
            args = [y if t is x else t for t in (batch.gq, batch.gk, batch.gv)]
            out.append((fa.attention_window_fwd(*args, 90, 4)[0].double() * do.double()).sum())
        want = (grad.double() * (up.double() - down.double())).sum()
        assert want > 50
        assert abs(out[0] - out[1] - want) <= 0.05 * want + 4 * 2.0 ** -8 * (2 * 400 * 256) ** 0.5


def test_same_bits_and_replayed_graph():
    batch, o, lse, do, how, grads = run([2000], 4, 2, 128, "dense", 64, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, 64, 4)
    for _ in range(2):
        g.replay()
        assert all(torch.equal(x, y) for x, y in zip(grads, again))
    device_error_clear()


def test_graphs_of_two_streams():
    """Two calls captured on two streams, replayed at once, each with a workspace of its own."""
    batch, o, lse, do, how, grads = run([2000], 2, 2, 64, "dense", 64, 4)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs, outs = [], []
    for x in s:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=x):
            outs.append(fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, 64, 4))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for x, g in zip(s, graphs):
            with torch.cuda.stream(x):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for out in outs for x, y in zip(grads, out))


def test_timed_out_wait():
    batch, o, lse, do, how, grads = run([300], 4, 2, 128, "dense", 100, 4)
    dq = torch.full_like(grads[0], 7.0)
    fa.fa_debug_expire_next_wait(1_000_000)
    fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, 100, 4, dq=dq)
    assert fa.fa_get_device_error() == fa.FA_DEVERR_WAIT_TIMEOUT
    assert (dq == 7).all()
    again = fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, 100, 4)
    device_error_clear()
    assert all(torch.equal(x, y) for x, y in zip(grads, again))


def test_bad_counts_are_flagged_and_left_out():
    batch, o, lse, do, how, grads = run([200, 61], 4, 2, 64, "packed", 64, 4)
    out = [torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in grads]
    fa.attention_window_bwd(batch.gq, batch.gk, batch.gv, o, do, lse, 64, 4, cu_seqlens=how["cu_seqlens"],
                            max_seqlen=199, dq=out[0], dk=out[1], dv=out[2])
    assert fa.fa_get_device_error() == fa.FA_DEVERR_BAD_SEQLENS
    for x, y in zip(out, grads):
        assert (x[:200] == 7).all() and torch.equal(x[200:261], y[200:261])


def test_tensor_refusals():
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(2, 4, 3, device="cuda")
    for bad in (dict(do=q.float()), dict(o=q[:1]), dict(lse=lse[:, :, :2]), dict(dk=q), dict(k=k[:, :2], v=k[:, :2]),
                dict(do=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(workspace=lse)):
        args = dict(q=q, k=k, v=k, o=q, do=q, lse=lse, window=4)
        args.update(bad)
        with pytest.raises(ValueError):
            fa.attention_window_bwd(**args)
    with pytest.raises(fa.FaError):
        fa.attention_window_bwd(q, k, k, q, q, lse, 4,
                                workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
