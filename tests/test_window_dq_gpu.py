"""dQ of the window attention: which keys it depends on, and how exact it is in norm (GB300).

The bound in norm.  dS is rounded to bf16 for the product and dQ (dK) at the end, P and dV likewise:
each off by half a step at most, 2^-8 of the value, evenly spread, so 2^-8 / sqrt(3) rms; the roundings
of single values are independent, so that a sum of many terms is off by the same share of its norm
where the terms do not cancel: together 2^-8 sqrt(2 / 3).  Terms that cancel are those along what a
row's keys have in common (a row's dS add up to 0): there dQ has the sum of dS, roundings and all,
taken off.  D comes from O rounded to bf16; what that adds to a row's dS adds to their sum and goes
with it.
"""
import numpy as np
import pytest
import torch

import online_softmax_06_gb300 as fa
from gpu_common import device_error_clear, require_gpu
from window_common import bf16, f64, layer

pytestmark = pytest.mark.gpu
IN_NORM = 2.0 ** -8 * (2 / 3) ** 0.5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def gradients(q, k, v, do, window, sinks, cu=None, most=None):
    fwd = {} if cu is None else dict(cu_seqlens_q=cu, cu_seqlens_k=cu, max_q=most, max_k=most)
    bwd = {} if cu is None else dict(cu_seqlens=cu, max_seqlen=most)
    o, lse = fa.attention_window_fwd(q, k, v, window, sinks, **fwd)
    return fa.attention_window_bwd(q, k, v, o, do, lse, window, sinks, **bwd)


@pytest.mark.parametrize("H,Hkv,d", [(1, 1, 128), (4, 1, 128), (4, 2, 64), (6, 2, 128)])
@pytest.mark.parametrize("window,sinks", [(128, 0), (128, 4), (300, 0), (40, 0)])
def test_keys_that_a_query_does_not_see(H, Hkv, d, window, sinks):
    """A key 128 times as large changes no bit of dQ of the queries that do not see it."""
    N, rng = 900, np.random.default_rng(window + H)
    q, k, v, do = (bf16(rng.standard_normal((1, N, h, d))).cuda() for h in (H, Hkv, Hkv, H))
    v = v + bf16(rng.standard_normal((Hkv, d))).cuda()            # values with a part in common
    want = gradients(q, k, v, do, window, sinks)[0]
    P = 128 // (H // Hkv)
    tiles = [i // P * P for i in (N // 2, N - 1)]
    # the first key of a tile's first query and the last of its last, and ones between
    for key in {max(sinks, t + x) for t in tiles for x in (1 - window, 33 - window, -7, min(P, N - t) - 1)}:
        far = k.clone()
        far[:, key] *= 128
        got = gradients(q, far, v, do, window, sinks)[0]
        rows = np.r_[0:key, min(N, key + window):N]
        assert torch.equal(got[:, rows], want[:, rows]), (key, (got - want)[0, rows].abs().amax((-1, -2)).argmax())
        assert not torch.equal(got, want)
    device_error_clear()


def share(got, want):
    return float(np.linalg.norm(f64(got) - want) / np.linalg.norm(want))


def compare(lens, H, Hkv, d, window, sinks, k_off, v_off, seed=0, first=1.0):
    """Packed sequences whose kv heads' keys and values have unlike parts in common; `first`: what the first
    key of each is multiplied by."""
    rng = np.random.default_rng(seed)
    T = sum(lens)
    q, do = (bf16(rng.standard_normal((T, H, d))) for _ in "qo")
    k, v = (rng.standard_normal((T, Hkv, d)) + off * rng.standard_normal((Hkv, d)) for off in (k_off, v_off))
    at = np.concatenate(([0], np.cumsum(lens)))
    k[[a for a, n in zip(at, lens) if n]] *= first
    k, v = bf16(k), bf16(v)
    cu = torch.tensor(at, dtype=torch.int32, device="cuda")
    grads = gradients(q.cuda(), k.cuda(), v.cuda(), do.cuda(), window, sinks, cu, max(lens))
    device_error_clear()
    want = [np.concatenate(x) for x in zip(*(
        layer.window_attention_bwd(*(f64(x[a:b]) for x in (q, k, v, do)), window, sinks, d ** -0.5)
        for a, b in zip(at, at[1:])))]
    for name, g, w in zip("qkv", grads, want):
        assert share(g, w) <= IN_NORM, (name, share(g, w), [share(x, y) for x, y in zip(grads, want)])


@pytest.mark.parametrize("k_off,v_off", [(0, 0), (1, 0.1), (0, 1), (0, 2), (2, 2)])
@pytest.mark.parametrize("lens,H,Hkv,d,window,sinks", [
    ([1500, 1400], 4, 2, 128, 700, 4), ([1300, 700], 6, 6, 64, 150, 0), ([1800], 4, 1, 64, 1024, 0)])
def test_parts_in_common(lens, H, Hkv, d, window, sinks, k_off, v_off):
    compare(lens, H, Hkv, d, window, sinks, k_off, v_off)


@pytest.mark.parametrize("H,Hkv,d", [(20, 10, 64), (16, 16, 128)])
def test_parts_in_common_of_many_items(H, Hkv, d):
    """Several tiles of rows a CTA, of kv heads that are unlike."""
    compare([900, 1, 200, 1000, 333], H, Hkv, d, 200, 3, 2, 1)


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_shorter_than_the_window(d):
    compare([200, 150, 33, 400, 128, 7, 1, 0, 260], 8, 2, d, 4096, 4, 1, 1)


@pytest.mark.parametrize("first", [8.0, 64.0])
@pytest.mark.parametrize("window,sinks", [(500, 0), (500, 4), (150, 1)])
def test_a_large_first_key(window, sinks, first):
    """The first key takes most of a row's weight, or next to none."""
    compare([1300], 4, 2, 128, window, sinks, 0, 0, first=first)


@pytest.mark.parametrize("n", [1, 2, 3, 129])
def test_single_keys(n):
    """A query that sees its own key alone has no gradient: what dS holds is taken off whole."""
    rng = np.random.default_rng(n)
    q, k, v, do = (bf16(rng.standard_normal((1, n, 2, 64))).cuda() for _ in "qkvo")
    dq = gradients(q, k, v, do, 1, 0)[0]
    # P is off by 2^-18 of itself (scores, exp2 and log2 of magnitudes below 32), times dP (below 64) and the key (4)
    assert dq.abs().max() <= 2.0 ** -18 * 64 * 4
