"""Refusals of the window attention's C entry points: all return before any CUDA call (no GPU); and the
oracle's gradient against differences of its forward."""
import numpy as np
import pytest

import online_softmax_06_gb300 as fa
from oracle import layer

P = 0x1000   # an address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


def fwd(**kw):
    a = dict(q=P, qs=512, k=P, ks=256, v=P, vs=256, o=P, lse=P, B=2, Nq=4, total_q=8, Nk=10, total_k=20, H=4, Hkv=2,
             d=128, scale=0.1, window=8, sinks=2, cu_q=None, cu_k=None, sl=None)
    a.update(kw)
    return fa.fa_attention_window_fwd(*a.values())


def test_forward_refusals():
    for bad in (dict(B=-1), dict(Nq=-1), dict(total_q=9), dict(total_k=21), dict(window=0), dict(sinks=-1),
                dict(H=5), dict(Hkv=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(qs=504), dict(ks=248), dict(vs=128)):
        assert fwd(**bad) == fa.FA_ERR_BAD_SIZE, bad
    for bad in (dict(d=96), dict(H=258, qs=258 * 128)):
        assert fwd(**bad) == fa.FA_ERR_UNSUPPORTED, bad
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(lse=None)):
        assert fwd(**bad) == fa.FA_ERR_NULL_POINTER, bad
    for bad in (dict(q=P + 8), dict(k=P + 2), dict(o=P + 4), dict(lse=P + 2), dict(cu_q=P + 1), dict(cu_k=P + 2),
                dict(sl=P + 1), dict(qs=516), dict(ks=257)):
        assert fwd(**bad) == fa.FA_ERR_MISALIGNED, bad
    for bad in (dict(B=1, Nk=2 ** 31 - 1, total_k=2 ** 31 - 1, total_q=4), dict(qs=1 << 32)):
        assert fwd(**bad) == fa.FA_ERR_TOO_LARGE, bad
    assert fwd(B=0, total_q=0, total_k=0) == fa.FA_OK
    assert fwd(Nq=0, total_q=0) == fa.FA_OK
    assert fwd(H=0, Hkv=0) == fa.FA_OK


def bwd(**kw):
    a = dict(q=P, qs=512, k=P, ks=256, v=P, vs=256, o=P, do=P, lse=P, dq=P, dqs=512, dk=P, dks=256, dv=P, dvs=256, B=2,
             N=40, total=80, H=4, Hkv=2, d=128, scale=0.1, window=8, sinks=2, cu=None, ws=P, n=1 << 30)
    a.update(kw)
    return fa.fa_attention_window_bwd(*a.values())


def test_gradient_refusals():
    for bad in (dict(B=-1), dict(N=-1), dict(total=81), dict(window=0), dict(sinks=-1), dict(H=5), dict(Hkv=0),
                dict(scale=0.0), dict(qs=504), dict(dqs=504), dict(dks=128), dict(dvs=248), dict(n=100)):
        assert bwd(**bad) == fa.FA_ERR_BAD_SIZE, bad
    for bad in (dict(d=96), dict(H=258, qs=258 * 128)):
        assert bwd(**bad) == fa.FA_ERR_UNSUPPORTED, bad
    for x in ("q", "k", "v", "o", "do", "lse", "dq", "dk", "dv", "ws"):
        assert bwd(**{x: None}) == fa.FA_ERR_NULL_POINTER, x
    for bad in (dict(do=P + 8), dict(dq=P + 2), dict(dv=P + 8), dict(ws=P + 128), dict(cu=P + 2), dict(dks=260)):
        assert bwd(**bad) == fa.FA_ERR_MISALIGNED, bad
    assert bwd(total=1 << 31, cu=P) == fa.FA_ERR_TOO_LARGE
    assert bwd(total=0, cu=P) == fa.FA_OK


def test_gradient_workspace():
    n = fa.fa_attention_window_bwd_workspace_bytes
    assert n(1, 100, 100, 4, 2, 96, 8, 0) == fa.FA_ERR_UNSUPPORTED
    assert n(1, 100, 100, 4, 3, 64, 8, 0) == fa.FA_ERR_BAD_SIZE
    assert n(0, 100, 0, 4, 2, 64, 8, 0) == 0
    assert n(2, 1000, 2000, 4, 2, 64, 8, 0) == 2000 * 4 * 4                     # D alone
    assert n(2, 1000, 2000, 4, 2, 64, 1000, 4) == 2000 * 4 * 4                  # no query behind the window
    assert n(2, 1000, 2000, 4, 2, 64, 8, 1000) == 2000 * 4 * 4                  # all keys are sinks
    # 1000 tokens: eight tiles, two of them near the sinks' tile: one piece behind
    assert n(2, 1000, 2000, 4, 2, 64, 8, 4) == 2000 * 4 * 4 + 2 * 2 * 2 * 2 * 128 * 64 * 4


def test_gradient_workspace_of_unlike_sequences():
    """One long sequence among many: room for its parts, not for as many of each."""
    n = fa.fa_attention_window_bwd_workspace_bytes
    part = 2 * 128 * 64 * 4
    places = (n(1000, 32768, 100000, 2, 1, 64, 1024, 4) - 100000 * 2 * 4) // part
    assert places == 3 * 100000 // (128 * 9)
    # every sequence's parts fit its places
    rng = np.random.default_rng(0)
    for _ in range(2000):
        window = int(rng.integers(1, 3000))
        near = (window + 254) // 128
        lens = rng.integers(0, 20000, 20) * (rng.random(20) < 0.4)
        cu = np.concatenate(([0], np.cumsum(lens)))
        piece = max(8, near)
        for b, x in enumerate(lens):
            tiles = -(-int(x) // 128)
            if tiles > near:
                parts = 1 + -(-(tiles - near) // piece)
                at = [3 * int(c) // (128 * near) for c in cu[b:b + 2]]
                assert at[1] - at[0] >= parts


def test_oracle_gradient():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((7, 2, 8)), rng.standard_normal((7, 2, 8))
    do = rng.standard_normal(q.shape)
    f = lambda q, k, v: (layer.window_attention(q, k, v, 3, 1, 0.3)[0] * do).sum()  # noqa: E731
    grads = layer.window_attention_bwd(q, k, v, do, 3, 1, 0.3)
    for _ in range(10):
        e = [rng.standard_normal(x.shape) for x in (q, k, v)]
        h = 1e-5
        d = (f(*(x + h * y for x, y in zip((q, k, v), e))) - f(*(x - h * y for x, y in zip((q, k, v), e)))) / (2 * h)
        want = sum((g * y).sum() for g, y in zip(grads, e))
        assert abs(d - want) <= 1e-7 * sum(np.abs(g * y).sum() for g, y in zip(grads, e))


def test_oracle_mask():
    seen = layer.window_seen(3, 6, 2, 1)
    assert seen.astype(int).tolist() == [[1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert layer.window_seen(2, 1, 5, 5).astype(int).tolist() == [[0], [1]]
