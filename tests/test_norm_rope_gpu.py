"""Norm and rotation of queries and keys, and its gradient, against the fp64 oracle (GB300).

Tolerances.  An output is rounded once to bf16: half a step, 2^-8 of its value.  Before that, in
fp32: the sum of squares (a tree of 12 additions), the root, four products, sine and cosine, each
within a few 2^-24, together below 2^-18 of the largest value that goes into the row.  The
weights' gradient is a chain of at most some hundred fp32 additions of such terms: 2^-16 of the
sum of their magnitudes.
"""
import numpy as np
import pytest
import torch

import online_softmax_06_gb300 as fa
from gpu_common import device_error_clear, require_gpu
from oracle import layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def freqs(rot, base=10000.0):
    return torch.from_numpy(base ** (-np.arange(0, rot, 2) / max(rot, 1))).cuda()


def rows(rng, T, heads, d, scale=1.0):
    x = rng.standard_normal((T, heads, d)) * np.exp(rng.standard_normal((heads, d))) * scale
    return torch.from_numpy(x).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def check_out(got, ref, extra=0.0):
    top = np.abs(ref).max(-1, keepdims=True) if ref.size else ref
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * (top + extra) + 1e-30
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), (err / tol).max()


CASES = [
    # T, H, Hkv, d, rot, interleaved, far
    (1, 16, 2, 64, 64, False, 600),
    (1, 1, 1, 128, 128, False, 2 ** 31 - 1),
    (3, 5, 3, 128, 64, False, 100000),
    (33, 33, 1, 64, 8, True, 4000000),
    (257, 7, 7, 128, 128, True, 131072),
    (100, 32, 8, 128, 0, False, 10),
    (1001, 15, 5, 64, 32, True, 131072),
    (700, 8, 0, 128, 96, False, 1000),
    (700, 0, 9, 64, 56, False, 1000),
    (6000, 3, 2, 128, 128, False, 6000),
]


def inputs(case, seed=0):
    T, H, Hkv, d, rot, inter, far = case
    rng = np.random.default_rng(seed)
    q, k = rows(rng, T, H, d), rows(rng, T, Hkv, d)
    w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).float() for _ in "qk"]
    pos = torch.from_numpy(rng.integers(-far // 2, far, T)).int()
    pos[0] = far
    return rng, q, k, w, pos


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("fused", [False, True])
def test_forward(case, fused):
    T, H, Hkv, d, rot, inter, far = case
    rng, q, k, w, pos = inputs(case)
    if fused:                             # slices of a projection's rows
        both = torch.cat((q, k, torch.full((T, 2, d), float("nan"), dtype=q.dtype)), 1).cuda()
        gq, gk = both[:, :H], both[:, H:H + Hkv]
    else:
        gq, gk = q.cuda(), k.cuda()
    yq, yk = fa.qk_norm_rope_fwd(gq, gk, w[0].cuda(), w[1].cuda(), freqs(rot), pos.cuda(),
                                 interleaved=inter)
    fr = f64(freqs(rot))
    for y, x, ww in ((yq, q, w[0]), (yk, k, w[1])):
        check_out(y, layer.norm_rope(f64(x), f64(ww), pos.numpy(), fr, 1e-6, inter))
    device_error_clear()


@pytest.mark.parametrize("case", CASES)
def test_gradient(case):
    T, H, Hkv, d, rot, inter, far = case
    rng, q, k, w, pos = inputs(case, 1)
    dy = [torch.from_numpy(rng.standard_normal(x.shape)).to(torch.bfloat16) for x in (q, k)]
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q.cuda(), k.cuda(), dy[0].cuda(), dy[1].cuda(),
                                           w[0].cuda(), w[1].cuda(), freqs(rot), pos.cuda(),
                                           interleaved=inter)
    fr = f64(freqs(rot))
    for dx, dw, x, g, ww in ((dq, dwq, q, dy[0], w[0]), (dk, dwk, k, dy[1], w[1])):
        rx, rw = layer.norm_rope_bwd(f64(x), f64(g), f64(ww), pos.numpy(), fr, 1e-6, inter)
        # what goes into dx: r h and r x^ mean(h x^), whose sum may cancel
        r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + 1e-6)
        h = layer.rotate(f64(g), pos.numpy(), fr, inter, back=True)
        hat = f64(x) * r
        into = r * (np.abs(h * f64(ww)).max(-1, keepdims=True) if x.numel() else 0)
        into = into + r * (np.abs(hat).max(-1, keepdims=True) if x.numel() else 0) * np.abs(
            h * f64(ww) * hat).mean(-1, keepdims=True)
        check_out(dx, rx, into)
        tol = 2.0 ** -16 * np.abs(h * hat).sum((0, 1)) + 1e-30
        err = np.abs(f64(dw) - rw)
        assert np.all(err <= tol), (err / tol).max()
    device_error_clear()


def test_gradient_against_differences():
    """The oracle's gradient is that of the oracle's forward."""
    rng, q, k, w, pos = inputs((2, 2, 0, 64, 32, True, 50), 2)
    x, ww, fr = f64(q), f64(w[0]), f64(freqs(32))
    up = rng.standard_normal(x.shape)
    f = lambda x, ww: (layer.norm_rope(x, ww, pos.numpy(), fr, 1e-6, True) * up).sum()  # noqa: E731
    dx, dw = layer.norm_rope_bwd(x, up, ww, pos.numpy(), fr, 1e-6, True)
    for _ in range(10):
        e, we = rng.standard_normal(x.shape), rng.standard_normal(ww.shape)
        h = 1e-6
        d = (f(x + h * e, ww + h * we) - f(x - h * e, ww - h * we)) / (2 * h)
        want = (dx * e).sum() + (dw * we).sum()
        assert abs(d - want) <= 1e-6 * (np.abs(dx * e).sum() + np.abs(dw * we).sum())


def test_in_place_same_bits_and_rows_beside():
    """In place as beside; what stands between the heads' rows stays as it was."""
    rng, q, k, w, pos = inputs((50, 6, 2, 128, 64, False, 1000), 3)
    rest = torch.full((50, 2, 128), float("nan"), dtype=q.dtype)
    both = torch.cat((q, k, rest), 1).cuda()
    args = (w[0].cuda(), w[1].cuda(), freqs(64), pos.cuda())
    want = fa.qk_norm_rope_fwd(q.cuda(), k.cuda(), *args)
    got = fa.qk_norm_rope_fwd(both[:, :6], both[:, 6:8], *args, q_out=both[:, :6],
                              k_out=both[:, 6:8])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.isnan(both[:, 8:]).all()
    gq, gk = torch.randn(q.shape).bfloat16().cuda(), torch.randn(k.shape).bfloat16().cuda()
    want = fa.qk_norm_rope_bwd(q.cuda(), k.cuda(), gq, gk, *args)
    got = fa.qk_norm_rope_bwd(q.cuda(), k.cuda(), gq, gk, *args, dq=gq, dk=gk)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_dense_batch_no_weights_zero_rows_and_nan():
    rng = np.random.default_rng(5)
    q = rows(rng, 6, 4, 64).reshape(2, 3, 4, 64)
    q[0, 1, 2] = 0
    q[1, 0, 3, 5] = float("nan")
    pos = torch.arange(6).reshape(2, 3).int()
    yq, yk = fa.qk_norm_rope_fwd(q.cuda(), q.cuda(), None, None, freqs(64), pos.cuda(), eps=1e-5)
    assert yq.shape == q.shape and (yq[0, 1, 2] == 0).all()
    assert torch.isnan(yq[1, 0, 3]).all() and torch.isnan(yq).sum() == 64   # its own row alone
    ok = ~np.isnan(f64(q)).any(-1).reshape(6, 4)
    ref = layer.norm_rope(np.nan_to_num(f64(q)).reshape(6, 4, 64), 1.0, np.arange(6),
                          f64(freqs(64)), 1e-5, False)
    for y in (yq, yk):
        err = np.abs(np.nan_to_num(f64(y)).reshape(6, 4, 64) - ref)[ok]
        assert np.all(err <= 2.0 ** -8 * np.abs(ref[ok]) + 2.0 ** -16)
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q.cuda(), q.cuda(), yq, yk, None, None, freqs(64),
                                           pos.cuda(), eps=1e-5)
    assert dwq is None and dwk is None and dq.shape == q.shape


def test_no_tokens():
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    w, pos = torch.ones(64, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    assert fa.qk_norm_rope_fwd(e, e, w, w, freqs(64), pos)[0].shape == e.shape
    out = fa.qk_norm_rope_bwd(e, e, e, e, w, w, freqs(64), pos)
    assert (out[2] == 0).all() and (out[3] == 0).all()


def test_replayed_graph_other_stream():
    rng, q, k, w, pos = inputs((40, 6, 2, 128, 128, False, 1000), 6)
    q, k, pos = q.cuda(), k.cuda(), pos.cuda()
    args = (w[0].cuda(), w[1].cuda(), freqs(128), pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fa.qk_norm_rope_fwd(q, k, *args)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = fa.qk_norm_rope_fwd(q, k, *args)
        out = fa.qk_norm_rope_bwd(q, k, *y, *args)
    q.copy_(torch.randn(q.shape))
    g.replay()
    want = fa.qk_norm_rope_fwd(q, k, *args)
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
    assert all(torch.equal(a, b) for a, b in zip(out, fa.qk_norm_rope_bwd(q, k, *want, *args)))


def test_tensor_refusals():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (dict(q=q.float()), dict(positions=pos[:3]), dict(positions=pos.long()),
                dict(positions=None), dict(q_weight=w.half()), dict(q_weight=w[:32].contiguous()),
                dict(inv_freq=freqs(64).float()), dict(q=q.transpose(0, 1)),
                dict(k=torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")),
                dict(q_out=torch.zeros(4, 3, 64, dtype=torch.bfloat16, device="cuda")),
                dict(q=q.cpu())):
        args = dict(q=q, k=q, q_weight=w, k_weight=w, inv_freq=freqs(64), positions=pos)
        args.update(bad)
        with pytest.raises(ValueError):
            fa.qk_norm_rope_fwd(**args)
    with pytest.raises(fa.FaError):
        fa.qk_norm_rope_fwd(q, q, w, w, freqs(12), pos)
    with pytest.raises(fa.FaError):
        fa.qk_norm_rope_fwd(q, q, w, w, freqs(64), pos, eps=-1.0)
