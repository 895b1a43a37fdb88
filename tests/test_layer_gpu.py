"""The operators of an attention layer together, as they would be used: a fused projection's rows normed
and rotated, window attention, and the gradients back into the fused rows; and a decode step over caches
in bf16 and in 4 bits (GB300)."""
import numpy as np
import pytest
import torch

import online_softmax_06_gb300 as fa
from gpu_common import device_error_clear, require_gpu
from oracle import kv4, layer
from window_common import bf16, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def cuda_i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def half_step(x):
    """x as bf16 holds it."""
    return f64(bf16(x))


def training(lens, H, Hkv, d, window, sinks, interleaved, seed):
    """One layer's training step into a fused gradient; and the oracle's, whose rows take the roundings
    to bf16 that the kernels' outputs have (normed Q and K, O, the gradients of those)."""
    rng = np.random.default_rng(seed)
    T, rows = sum(lens), H + 2 * Hkv
    fused = bf16(rng.standard_normal((T, rows, d)))
    wq, wk = (1 + 0.2 * rng.standard_normal(d) for _ in "qk")
    freq = 10000.0 ** (-np.arange(0, d // 2, 2) / (d // 2))
    pos = np.concatenate([np.arange(n) for n in lens])
    do = bf16(rng.standard_normal((T, H, d)))
    x, gdo = fused.cuda(), do.cuda()
    args = (torch.tensor(wq, dtype=torch.float32, device="cuda"), torch.tensor(wk, dtype=torch.float32, device="cuda"),
            torch.tensor(freq, device="cuda"), cuda_i32(pos))
    cu, most = cuda_i32(np.concatenate(([0], np.cumsum(lens)))), max(lens)
    how = dict(window=window, sinks=sinks)
    k0, v0 = H, H + Hkv
    grad = torch.full_like(x, float("nan"))

    def step():
        q, k = fa.qk_norm_rope_fwd(x[:, :k0], x[:, k0:v0], *args, interleaved=interleaved)
        o, lse = fa.attention_window_fwd(q, k, x[:, v0:], cu_seqlens_q=cu, cu_seqlens_k=cu, max_q=most, max_k=most, **how)
        fa.attention_window_bwd(q, k, x[:, v0:], o, gdo, lse, cu_seqlens=cu, max_seqlen=most, dq=grad[:, :k0],
                                dk=grad[:, k0:v0], dv=grad[:, v0:], **how)
        dw = fa.qk_norm_rope_bwd(x[:, :k0], x[:, k0:v0], grad[:, :k0], grad[:, k0:v0], *args, interleaved=interleaved,
                                 dq=grad[:, :k0], dk=grad[:, k0:v0])[2:]
        return o, dw

    o, dw = step()
    device_error_clear()
    xf, dof = f64(fused), f64(do)
    w32 = [f64(a) for a in args[:2]]
    q = half_step(layer.norm_rope(xf[:, :k0], w32[0], pos, freq, 1e-6, interleaved))
    k = half_step(layer.norm_rope(xf[:, k0:v0], w32[1], pos, freq, 1e-6, interleaved))
    want = np.zeros_like(xf)
    out = np.zeros((T, H, d))
    at = 0
    for n in lens:
        s = slice(at, at + n)
        out[s] = layer.window_attention(q[s], k[s], xf[s, v0:], window, sinks, d ** -0.5)[0]
        want[s, :k0], want[s, k0:v0], want[s, v0:] = layer.window_attention_bwd(q[s], k[s], xf[s, v0:], dof[s], window,
                                                                                sinks, d ** -0.5)
        at += n
    dws = []
    for a, b, w in ((0, k0, w32[0]), (k0, v0, w32[1])):
        want[:, a:b], g = layer.norm_rope_bwd(xf[:, a:b], want[:, a:b], w, pos, freq, 1e-6, interleaved)
        dws.append(g)
    return x, step, grad, o, dw, out, want, dws


def close(got, want, share):
    """In norm: roundings are independent, so that a share of the whole is what they come to."""
    err = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
    assert err <= share, err


@pytest.mark.parametrize("lens,H,Hkv,d,window,sinks,interleaved", [
    ([300, 1, 700], 8, 2, 64, 128, 4, False), ([513], 6, 3, 128, 200, 0, True), ([1500, 40], 2, 1, 128, 100, 20, False)])
def test_training_step(lens, H, Hkv, d, window, sinks, interleaved):
    x, step, grad, o, dw, out, want, dws = training(lens, H, Hkv, d, window, sinks, interleaved, sum(lens))
    k0, v0 = H, H + Hkv
    # bf16 operands and results, each 2^-9 rms of its value at most: q, k, P and O for O; those, dS, the
    # gradients of q and k and the result (six, of which sums over keys keep their share) for the rest
    close(o, out, 4 * 2.0 ** -9)
    for a, b in ((0, k0), (k0, v0), (v0, v0 + Hkv)):
        close(grad[:, a:b], want[:, a:b], 7 * 2.0 ** -9)
    for g, r in zip(dw, dws):
        close(g, r, 7 * 2.0 ** -9)


def test_training_step_captured_while_an_eager_one_lives():
    x, step, grad, o, dw, out, want, dws = training([300, 500], 4, 2, 64, 128, 4, False, 7)
    eager = [grad.clone(), o.clone(), dw[0].clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        o2, dw2 = step()
    grad.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(grad, eager[0]) and torch.equal(o2, eager[1]) and torch.equal(dw2[0], eager[2])
    assert torch.equal(step()[0], eager[1])
    device_error_clear()


def test_gradient_through_autograd():
    """The two operators as autograd functions: leaves get what the calls give, added to what they have."""

    class NormRope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, wq, wk, freq, pos):
            ctx.save_for_backward(q, k, wq, wk, freq, pos)
            return fa.qk_norm_rope_fwd(q, k, wq, wk, freq, pos)

        @staticmethod
        def backward(ctx, gq, gk):
            q, k, wq, wk, freq, pos = ctx.saved_tensors
            return (*fa.qk_norm_rope_bwd(q, k, gq.contiguous(), gk.contiguous(), wq, wk, freq, pos), None, None)

    class Window(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v):
            o, lse = fa.attention_window_fwd(q, k, v, 100, 4)
            ctx.save_for_backward(q, k, v, o, lse)
            return o

        @staticmethod
        def backward(ctx, do):
            q, k, v, o, lse = ctx.saved_tensors
            return fa.attention_window_bwd(q, k, v, o, do.contiguous(), lse, 100, 4)

    gen = torch.Generator("cuda").manual_seed(3)
    leaf = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16().requires_grad_()  # noqa: E731
    q, k, v = leaf(2, 300, 4, 64), leaf(2, 300, 2, 64), leaf(2, 300, 2, 64)
    wq, wk = (torch.ones(64, device="cuda", requires_grad=True) for _ in "qk")
    freq = torch.tensor(10000.0 ** (-np.arange(0, 64, 2) / 64), device="cuda")
    pos = torch.arange(300, dtype=torch.int32, device="cuda").repeat(2, 1).contiguous()
    do = torch.randn(2, 300, 4, 64, generator=gen, device="cuda").bfloat16()
    for _ in range(2):
        Window.apply(*NormRope.apply(q, k, wq, wk, freq, pos), v).backward(do)
    qq, kk = fa.qk_norm_rope_fwd(q.detach(), k.detach(), wq.detach(), wk.detach(), freq, pos)
    o, lse = fa.attention_window_fwd(qq, kk, v.detach(), 100, 4)
    gq, gk, gv = fa.attention_window_bwd(qq, kk, v.detach(), o, do, lse, 100, 4)
    gq, gk, gwq, gwk = fa.qk_norm_rope_bwd(q.detach(), k.detach(), gq, gk, wq.detach(), wk.detach(), freq, pos)
    for x, g in zip((q, k, v, wq, wk), (gq, gk, gv, gwq, gwk)):
        assert torch.equal(x.grad, g + g)


def test_decode_steps():
    """Prompts written and steps taken: each new token normed, rotated, put into a bf16 cache and a 4-bit
    one; the window's attention over the former, the whole one's over the latter."""
    rng = np.random.default_rng(11)
    H, Hkv, d, room, page = 8, 2, 64, 400, 32
    L = [300, 37, 0]
    B, steps, window, sinks = len(L), 3, 90, 4
    freq = 10000.0 ** (-np.arange(0, d, 2) / d)
    w = 1 + 0.2 * rng.standard_normal((2, d))
    dev = [torch.tensor(x, dtype=torch.float32, device="cuda") for x in w]
    gf = torch.tensor(freq, device="cuda")
    table = cuda_i32(np.arange(B * -(-room // page)).reshape(B, -1))
    cache4 = fa.kv4_cache(table.numel(), Hkv, page, d)
    cache = torch.full((2, B, room, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    held = [np.zeros((2, 0, Hkv, d)) for _ in L]

    def put(x, lens, n):
        """The last n[b] tokens of lens[b], packed rows x of a fused projection."""
        T = len(x)
        pos = np.concatenate([np.arange(a - m, a) for a, m in zip(lens, n)]).astype(int)
        gx = x.cuda()
        q, k = fa.qk_norm_rope_fwd(gx[:, :H], gx[:, H:H + Hkv], *dev, gf, cuda_i32(pos))
        v = gx[:, H + Hkv:]
        seq = np.repeat(np.arange(B), n)
        cache[0][seq, pos], cache[1][seq, pos] = k, v.contiguous()
        fa.kv4_append(k, v, cache4, table, cuda_i32(lens), cuda_i32(np.concatenate(([0], np.cumsum(n)))), max(n))
        xf = f64(x)
        rq = half_step(layer.norm_rope(xf[:, :H], f64(dev[0]), pos, freq, 1e-6, False))
        rk = half_step(layer.norm_rope(xf[:, H:H + Hkv], f64(dev[1]), pos, freq, 1e-6, False))
        for b in range(B):
            held[b] = np.concatenate((held[b], np.stack((rk[seq == b], xf[seq == b, H + Hkv:]))), 1)
        return q, rq.reshape(T, H, d)

    rows = lambda n: bf16(rng.standard_normal((n, H + 2 * Hkv, d)))  # noqa: E731
    put(rows(sum(L)), L, L)
    for t in range(1, steps + 1):
        lens = [x + t for x in L]
        q, rq = put(rows(B), lens, [1] * B)
        o, lse = fa.attention_window_fwd(q[:, None], cache[0], cache[1], window, sinks, seqlens_k=cuda_i32(lens))
        o4, lse4 = fa.attention_kv4(q[:, None].contiguous(), cache4, table, cuda_i32(lens))
        device_error_clear()
        for b in range(B):
            ro, rl = layer.window_attention(rq[b:b + 1], held[b][0], held[b][1], window, sinks, d ** -0.5)
            assert np.abs(f64(o[b]) - ro).max() <= 2.0 ** -6 * np.abs(ro).max()
            assert np.abs(f64(lse[b]) - rl).max() <= 2.0 ** -7     # keys a half step of bf16 apart at most
            vals = [kv4.values(*kv4.quantise(x, 64)) for x in held[b]]
            r4 = kv4.attention(rq[b:b + 1], vals[0], vals[1], d ** -0.5, True)[0]
            assert np.abs(f64(o4[b]) - r4).max() <= 0.05 * max(1.0, np.abs(r4).max())
