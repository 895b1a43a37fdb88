"""The operators of a layer where rows of Q, O and the gradients lie behind 2^31 elements (GB300): the last
sequence gets what it gets alone."""
import pytest
import torch

import online_softmax_06_gb300 as fa
from gpu_common import device_error_clear, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def rows(gen, T, heads, d):
    x = torch.empty(T, heads, d, dtype=torch.bfloat16, device="cuda")
    for part in x.split(16384):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda", dtype=torch.bfloat16))
    return x


def test_window_attention_and_gradients():
    H, Hkv, d, window, sinks, lens = 64, 4, 128, 300, 4, [264000, 9001]
    T, first = sum(lens), lens[0]
    assert first * H * d > 2 ** 31
    gen = torch.Generator("cuda").manual_seed(1)
    q, do = rows(gen, T, H, d), rows(gen, T, H, d)
    k, v = rows(gen, T, Hkv, d), rows(gen, T, Hkv, d)

    def step(cu, most, q, k, v, do):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, lse = fa.attention_window_fwd(q, k, v, window, sinks, cu_seqlens_q=cu, cu_seqlens_k=cu, max_q=most, max_k=most)
        return o, lse, fa.attention_window_bwd(q, k, v, o, do, lse, window, sinks, cu_seqlens=cu, max_seqlen=most)

    o, lse, grads = step([0, first, T], first, q, k, v, do)
    wo, wl, want = step([0, lens[1]], lens[1], *(x[first:] for x in (q, k, v, do)))
    device_error_clear()
    assert torch.equal(o[first:], wo) and torch.equal(lse[:, first:], wl)
    for x, y in zip(grads, want):
        assert torch.equal(x[first:], y)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_and_rotation(interleaved):
    H, Hkv, d, T, last = 64, 16, 128, 212000, 500
    assert (T - last) * (H + Hkv) * d > 2 ** 31
    gen = torch.Generator("cuda").manual_seed(2)
    x, g = rows(gen, T, H + Hkv, d), rows(gen, T, H + Hkv, d)
    freq = 10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    part = lambda t: (t[:, :H], t[:, H:])                         # noqa: E731
    how = dict(inv_freq=freq, interleaved=interleaved)
    want = fa.qk_norm_rope_fwd(*part(x[-last:].clone()), positions=pos[-last:].clone(), **how)
    back = fa.qk_norm_rope_bwd(*part(x[-last:].clone()), *part(g[-last:].clone()), positions=pos[-last:].clone(), **how)
    fa.qk_norm_rope_bwd(*part(x), *part(g), positions=pos, dq=g[:, :H], dk=g[:, H:], **how)
    fa.qk_norm_rope_fwd(*part(x), positions=pos, q_out=x[:, :H], k_out=x[:, H:], **how)
    device_error_clear()
    assert torch.equal(x[-last:], torch.cat(want, 1)) and torch.equal(g[-last:], torch.cat(back[:2], 1))
