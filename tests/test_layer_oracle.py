"""The float64 oracle of the norm, the rotation and the window attention, against torch's operations and
their automatic gradients in float64 (CPU)."""
import numpy as np
import pytest
import torch

from oracle import layer


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_norm_and_rotation(rot, interleaved):
    rng = np.random.default_rng(rot)
    x = torch.tensor(rng.standard_normal((5, 3, 8)), requires_grad=True)
    w = torch.tensor(rng.standard_normal(8), requires_grad=True)
    dy = rng.standard_normal((5, 3, 8))
    pos, freq = np.array([0, 7, 2, 100000, 1]), rng.random(rot // 2)
    n = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w
    turn = torch.polar(torch.ones(5, 1, rot // 2, dtype=torch.float64), torch.tensor(pos[:, None, None] * freq))
    head = n[..., :rot]
    if interleaved:
        z = torch.complex(head[..., 0::2], head[..., 1::2]) * turn
        head = torch.stack((z.real, z.imag), -1).flatten(-2)
    else:
        z = torch.complex(head[..., :rot // 2], head[..., rot // 2:]) * turn
        head = torch.cat((z.real, z.imag), -1)
    y = torch.cat((head, n[..., rot:]), -1)
    y.backward(torch.tensor(dy))
    args = (w.detach().numpy(), pos, freq, 1e-5, interleaved)
    np.testing.assert_allclose(layer.norm_rope(x.detach().numpy(), *args), y.detach().numpy(), atol=1e-12)
    dx, dw = layer.norm_rope_bwd(x.detach().numpy(), dy, *args)
    np.testing.assert_allclose(dx, x.grad.numpy(), atol=1e-12)
    np.testing.assert_allclose(dw, w.grad.numpy(), atol=1e-12)


@pytest.mark.parametrize("n,L,window,sinks", [(9, 9, 3, 0), (9, 9, 4, 2), (4, 11, 100, 1), (1, 12, 1, 3)])
def test_window_attention(n, L, window, sinks):
    rng = np.random.default_rng(L)
    q, k, v, do = (torch.tensor(rng.standard_normal((r, h, 8)), requires_grad=True)
                   for r, h in ((n, 4), (L, 2), (L, 2), (n, 4)))
    where = torch.zeros(n, L, dtype=torch.bool)
    for i in range(n):
        for j in range(i + L - n + 1):
            where[i, j] = j < sinks or i + L - n - j < window
    kk, vv = (x.repeat_interleave(2, 1) for x in (k, v))
    s = (torch.einsum("ihd,jhd->hij", q, kk) * 0.4).masked_fill(~where, float("-inf"))
    o = torch.einsum("hij,jhd->ihd", s.softmax(-1), vv)
    o.backward(do.detach())
    args = [x.detach().numpy() for x in (q, k, v)]
    O, lse = layer.window_attention(*args, window, sinks, 0.4)
    np.testing.assert_allclose(O, o.detach().numpy(), atol=1e-12)
    np.testing.assert_allclose(lse, s.logsumexp(-1).detach().numpy(), atol=1e-12)
    for g, x in zip(layer.window_attention_bwd(*args, do.detach().numpy(), window, sinks, 0.4), (q, k, v)):
        np.testing.assert_allclose(g, x.grad.numpy(), atol=1e-12)
