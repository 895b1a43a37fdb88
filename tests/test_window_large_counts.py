"""Window attention: windows, sinks and bounds of lengths that do not fit 32 bits."""
import pytest
import torch

import online_softmax_06_gb300 as fa
from gpu_common import device_error_clear, require_gpu

ALL = [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 8, 2 ** 40]


@pytest.mark.parametrize("n", ALL)
def test_workspace(n):
    fa.build()
    size = lambda window, sinks: fa.fa_attention_window_bwd_workspace_bytes(2, 1000, 2000, 4, 2, 64, window, sinks)  # noqa: E731
    assert size(n, 4) == size(1000, 4) != size(8, 4)
    assert size(8, n) == size(8, 1000) != size(8, 4)
    assert size(-n, 0) == size(8, -n) == fa.FA_ERR_BAD_SIZE
    assert size(8 - 2 ** 32, 0) == fa.FA_ERR_BAD_SIZE


def args(nq, N=300):
    gen = torch.Generator("cuda").manual_seed(nq)
    make = lambda n, h: torch.randn(1, n, h, 64, generator=gen, device="cuda").bfloat16()  # noqa: E731
    return make(nq, 4), make(N, 2), make(N, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("nq", [1, 300])
@pytest.mark.parametrize("n", ALL)
def test_forward(n, nq):
    require_gpu()
    q, k, v = args(nq)
    o, lse = fa.attention_window_fwd(q, k, v, 300)
    for window, sinks in ((n, 0), (n, n), (5, n)):
        got = fa.attention_window_fwd(q, k, v, window, sinks)
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
    for window, sinks in ((8 - 2 ** 32, 0), (8, 8 - 2 ** 32)):
        with pytest.raises(fa.FaError):
            fa.attention_window_fwd(q, k, v, window, sinks)
    device_error_clear()


@pytest.mark.gpu
@pytest.mark.parametrize("n", ALL)
def test_gradient(n):
    require_gpu()
    q, k, v = args(300)
    o, lse = fa.attention_window_fwd(q, k, v, 300)
    do = torch.randn(o.shape, device="cuda").bfloat16()
    want = fa.attention_window_bwd(q, k, v, o, do, lse, 300)
    for window, sinks in ((n, 0), (n, n), (5, n)):
        got = fa.attention_window_bwd(q, k, v, o, do, lse, window, sinks)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    with pytest.raises(fa.FaError):
        fa.attention_window_bwd(q, k, v, o, do, lse, 8 - 2 ** 32)
    device_error_clear()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 300, -1])
def test_bounds_of_lengths(n):
    require_gpu()
    q, k, v = (x[0] for x in args(300))
    cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    for bad in (dict(max_q=n), dict(max_k=n)):
        with pytest.raises(ValueError):
            fa.attention_window_fwd(q, k, v, 8, cu_seqlens_q=cu, cu_seqlens_k=cu, **bad)
    o, lse = fa.attention_window_fwd(q, k, v, 8, cu_seqlens_q=cu, cu_seqlens_k=cu)
    with pytest.raises(ValueError):
        fa.attention_window_bwd(q, k, v, o, o, lse, 8, cu_seqlens=cu, max_seqlen=n)
