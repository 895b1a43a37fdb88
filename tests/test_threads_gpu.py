"""Calls from a host thread that has made no CUDA call before, as a training framework's gradients do."""
import threading

import pytest
import torch

import online_softmax_06_gb300 as fa
from gpu_common import device_error_clear, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def calls(q, k):
    pos = torch.arange(q.shape[0] * q.shape[1], dtype=torch.int32, device="cuda").view(q.shape[:2])
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    o, lse = fa.attention_window_fwd(q, k, k, 50, 4)
    of, lf = fa.attention_fwd(q, q, q, causal=True)
    return {
        "window": lambda: (o, lse), "window_new": lambda: fa.attention_window_fwd(q, k, k, 50, 4),
        "window_few": lambda: fa.attention_window_fwd(q[:, :1].contiguous(), k, k, 50, 4),
        "window_bwd": lambda: fa.attention_window_bwd(q, k, k, o, q, lse, 50, 4),
        "rope": lambda: fa.qk_norm_rope_fwd(q, k, None, None, f, pos),
        "rope_bwd": lambda: fa.qk_norm_rope_bwd(q, k, q, k, None, None, f, pos)[:2],
        "fwd": lambda: fa.attention_fwd(q, q, q, causal=True),
        "bwd": lambda: fa.attention_bwd(q, q, q, of, q, lf, causal=True),
    }


@pytest.mark.parametrize("name", ["window_new", "window_few", "window_bwd", "rope", "rope_bwd", "fwd", "bwd"])
def test_first_call_of_a_thread(name):
    gen = torch.Generator("cuda").manual_seed(5)
    q = torch.randn(2, 300, 4, 64, generator=gen, device="cuda").bfloat16()
    k = torch.randn(2, 300, 2, 64, generator=gen, device="cuda").bfloat16()
    call = calls(q, k)[name]
    want = call()
    got = []

    def work():
        try:
            got.append(call())
        except Exception as e:                       # handed to the test's own thread
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not isinstance(got[0], Exception), got[0]
    torch.cuda.synchronize()
    device_error_clear()
    assert all(torch.equal(a, b) for a, b in zip(want, got[0]))
