"""Window attention over packed rows of which most lie behind the last sequence (GB300)."""
import numpy as np
import pytest
import torch

import online_softmax_06_gb300 as fa
from gpu_common import device_error_clear, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,spare,most", [([60] * 400 + [3], 100000, 300), ([300, 1, 299] * 40, 30000, 300),
                                             ([0] * 500 + [1], 60000, 257)])
def test_rows_behind_change_nothing(lens, spare, most, d):
    H, Hkv, T, window, sinks = 4, 2, sum(lens), 50, 2
    gen = torch.Generator("cuda").manual_seed(T)
    make = lambda h: torch.randn(T, h, d, generator=gen, device="cuda").bfloat16()  # noqa: E731
    rows = [make(h) for h in (H, Hkv, Hkv, H)]
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")

    def step(q, k, v, do, out):
        o, lse = fa.attention_window_fwd(q, k, v, window, sinks, cu_seqlens_q=cu, cu_seqlens_k=cu, max_q=most, max_k=most)
        return (o, lse, *fa.attention_window_bwd(q, k, v, o, do, lse, window, sinks, cu_seqlens=cu, max_seqlen=most,
                                                 dq=out[0], dk=out[1], dv=out[2]))

    want = step(*rows, [torch.empty_like(x) for x in rows[:3]])
    more = [torch.cat((x, torch.full((spare, *x.shape[1:]), float("nan"), dtype=x.dtype, device="cuda"))) for x in rows]
    got = step(*more, [torch.full_like(x, 7.0) for x in more[:3]])
    device_error_clear()
    for i, (x, y) in enumerate(zip(got, want)):
        assert torch.equal(x[:, :T] if i == 1 else x[:T], y)
    assert all((x[T:] == 7).all() for x in got[2:])
