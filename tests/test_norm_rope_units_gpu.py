"""Norm and rotation where a token's passes are cut into a few units of several passes each, the last
one short, one of them from Q's heads into K's (GB300).

A warp's pass takes 4 rows a lane forward and 2 backward, 32 * 8 / d lanes' rows at once; a unit has
ceil(tokens * passes / 4864) passes.  1000 tokens of 32 + 8 heads of 128: 10 passes backward in units of 3;
2500: 5 passes forward in units of 3, backward of 6; 40 + 10 heads of 64, 1500 tokens: 7 passes backward, of 3."""
import pytest
import torch

import online_softmax_06_gb300 as fa
import test_norm_rope_gpu as whole
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

CASES = [(T, H, Hkv, d, rot, inter, 100000) for T, H, Hkv, d, rot in (
    (1000, 32, 8, 128, 128), (2500, 32, 8, 128, 64), (1500, 40, 10, 64, 64), (2499, 31, 9, 128, 128))
    for inter in (False, True)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    whole.test_forward(case, True)


@pytest.mark.parametrize("case", CASES)
def test_gradient(case):
    whole.test_gradient(case)


@pytest.mark.parametrize("case", CASES)
def test_in_place(case):
    T, H, Hkv, d, rot, inter, far = case
    rng, q, k, w, pos = whole.inputs(case, 3)
    args = (w[0].cuda(), w[1].cuda(), whole.freqs(rot), pos.cuda())
    x, y = torch.cat((q, k), 1).cuda(), torch.randn(T, H + Hkv, d).bfloat16().cuda()
    want = fa.qk_norm_rope_fwd(q.cuda(), k.cuda(), *args, interleaved=inter)
    back = fa.qk_norm_rope_bwd(q.cuda(), k.cuda(), y[:, :H].contiguous(), y[:, H:].contiguous(), *args, interleaved=inter)
    got = fa.qk_norm_rope_bwd(x[:, :H], x[:, H:], y[:, :H], y[:, H:], *args, interleaved=inter, dq=y[:, :H], dk=y[:, H:])
    assert all(torch.equal(a, b) for a, b in zip(back, got))
    got = fa.qk_norm_rope_fwd(x[:, :H], x[:, H:], *args, interleaved=inter, q_out=x[:, :H], k_out=x[:, H:])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
