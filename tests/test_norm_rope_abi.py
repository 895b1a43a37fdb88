"""Refusals of the norm and rotation's C entry points: all return before any CUDA call (no GPU)."""
import pytest

import online_softmax_06_gb300 as fa

P = 0x1000   # an address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()


def fwd(**kw):
    a = dict(q=P, qs=256, k=P, ks=128, wq=P, wk=P, f=P, pos=P, qo=P, qos=256, ko=P, kos=128, total=4, H=2, Hkv=1, d=128,
             rot=128, inter=0, eps=1e-6)
    a.update(kw)
    return fa.fa_qk_norm_rope_fwd(*a.values())


def bwd(**kw):
    a = dict(q=P, qs=256, k=P, ks=128, gq=P, gqs=256, gk=P, gks=128, wq=P, wk=P, f=P, pos=P, dq=P, dqs=256, dk=P,
             dks=128, dwq=P, dwk=P, total=4, H=2, Hkv=1, d=128, rot=128, inter=0, eps=1e-6, ws=P, n=1 << 20)
    a.update(kw)
    return fa.fa_qk_norm_rope_bwd(*a.values())


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(call):
    assert call(total=-1) == fa.FA_ERR_BAD_SIZE
    assert call(H=-1) == fa.FA_ERR_BAD_SIZE
    assert call(rot=136) == fa.FA_ERR_BAD_SIZE
    assert call(rot=-8) == fa.FA_ERR_BAD_SIZE
    assert call(rot=12) == fa.FA_ERR_UNSUPPORTED
    assert call(d=96, rot=0) == fa.FA_ERR_UNSUPPORTED
    assert call(eps=-1.0) == fa.FA_ERR_BAD_SIZE
    assert call(eps=float("nan")) == fa.FA_ERR_BAD_SIZE
    assert call(q=None) == fa.FA_ERR_NULL_POINTER
    assert call(k=None) == fa.FA_ERR_NULL_POINTER
    assert call(pos=None) == fa.FA_ERR_NULL_POINTER
    assert call(f=None) == fa.FA_ERR_NULL_POINTER
    assert call(qs=128) == fa.FA_ERR_BAD_SIZE
    assert call(ks=132) == fa.FA_ERR_MISALIGNED
    assert call(q=P + 8) == fa.FA_ERR_MISALIGNED
    assert call(f=P + 4) == fa.FA_ERR_MISALIGNED
    assert call(pos=P + 2) == fa.FA_ERR_MISALIGNED
    assert call(total=1 << 31) == fa.FA_ERR_TOO_LARGE
    assert call(qs=1 << 32) == fa.FA_ERR_TOO_LARGE


def test_forward_only():
    assert fwd(qo=None) == fa.FA_ERR_NULL_POINTER
    assert fwd(kos=64) == fa.FA_ERR_BAD_SIZE
    assert fwd(total=0, q=None) == fa.FA_OK
    assert fwd(H=0, Hkv=0) == fa.FA_OK


def test_gradient_only():
    assert bwd(gq=None) == fa.FA_ERR_NULL_POINTER
    assert bwd(gqs=248) == fa.FA_ERR_BAD_SIZE
    assert bwd(dks=129) == fa.FA_ERR_MISALIGNED
    assert bwd(ws=None) == fa.FA_ERR_NULL_POINTER
    assert bwd(ws=P + 128) == fa.FA_ERR_MISALIGNED
    assert bwd(n=100) == fa.FA_ERR_BAD_SIZE
    assert bwd(total=0, dwq=None, dwk=None) == fa.FA_OK
    assert fa.fa_qk_norm_rope_bwd_workspace_bytes(-1, 1, 1, 64) == fa.FA_ERR_BAD_SIZE
    assert fa.fa_qk_norm_rope_bwd_workspace_bytes(1, 1, 1, 80) == fa.FA_ERR_UNSUPPORTED
    assert fa.fa_qk_norm_rope_bwd_workspace_bytes(0, 1, 1, 64) == 0
