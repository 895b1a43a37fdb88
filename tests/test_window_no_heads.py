"""Window attention's gradient without query heads: kv heads' gradients are not left unwritten (no GPU:
the C entry points return before any CUDA call)."""
import online_softmax_06_gb300 as fa

P = 0x1000   # an address that nothing reads


def bwd(**kw):
    a = dict(q=P, qs=0, k=P, ks=256, v=P, vs=256, o=P, do=P, lse=P, dq=P, dqs=0, dk=P, dks=256, dv=P, dvs=256, B=2,
             N=40, total=80, H=0, Hkv=2, d=128, scale=0.1, window=8, sinks=2, cu=None, ws=P, n=1 << 30)
    a.update(kw)
    return fa.fa_attention_window_bwd(*a.values())


def test_no_query_heads():
    fa.build()
    assert bwd() == fa.FA_ERR_BAD_SIZE
    assert bwd(cu=P) == fa.FA_ERR_BAD_SIZE
    assert bwd(Hkv=0) == fa.FA_OK                       # nothing to write
    for rows in (dict(B=0, total=0), dict(N=0, total=0), dict(total=0, cu=P)):
        assert bwd(**rows) == fa.FA_OK
