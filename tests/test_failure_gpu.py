"""Failure detection on the GPU without a fault: a bounded wait that runs out.

Every mbarrier wait of the attention kernels is bounded.  A wait that gives up
sets FA_DEVERR_WAIT_TIMEOUT in the device error word and raises the CTA's abort
flag; the other roles then leave their loops, the copies and tensor-core work
already issued are waited for, tensor memory is freed, and the CTA exits.
fa_debug_expire_next_wait makes one launch wait, with a short bound, on a
barrier that nothing arrives at (a flag nothing sets), so that this path runs
for real; the test checks the error word, that the context is still usable
and that the next call on the same stream matches the oracle.
"""
import math
import time

import numpy as np
import pytest
import torch

import online_softmax_06_gb300 as fa
import oracle
import workloads
from kv4_common import Pool, bf16_rows, gpu_bf16, gpu_i32, kv4
from gpu_common import ATTN_BF16_LSE_TOL, ATTN_BF16_O_TOL, max_abs, require_gpu
from test_kv4_attention_gpu import params

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


@pytest.mark.parametrize("N,d,causal", [(256, 128, True), (300, 64, False), (1000, 128, True)])
def test_expired_wait_is_reported_and_the_next_call_is_correct(dev, N, d, causal):
    B, H = 2, 3
    Q, K, V = workloads.attention_inputs((B, N, H, d), seed=N + d)
    q, k, v = (t.to(dev) for t in (Q, K, V))
    stream = torch.cuda.current_stream(dev)
    fa.fa_set_stream(stream.cuda_stream)
    assert fa.fa_get_device_error() == 0
    o = torch.full_like(q, 3.0)
    lse = torch.full((B, H, N), 3.0, dtype=torch.float32, device=dev)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d,
            1 / math.sqrt(d), int(causal), None)
    assert fa.fa_debug_expire_next_wait(20_000) == 0          # 20 us
    t0 = time.perf_counter()
    assert fa.fa_attention_fwd(*args) == 0
    torch.cuda.synchronize(dev)
    elapsed = time.perf_counter() - t0
    assert fa.fa_get_device_error() == fa.FA_DEVERR_WAIT_TIMEOUT
    assert fa.fa_get_device_error() == 0                       # read and cleared
    # the aborted launch wrote nothing and ended well before any 2 s bound
    assert bool((o == 3.0).all()) and bool((lse == 3.0).all())
    assert elapsed < 1.5, elapsed
    # the switch was one-shot: the next call on the same stream runs normally
    assert fa.fa_attention_fwd(*args) == 0
    torch.cuda.synchronize(dev)
    assert fa.fa_get_device_error() == 0
    Or, lr = oracle.attention_dense(Q.float().numpy(), K.float().numpy(), V.float().numpy(),
                                    1 / math.sqrt(d), causal)
    assert max_abs(o.float().cpu().numpy(), Or) <= ATTN_BF16_O_TOL
    assert max_abs(lse.cpu().numpy(), lr) <= ATTN_BF16_LSE_TOL


BWD_TOL = 2.0 ** -6          # the one-pass backward's parity bound (normwise)


def _normwise(g, ref):
    return float(np.abs(g - ref).max() / max(np.abs(ref).max(), 1e-3))


@pytest.mark.parametrize("packed,lens,d,causal", [
    (False, (256, 256), 128, True),       # dense B=2: two or four 64-query steps per CTA
    (False, (300, 300), 64, False),       # dense B=2, d = 64 (zero rows of K^T)
    (False, (1000, 1000), 128, True),     # dense B=2: up to 16 steps, the 3-stage ring wraps
    (True, (1, 129, 700, 0, 64), 128, True),   # packed: ragged, one token, an empty sequence
])
def test_expired_wait_in_one_pass_backward(dev, packed, lens, d, causal):
    """The same switch on the one-pass backward: its tensor-core warp gives up,
    the row warps and the copy warp leave their loops, dK and dV stay
    unwritten, dQ is converted from an accumulator that received nothing
    (zero), and the next call matches the oracle."""
    H = 3
    B, N = len(lens), max(lens)
    cu = workloads.cu_seqlens_of(lens)
    total = int(cu[-1])
    shape = (total, H, d) if packed else (B, N, H, d)
    Q, K, V = workloads.attention_inputs(shape, seed=7 * N + d)
    dO = workloads.attention_inputs(shape, seed=7 * N + d + 1)[0]
    q, k, v, do = (t.to(dev) for t in (Q, K, V, dO))
    stream = torch.cuda.current_stream(dev)
    fa.fa_set_stream(stream.cuda_stream)
    cu_d = torch.from_numpy(cu).to(dev) if packed else None
    if packed:
        o, lse = fa.attention_fwd(q, k, v, causal=causal, cu_seqlens=cu_d, max_seqlen=N)
        nbytes = fa.fa_attention_bwd_atomic_varlen_workspace_bytes(B, H, N, total, d)
        lse_shape = (H, total)
    else:
        o, lse = fa.attention_fwd(q, k, v, causal=causal)
        nbytes = fa.fa_attention_bwd_atomic_workspace_bytes(B, H, N, d)
        lse_shape = (B, H, N)
    torch.cuda.synchronize(dev)
    assert nbytes > 0 and fa.fa_get_device_error() == 0
    ws = torch.empty(nbytes // 4, dtype=torch.float32, device=dev)
    d_buf = torch.empty(lse_shape, dtype=torch.float32, device=dev)
    dq, dk, dv = (torch.full_like(q, 3.0) for _ in range(3))
    ptrs = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
            lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), d_buf.data_ptr())

    def call():
        if packed:
            return fa.fa_attention_bwd_atomic_varlen(*ptrs, B, H, N, total, d, 1 / math.sqrt(d),
                                                     int(causal), cu_d.data_ptr(),
                                                     ws.data_ptr(), nbytes)
        return fa.fa_attention_bwd_atomic(*ptrs, B, H, N, d, 1 / math.sqrt(d), int(causal),
                                          ws.data_ptr(), nbytes)

    assert fa.fa_debug_expire_next_wait(20_000) == 0          # 20 us
    t0 = time.perf_counter()
    assert call() == 0
    torch.cuda.synchronize(dev)
    elapsed = time.perf_counter() - t0
    assert fa.fa_get_device_error() == fa.FA_DEVERR_WAIT_TIMEOUT
    assert fa.fa_get_device_error() == 0                       # read and cleared
    assert bool((dk == 3.0).all()) and bool((dv == 3.0).all())
    assert bool((dq == 0.0).all())
    assert elapsed < 1.5, elapsed
    # one-shot: the next call on the same stream runs normally
    assert call() == 0
    torch.cuda.synchronize(dev)
    assert fa.fa_get_device_error() == 0
    args = [t.float().numpy() for t in (Q, K, V, dO)]
    if packed:
        ref = oracle.attention_bwd_packed(*args, cu, 1 / math.sqrt(d), causal)
    else:
        ref = oracle.attention_bwd(*args, 1 / math.sqrt(d), causal)
    for name, g in (("dQ", dq), ("dK", dk), ("dV", dv)):
        e = _normwise(g.float().cpu().numpy(), ref[name])
        assert e <= BWD_TOL, f"{name}: {e}"


def _kv4_expired(lens, nq, H, Hkv, d, form, max_seqlen=None):
    """One call with a wait that runs out, then one without: (rows written right, rows
    untouched) of the first as masks [total, H], having checked both against the oracle."""
    rng = np.random.default_rng(sum(lens) + nq)
    pool = Pool(lens, Hkv, d, 64, 32, seed=7)
    pool.fill([bf16_rows(rng, n, Hkv, d) for n in lens], [bf16_rows(rng, n, Hkv, d) for n in lens])
    q = [bf16_rows(rng, nq, H, d) for _ in lens]
    x, cache, table = gpu_bf16(np.stack(q)), torch.from_numpy(pool.bytes).cuda(), gpu_i32(pool.table)
    o = torch.full_like(x, 3.0)
    lse = torch.full((len(lens), H, nq), 3.0, device="cuda")
    # the workspace holds what an earlier call may have left: parts that would count
    ws = torch.full((fa.fa_attention_kv4_workspace_bytes(len(lens), nq, len(lens) * nq, max_seqlen, H,
                                                         Hkv, d),), 0x3f, dtype=torch.uint8, device="cuda")
    call = lambda: fa.attention_kv4(x, cache, table, gpu_i32(lens), max_seqlen=max_seqlen,  # noqa: E731
                                    out=o, lse=lse, workspace=ws)
    assert fa.fa_get_device_error() == 0
    assert fa.fa_debug_expire_next_wait(20_000) == 0
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert fa.fa_get_device_error() == fa.FA_DEVERR_WAIT_TIMEOUT
    assert fa.fa_get_device_error() == 0
    assert elapsed < 1.5, elapsed
    # the tolerances of the cache's own tests, with the largest of all sequences
    ref = [kv4.attention(y, *pool.rows(b), 1 / math.sqrt(d), True) for b, y in enumerate(q)]
    Or, lr = np.concatenate([r[0] for r in ref]), np.concatenate([r[1].T for r in ref])
    par = [params(pool, b) for b in range(len(lens))]
    s_v, v_max = max(p[1] for p in par), max(p[2] for p in par)
    dots = lambda ks: max(float((np.abs(y[:, h]) @ np.abs(k[:, h // (H // Hkv)]).T).max())  # noqa: E731
                          for y, k in zip(q, ks) for h in range(H)) / math.sqrt(d)
    eS = dots([p[0] for p in par]) * 2.0 ** -19
    if form == "many":
        eS += dots([pool.rows(b)[0] for b in range(len(lens))]) * 2.0 ** -11
    tol = 4 * eS * v_max + 2.0 ** -8 * np.abs(Or) + 2.0 ** -10 * (v_max if form == "many" else 15 * s_v)
    tol_l = 2 * eS + 2.0 ** -20 + 2.0 ** -22 * np.abs(lr)

    def right():
        oo = o.double().cpu().numpy().reshape(-1, H, d)
        ll = lse.transpose(1, 2).reshape(-1, H).double().cpu().numpy()
        return oo, ll, (np.abs(oo - Or) <= tol).all(-1) & (np.abs(ll - lr) <= tol_l)

    oo, ll, good = right()
    stay = (oo == 3.0).all(-1) & (ll == 3.0)
    call()
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == 0
    assert right()[2].all()
    return good, stay


@pytest.mark.parametrize("lens,nq,H,Hkv,d", [
    ([30000], 1, 8, 2, 64),               # two items over all ranges, joined from many parts
    ([9000, 40, 5000, 700], 2, 4, 2, 128),
    ([1000, 33, 600], 1, 4, 2, 64),       # heads whole, no join
])
def test_expired_wait_in_cache_attention(dev, lens, nq, H, Hkv, d):
    """Few query rows: no item with a part in the range of the warp that gave up is
    written, whatever the parts' memory held; the rest is right."""
    bound = max(lens)
    good, stay = _kv4_expired(lens, nq, H, Hkv, d, "few", bound)
    assert (good | stay).all()
    assert stay.any()
    # rows of a (sequence, kv head) item go together
    for b in range(len(lens)):
        for h in range(Hkv):
            rows, heads = slice(b * nq, (b + 1) * nq), slice(h * H // Hkv, (h + 1) * H // Hkv)
            assert len(set(stay[rows, heads].flatten())) == 1
    if len(lens) > 1:
        assert good.any()


@pytest.mark.parametrize("lens", [[2300, 4500], [513, 700]], ids=["ranges", "whole"])
def test_expired_wait_in_cache_attention_many_rows(dev, lens):
    """Many query rows: the 256 rows of the CTA whose wait ran out (those of the longest
    sequence's first head) stay, with one range of keys or several; the rest is right."""
    good, stay = _kv4_expired(lens, 300, 16, 16, 64, "many", max(lens))
    want = np.zeros_like(stay)
    want[300:556, 0] = True
    assert np.array_equal(stay, want)
    assert good[~want].all()
