// attn_window_bwd.cu -- gradients of the window attention (dQ, dK, dV) on the
// sm_103a tensor cores.
//
// With P = exp(scale Q K^T - lse) at the seen keys, formed again tile by tile, and
// D_i = dO_i . O_i:
//     dV = P^T dO,  dS = P o (dO V^T - D),  dQ = scale dS K,  dK = scale dS^T Q,
// dK and dV summed over the G query heads that share a kv head.  Two kernels as in
// attn_bwd.cu, whose roles, tensor memory and order of products they have, and no
// atomics; then, where sinks are seen from outside their tile's window, a third:
//   * attn_window_dq_kernel: an item per (sequence, kv head, 128 rows: queries x G
//     heads), the keys that they see in 128-key steps, the window's behind the
//     sinks' as in the forward (window.cuh).  Also writes D.  D comes from O rounded
//     to bf16, an error e that all keys of a row share: dQ is off by e sum_j P_ij K_j,
//     which grows against dQ where a row's keys have a part in common (2^-9 of dQ
//     becomes 2^-7.5 with a window of 2048, 2^-3.4 with keys and values whose common
//     parts are twice the rest).  But sum_j dS_ij is 0, so its computed value r_i, of dS as
//     rounded, is the errors' sum, and r_i sum_j P_ij K_j, a fourth product, is taken off:
//     each key by its own weight, so that dQ depends on no key that the row does not see.
//     D_i + r_i is what dK takes.
//   * attn_window_dkdv_kernel: a CTA per (sequence, kv head, 128 keys); 128-query
//     steps over the queries that have these keys in their window, one head of the
//     group after the other into the same accumulators.  Keys below `sinks` are seen
//     by all later queries too: these steps, of which a long sequence has many more
//     than a window, go to CTAs of their own in pieces as long as a window's, and
//     all pieces of such a tile write fp32 parts.
//   * attn_window_join_kernel adds a tile's parts in order.
// P and dS are rounded to bf16 (2^-9 relative each) as operands; all sums are fp32.
// Rows behind a sequence's end (the next sequence, room at the end of the batch) are
// zeroed in shared memory before a product sums over them: their P is 0, but they may
// hold NaN.  Every wait is bounded; a timed-out one leaves its CTA's rows unwritten.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fa.h"
#include "fa_error.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "window.cuh"

namespace fa {
namespace {

constexpr int BT = 128;                     // rows of a tile, resident or streamed
constexpr int kPad = 32;                    // sinks fill whole pieces of a tile
constexpr int kRowWarps = 16;               // four threads a row: see the kernels
constexpr int kThreads = 32 * (kRowWarps + 2);
constexpr int kWarpLoad = kRowWarps, kWarpMma = kRowWarps + 1;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kChunkBytes = BT * 128;     // 128 rows of 64 bf16
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
    CUtensorMap tm_o;                  // dQ: as tm_q
    CUtensorMap tm_d0, tm_d1;          // outputs: dQ as tm_q; or dV and dK as tm_k
    CUtensorMap tm_q, tm_do;           // dQ: P rows of G heads, q_chunks chunks a copy; dK/dV:
                                       // 128 rows of a head
    CUtensorMap tm_k, tm_v;            // 128 rows of a head
    CUtensorMap tm_k32, tm_v32;        // dQ: 32 rows, a chunk a copy
    WindowArgs a;                      // O read; queries and keys are the same tokens
    float *D;                          // as lse
    __nv_bfloat16 *dQ, *dK, *dV;
    int64_t dq_stride, dk_stride, dv_stride;
    float *parts;                      // [places][Hkv][sink tiles][dV, dK][128][d]
    WindowCut part_cut;                // places of packed sequences (div 0: b * slots)
    int far_items;                     // CTAs for them
    int q_chunks;
    uint32_t div_g;                    // r / G = r * div_g >> 16 for r < 128
    int G, P;
    WindowGrid grid;                   // of P queries (dQ), of 128 keys (dK/dV)
    int sink_tiles, slots, piece;      // piece: 128-query tiles of a far piece
    float scale_log2;
};

// A row warp's wait: one lane polls and shares the outcome.
__device__ __forceinline__ bool row_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                         int *err_word)
{
    int ok = 1;
    if ((threadIdx.x & 31) == 0)
        ok = ptx::mbar_poll(bar, parity, abort, err_word) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    return ok != 0;
}

// Rows [r0, rows) of a tile of 64-value chunks (`stride` bytes apart) cleared by a warp.
template <int CHUNKS>
__device__ __forceinline__ void clear_rows(uint8_t *tile, int r0, int rows, uint32_t stride)
{
    const int lane = threadIdx.x & 31;
    for (int r = (r0 > 0 ? r0 : 0) + (lane >> 3); r < rows; r += 4)
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
            *reinterpret_cast<uint4 *>(tile + c * stride + r * 128 + (lane & 7) * 16) =
                make_uint4(0, 0, 0, 0);
}

// Shared-memory descriptor offset of K step kk (16 bf16) in a K-major tile.
__device__ __forceinline__ uint64_t kmajor_off(int kk, uint32_t chunk_bytes)
{
    return uint64_t(((kk >> 2) * chunk_bytes + (kk & 3) * 32) >> 4);
}

// Columns [32 c0, 32 c1) of this thread's row r of an accumulator (TWO: plus `more` times
// those of the one at t_more), times `mul`, as bf16: to `dst` (the row's first value; null:
// nowhere), or into a tile in shared memory laid out as a copy's (128-byte swizzle).
template <bool TWO = false>
__device__ __forceinline__ void store_row(uint32_t t_acc, float mul, __nv_bfloat16 *dst,
                                          uint8_t *tile, int r, int c0, int c1, float more = 0.f,
                                          uint32_t t_more = 0)
{
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
        uint32_t o[32];
        ptx::tmem_ld32(t_acc + c * 32, o);
        if constexpr (TWO) {
            uint32_t x[32];
            ptx::tmem_ld32(t_more + c * 32, x);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
                o[e] = __float_as_uint(fmaf(more, __uint_as_float(x[e]), __uint_as_float(o[e])));
        } else {
            ptx::tmem_wait_ld();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                u[e] = ptx::pack_bf16x2(__uint_as_float(o[8 * q + 2 * e]) * mul,
                                        __uint_as_float(o[8 * q + 2 * e + 1]) * mul);
            const uint4 v = make_uint4(u[0], u[1], u[2], u[3]);
            if (tile != nullptr) {
                const int un = (c & 1) * 4 + q;
                *reinterpret_cast<uint4 *>(tile + (c >> 1) * kChunkBytes + r * 128 +
                                           ((un ^ (r & 7)) << 4)) = v;
            } else if (dst != nullptr) {
                *reinterpret_cast<uint4 *>(dst + c * 32 + q * 8) = v;
            }
        }
    }
}

// Index of the row statistic (lse, D) of a sequence's first query, head h.
__device__ __forceinline__ int64_t stat_row(const WindowArgs &a, int b, int h, int64_t q0)
{
    return a.cu_seqlens_q != nullptr ? int64_t(h) * a.total_q + q0
                                     : (int64_t(b) * a.H + h) * a.Nq;
}

// =============================================================================
// dQ and D
// =============================================================================
// S_j (P_j packed into it) in columns [0, 128), dP_j (dS_j packed into it) in [128, 256),
// dS K from 256, P K behind it.  The MMA warp issues, per 128-key step j: P_j K_j once the
// rows have stored P_j, S_{j+1}, dS_j K_j once they have stored dS_j, then dP_{j+1}; sixteen
// row warps (four threads a row, 32 columns each) form P while dS K and dP run and dS while
// P K and S do.  A step takes 1.6 us (d = 128), its products 1.1: dS_j -> dQ_j -> dP_{j+1}
// -> dS_{j+1} is a chain.  With d = 64 there are columns for a second dP behind the
// accumulators (384), and dP_{j+1} goes ahead of dQ_j.
// A CTA, one an SM, does items one after the other, its own and then such as have not begun
// (it asks for their CTAs): Q and dO of the next come while this one's last step runs, and
// its first products run while the rows store this one's dQ.  2 x 4096, 32 heads on 8,
// d = 128, window 1024: 232 us; 1 x 32768, 16 heads on 4, window 2048: 800 us; 8 packed
// sequences of 3001 tokens at most, 16 heads, d = 64, window 256: 95 us.  (Without P K 180,
// 611 and 87 us, but dQ off by 0.0043 and 0.0050 of its norm for the first two's windows,
// keys with a common part as large as the rest and values with a tenth, where it is off by
// 0.0024 so; D from a pass over the keys before would be two products more, not one.)
template <int D>
struct CfgQ {
    static constexpr int kChunks = D / 64;
    static constexpr uint32_t kTileBytes = BT * D * 2;
    static constexpr uint32_t kStageBytes = 2 * kTileBytes;  // Q and dO, or K_j and V_j
    static constexpr int kStages = 3;
    // O's rows, where there is room two items', and dQ's on their way out
    static constexpr int kOBufs = D == 64 ? 2 : 1;
    static constexpr uint32_t kOffO = kStages * kStageBytes;
    static constexpr uint32_t kOffOut = kOffO + (kOBufs == 2 ? 2 : 0) * kTileBytes;
    // parts of D_i, and of the sums of dS, of the rows' four threads; items
    static constexpr uint32_t kOffXch = kOffOut + kTileBytes;
    static constexpr uint32_t kOffSum = kOffXch + (kOBufs == 2 ? 4 * BT * 4 : 0);
    static constexpr uint32_t kOffItem = kOffSum + 4 * BT * 4;
    static constexpr uint32_t kOffNext = kOffItem + 2 * 40;
    static constexpr uint32_t kOffBar = kOffNext + 16;
    // of dP and dS: where there are columns for two, dP_{j+1} need not wait for dQ_j
    static constexpr int kDPs = D == 64 ? 2 : 1;
    static __device__ __forceinline__ uint32_t col_dp(uint32_t step)
    {
        return kDPs == 2 && (step & 1u) ? 256 + 2 * D : 128;
    }
    static constexpr int kBars = 2 * kStages + kOBufs + kDPs + 10;
    static constexpr uint32_t kSmemBytes = kOffBar + 8 * kBars + 16;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};
// The stages of the ring, as all warps of a CTA number them: an item's Q and dO hold one,
// its steps' keys take the other two in turn.  The next item's Q and dO come where the
// step before the last was, which is free first.
struct DqRing {
    int hold = 0, a = 1, b = 2;
    __device__ __forceinline__ int of(int step) const { return step & 1 ? b : a; }
    __device__ __forceinline__ void next(int steps)
    {
        const int last = of(steps - 1), other = a + b - last;
        a = hold;
        hold = other;
        b = last;
    }
};
constexpr uint32_t kColAcc = 256, kColDP = 128;
// Column of the packed bf16 operand for the product's K step kk: the 32 values of each
// 32-column block go to the block's first 16 columns, so a thread only overwrites
// columns that it has read.
__host__ __device__ constexpr uint32_t packed_col(int kk)
{
    return uint32_t(32 * (kk >> 1) + 8 * (kk & 1));
}

// An item of dQ, as the load warp found it.
struct DqItem {
    int done, b, hk, i0, i1, L;
    int64_t q0, k0;
};
static_assert(sizeof(DqItem) == 40, "CfgQ");

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_window_dq_kernel(const __grid_constant__ Params p)
{
    using C = CfgQ<D>;
    constexpr uint32_t kColPK = kColAcc + D;         // P K beside dS K
    static_assert(kColPK + D <= kTmemCols, "tensor memory");
    // aligned as the tiles need it, with no room to align it here
    extern __shared__ __align__(1024) uint8_t smem_aligned[];
    uint8_t *smem = smem_aligned;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *full = bars, *empty = bars + C::kStages, *o_in = bars + 2 * C::kStages;
    uint64_t *s_full = o_in + C::kOBufs, *ds_full = s_full + 1, *p_full = s_full + 2,
             *acc_full = s_full + 3, *drain = s_full + 4, *out_full = s_full + 5,
             *next_in = s_full + 6, *never = s_full + 7, *known = s_full + 8, *dp_full = s_full + 10;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffBar + 8 * C::kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    DqItem *items = reinterpret_cast<DqItem *>(smem + C::kOffItem);

    if (threadIdx.x == 32) {
        ptx::prefetch_tmap(&p.tm_q);
        ptx::prefetch_tmap(&p.tm_do);
        ptx::prefetch_tmap(&p.tm_k);
        ptx::prefetch_tmap(&p.tm_v);
        ptx::prefetch_tmap(&p.tm_k32);
        ptx::prefetch_tmap(&p.tm_v32);
    }
    // nothing that a kernel before may still be writing is read ahead of this
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const WindowArgs &a = p.a;
    window_check(a, p.grid, blockIdx.x);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto keys_of = [&](const DqItem &it) {
        return window_keys(a.window, a.sinks, it.i0, it.i1, 0, kPad);
    };
    auto steps_of = [](const WindowKeys &w) { return (w.places + BT - 1) / BT; };   // at least one
    auto stage_ptr = [&](int st) { return smem + uint32_t(st) * C::kStageBytes; };
    DqRing ring;

    // ---- the load warp's ------------------------------------------------------------
    int o_tiles = 0;
    DqItem item{};
    int asked = 0;                                   // for other CTAs' items
    bool pending = false;
    auto ask = [&]() {
        if (lane == 0) {
            ptx::mbar_arrive_expect_tx(next_in, 16);
            ptx::cta_cancel(smem + C::kOffNext, next_in);
        }
        ++asked;
        pending = true;
        __syncwarp();
    };
    auto find = [&](bool first, DqItem &item) {      // the next item
        for (;; first = false) {
            int64_t idx = blockIdx.x;
            if (!first) {
                if (!pending)
                    ask();
                if (!ptx::mbar_wait_warp(next_in, uint32_t(asked + 1) & 1u, abort_flag, a.err_word))
                    return false;
                idx = ptx::cta_cancelled(smem + C::kOffNext);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                pending = false;
                if (idx < 0)
                    return false;                    // (nor may any be asked for again)
            }
            int tile;
            WindowSeq sq;
            if (!window_item(a, p.grid, unsigned(idx), item.b, item.hk, tile))
                continue;
            if (!window_seq(a, item.b, sq)) {
                if (lane == 0 && tile == 0 && item.hk == 0)
                    record_device_error(a.err_word, FA_DEVERR_BAD_SEQLENS);
                continue;
            }
            item.i0 = tile * p.P;
            if (item.i0 >= sq.L)
                continue;
            item.i1 = min(item.i0 + p.P, sq.L);
            item.L = sq.L;
            item.q0 = sq.q0;
            item.k0 = sq.k0;
            return true;
        }
    };
    // (a slot's copies are issued when the slot is free)
    auto issue_o = [&](int k) {
        if (lane == 0) {
            uint64_t *bar = &o_in[k % C::kOBufs];
            uint8_t *dst = smem + C::kOffO + uint32_t(k % C::kOBufs) * C::kTileBytes;
            ptx::mbar_arrive_expect_tx(bar, C::kChunks * p.P * p.G * 128);
            for (int c = 0; c < C::kChunks; c += p.q_chunks)
                ptx::tma_load_5d(dst + c * kChunkBytes, &p.tm_o, bar, 0, 0, int(item.q0 + item.i0), c,
                                 item.hk);
        }
        o_tiles = k + 1;
        __syncwarp();
    };
    auto tell = [&](int k, const DqItem &it) {
        if (lane == 0) {
            items[k & 1] = it;
            ptx::mbar_arrive(&known[k & 1]);
        }
        __syncwarp();
    };
    auto issue_q = [&](int k) {
        if (lane == 0) {
            uint64_t *bar = &full[ring.hold];
            ptx::mbar_arrive_expect_tx(bar, 2 * C::kChunks * p.P * p.G * 128);
            for (int c = 0; c < C::kChunks; c += p.q_chunks) {
                uint8_t *dst = stage_ptr(ring.hold) + c * kChunkBytes;
                const int row = int(item.q0 + item.i0);
                ptx::tma_load_5d(dst, &p.tm_q, bar, 0, 0, row, c, item.hk);
                ptx::tma_load_5d(dst + C::kTileBytes, &p.tm_do, bar, 0, 0, row, c, item.hk);
            }
        }
        __syncwarp();
        if (C::kOBufs == 2 || k == 0)
            issue_o(k);
    };
    auto issue_keys = [&](const WindowKeys &w, int j) {
        uint64_t *bar = &full[ring.of(j)];
        if (lane == 0)
            ptx::mbar_arrive_expect_tx(bar, C::kStageBytes);
        __syncwarp();
        uint8_t *dst = stage_ptr(ring.of(j));
        const int v0 = j * BT;
        if (v0 < w.sp && v0 + BT > w.sp) {
            // pieces of 32 rows, a lane each
            const int of = lane >> 4, c = lane / (BT / kPad) & 3, q = lane % (BT / kPad);
            const int v = v0 + q * kPad;
            if (c < C::kChunks)
                ptx::tma_load_5d(dst + of * C::kTileBytes + c * kChunkBytes + q * kPad * 128,
                                 of ? &p.tm_v32 : &p.tm_k32, bar, 0, 0,
                                 int(item.k0 + (v < w.sp ? v : w.lo + v - w.sp)), c, item.hk);
        } else if (lane < 2) {
            ptx::tma_load_5d(dst + lane * C::kTileBytes, lane ? &p.tm_v : &p.tm_k, bar, 0, 0,
                             int(item.k0 + (v0 < w.sp ? v0 : w.lo + v0 - w.sp)), 0, item.hk);
        }
        __syncwarp();
    };
    bool more = false;
    if (warp == kWarpLoad) {
        // the barriers, and the first copies while the others set up
        if (lane == 0) {
            for (int st = 0; st < C::kStages; ++st) {
                ptx::mbar_init(&full[st], 1);
                ptx::mbar_init(&empty[st], 1);
            }
            for (int st = 0; st < C::kOBufs; ++st)
                ptx::mbar_init(&o_in[st], 1);
            ptx::mbar_init(s_full, 1);
            for (int st = 0; st < C::kDPs; ++st)
                ptx::mbar_init(&dp_full[st], 1);
            ptx::mbar_init(ds_full, kRowWarps);
            ptx::mbar_init(p_full, kRowWarps);
            ptx::mbar_init(acc_full, 1);
            ptx::mbar_init(drain, 1);
            ptx::mbar_init(&known[0], 1);
            ptx::mbar_init(&known[1], 1);
            ptx::mbar_init(out_full, kRowWarps);
            ptx::mbar_init(next_in, 1);
            ptx::mbar_init(never, 1);
            *abort_flag = 0;
            ptx::fence_barrier_init();
        }
        __syncwarp();
        more = find(true, item);
        item.done = more ? 0 : 1;
        tell(0, item);
    }
    if (warp == kWarpMma) {
        ptx::tmem_alloc(tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    // (the load warp goes on)
    if (warp == kWarpLoad) {
        __threadfence_block();
        asm volatile("bar.arrive 3, %0;" ::"n"(kThreads) : "memory");
    } else {
        ptx::tc_fence_before_sync();
        asm volatile("bar.sync 3, %0;" ::"n"(kThreads) : "memory");
        ptx::tc_fence_after_sync();
    }
    const uint32_t tmem = warp == kWarpLoad ? 0u : *tmem_slot;
    bool aborted = false;

    // Named barriers 1 and 2: the row threads.  At 2, when an item's last step is done, whoever
    // gave up says so, and all leave together.
    constexpr int kRows = 32 * kRowWarps;
    if (warp == kWarpLoad) {
        // ======================= TMA producer =================================
        constexpr int kShort = 4;                    // steps: the answer takes longer than these
        uint32_t used = 0, fills = 0;                // a bit a stage: filled once; fills so far, odd
        auto free_stage = [&](int st) {
            // (the fill before this one is through when its phase of `empty` is)
            if ((used >> st & 1u) && !ptx::mbar_wait_warp(&empty[st], (fills >> st & 1u) ^ 1u,
                                                          abort_flag, a.err_word))
                aborted = true;
            if (!aborted) {
                used |= 1u << st;
                fills ^= 1u << st;
            }
            return !aborted;
        };
        // dQ of item k leaves; where O's place held it, O of the next one comes
        auto hand_over = [&](int k, bool next) {
            if (!ptx::mbar_wait_warp(out_full, uint32_t(k) & 1u, abort_flag, a.err_word)) {
                aborted = true;
                return;
            }
            const DqItem &it = items[k & 1];
            if (lane == 0 && it.i1 - it.i0 == p.P) {
                for (int c = 0; c < C::kChunks; c += p.q_chunks)
                    ptx::tma_store_5d(&p.tm_d0, smem + C::kOffOut + c * kChunkBytes, 0, 0,
                                      int(it.q0 + it.i0), c, it.hk);
                ptx::bulk_commit_and_wait_read();
            }
            __syncwarp();
            if (C::kOBufs == 1 && next)
                issue_o(k + 1);
        };
        DqItem next = item;
        int k = 0;                                   // items begun; all before k - 1 are handed over
        for (; more && !aborted; ++k) {
            const WindowKeys w = keys_of(item);
            const int n_kv = steps_of(w);
            bool found = false;
            if (!free_stage(ring.hold))
                break;
            issue_q(k);
            for (int j = 0;; ++j) {
                const bool begun = j >= min(2, n_kv);
                // (the item before this one ends without these steps' keys)
                if (k > 0 && j == min(2, n_kv))
                    hand_over(k - 1, true);
                if (aborted)
                    break;
                // The next item is asked for late in a long one, so that no CTA holds items that
                // others could have begun (2 x 4096 queries, 32 heads on 8, d = 128, window 4096, all
                // three kernels, when a step had three products: 797 us with each asked for an item
                // ahead, 773 so, 776 four steps before the end); its rows go to L2, a map a lane.
                if (!found && !pending && begun && j >= n_kv - 8)
                    ask();
                if (!found && begun && j >= n_kv - 5) {
                    more = find(false, next);
                    next.done = more ? 0 : 1;
                    tell(k + 1, next);
                    if (more && steps_of(keys_of(next)) <= kShort)
                        ask();
                    if (more && lane < 3)
                        for (int c = 0; c < C::kChunks; c += p.q_chunks)
                            ptx::tma_prefetch_5d(lane == 0 ? &p.tm_q : lane == 1 ? &p.tm_do : &p.tm_o,
                                                 0, 0, int(next.q0 + next.i0), c, next.hk);
                    found = true;
                }
                if (j == n_kv || !free_stage(ring.of(j)))
                    break;
                issue_keys(w, j);
            }
            ring.next(n_kv);
            item = next;
        }
        if (k > 0 && !aborted)
            hand_over(k - 1, false);
        if (*abort_flag && lane == 0) {
            ptx::drain_wait(next_in, uint32_t(asked + 1) & 1u);
            for (int st = 0; st < C::kStages; ++st)
                if (used >> st & 1u)
                    ptx::drain_wait(&full[st], (fills >> st & 1u) ^ 1u);
            for (int n = o_tiles > C::kOBufs ? o_tiles - C::kOBufs : 0; n < o_tiles; ++n)
                ptx::drain_wait(&o_in[n % C::kOBufs], uint32_t(n / C::kOBufs) & 1u);
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        // ======================= MMA issuer (whole warp) =====================
        constexpr uint32_t idesc_s = ptx::idesc_bf16_f32(BT, BT, false);
        constexpr uint32_t idesc_q = ptx::idesc_bf16_f32(BT, D, true);     // B MN-major
        constexpr uint64_t desc_kmajor = ptx::smem_desc_base(16, 1024);
        constexpr uint64_t desc_mnmajor = ptx::smem_desc_base(kChunkBytes, 1024);
        if (a.expire_wait_ns != 0u &&
            !__all_sync(0xffffffffu, ptx::mbar_wait_limited(never, 0, abort_flag, a.err_word,
                                                            a.expire_wait_ns)))
            aborted = true;
        uint32_t phases = 0, g = 0;                  // of the stages, a bit each; steps done
        auto wait_stage = [&](int st) {
            if (!aborted &&
                !ptx::mbar_wait_warp(&full[st], phases >> st & 1u, abort_flag, a.err_word))
                aborted = true;
            phases ^= 1u << st;
            return !aborted;
        };
        for (int k = 0; !aborted; ++k) {
            if (!ptx::mbar_wait_warp(&known[k & 1], uint32_t(k >> 1) & 1u, abort_flag, a.err_word)) {
                aborted = true;
                break;
            }
            if (items[k & 1].done)
                break;
            const int L = items[k & 1].L;
            const WindowKeys wk = keys_of(items[k & 1]);
            const int n_kv = steps_of(wk), end_place = wk.sp + (L - wk.lo);
            // K's and V's rows of step j behind the sequence's end are cleared
            auto clear_tail = [&](int j) {
                const int r0 = end_place - j * BT;
                if (r0 >= BT)
                    return;
                clear_rows<2 * C::kChunks>(stage_ptr(ring.of(j)), r0, BT, kChunkBytes);
                ptx::fence_proxy_async_smem();
                __syncwarp();
            };
            const uint32_t q_at = ptx::smem_u32(stage_ptr(ring.hold));
            // S = Q K^T (of = 0) and dP = dO V^T (of = 1)
            auto issue = [&](int of, int j, uint32_t to, uint64_t *bar) {
                const uint32_t at = uint32_t(of) * C::kTileBytes;
                const uint64_t da = ptx::smem_desc(desc_kmajor, q_at + at);
                const uint64_t db = ptx::smem_desc(desc_kmajor, ptx::smem_u32(stage_ptr(ring.of(j))) + at);
                if (ptx::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        ptx::mma_ss(tmem + to, da + kmajor_off(kk, kChunkBytes),
                                    db + kmajor_off(kk, kChunkBytes), idesc_s, kk > 0 ? 1u : 0u);
                    ptx::mma_commit(bar);
                }
                __syncwarp();
            };
            auto issue_dp = [&](int j, uint32_t step) {
                issue(1, j, C::col_dp(step), &dp_full[step % C::kDPs]);
            };
            // P_j K_j and dS_j K_j into `to`
            auto add = [&](int j, uint32_t to, uint32_t from) {
                const uint64_t db = ptx::smem_desc(desc_mnmajor, ptx::smem_u32(stage_ptr(ring.of(j))));
#pragma unroll
                for (int kk = 0; kk < BT / 16; ++kk)
                    ptx::mma_ts(tmem + to, tmem + from + packed_col(kk),
                                db + uint64_t((kk * 16 * 128) >> 4), idesc_q,
                                (j > 0 || kk > 0) ? 1u : 0u);
            };
            if (!wait_stage(ring.hold))
                break;
            for (int j = -1; j < n_kv; ++j) {
                const bool more_keys = j + 1 < n_kv;
                if (j >= 0) {
                    // (the rows have read the accumulators of the item before this one, too)
                    if (!ptx::mbar_wait_warp(p_full, g & 1u, abort_flag, a.err_word)) {
                        aborted = true;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    if (ptx::elect_one())
                        add(j, kColPK, 0);
                    __syncwarp();
                }
                if (more_keys) {
                    // S_{j+1} overwrites P_j, which its product has read
                    if (!wait_stage(ring.of(j + 1)))
                        break;
                    clear_tail(j + 1);
                    ptx::tc_fence_after_sync();
                    issue(0, j + 1, 0, s_full);
                    if (C::kDPs == 2)
                        issue_dp(j + 1, g + (j >= 0));
                }
                if (j >= 0) {
                    if (!ptx::mbar_wait_warp(ds_full, g & 1u, abort_flag, a.err_word)) {
                        aborted = true;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    if (ptx::elect_one()) {
                        add(j, kColAcc, C::col_dp(g));
                        ptx::mma_commit(&empty[ring.of(j)]);
                        if (!more_keys)
                            ptx::mma_commit(acc_full);
                    }
                    __syncwarp();
                    ++g;
                }
                // dP_{j+1} overwrites dS_j after the dQ product has read it
                if (more_keys && C::kDPs == 1)
                    issue_dp(j + 1, g);
                // Q and dO have no product ahead, and the rows have read dO
                if (j == max(n_kv - 2, 0)) {
                    if (ptx::elect_one())
                        ptx::mma_commit(&empty[ring.hold]);
                    __syncwarp();
                }
            }
            ring.next(n_kv);
        }
        if (ptx::elect_one()) {
            ptx::mma_commit(drain);
            ptx::drain_wait(drain, 0);
        }
        __syncwarp();
    } else {
        // ======================= query rows ================================
        const int r = (warp & 3) * 32 + lane, row_q = int(r * p.div_g >> 16);   // row = TMEM lane
        const int g = warp >> 2, col0 = 32 * g;      // of the row's four threads; its columns
        const uint32_t lane_bits = uint32_t((warp & 3) * 32) << 16;
        float *xch = reinterpret_cast<float *>(smem + C::kOffXch);
        float *xsum = reinterpret_cast<float *>(smem + C::kOffSum);
        const float sl = p.scale_log2;
        const uint32_t tS = tmem + lane_bits + uint32_t(col0);

        uint32_t step = 0, phases = 0;               // phases: of the stages, a bit each
        bool ready = !items[0].done;                 // there is an item k
        float lse = 0.f;
        // this thread's quarter of a row, from a tile (128-byte swizzle)
        auto unit = [&](const uint8_t *tile, int ul) {
            const int e0 = g * (D / 4) + ul * 8, un = (e0 & 63) >> 3;
            return *reinterpret_cast<const uint4 *>(tile + (e0 >> 6) * kChunkBytes + r * 128 +
                                                    ((un ^ (r & 7)) << 4));
        };
        auto stat_of = [&](const DqItem &it) {
            return stat_row(a, it.b, it.hk * p.G + r - row_q * p.G, it.q0) + it.i0 + row_q;
        };
        auto row_in = [&](const DqItem &it) { return row_q < p.P && it.i0 + row_q < it.i1; };
        // whether there is an item k; its statistic of this row
        auto prepare = [&](int k) {
            if (aborted || !row_wait(&known[k & 1], uint32_t(k >> 1) & 1u, abort_flag, a.err_word)) {
                aborted = true;
                return;
            }
            ready = !items[k & 1].done;
            if (ready && row_in(items[k & 1]))
                lse = a.lse[stat_of(items[k & 1])];
        };
        auto exchange = [&](float part) {            // the sum over a row's four threads
            xch[g * BT + r] = part;
            asm volatile("bar.sync 1, %0;" ::"n"(kRows) : "memory");
            return (xch[r] + xch[BT + r]) + (xch[2 * BT + r] + xch[3 * BT + r]);
        };
        if (ready)
            prepare(0);
        for (int k = 0; ready; ++k) {
            const DqItem &it = items[k & 1];         // (stays until out_full)
            const WindowKeys wk = keys_of(it);
            const int n_kv = steps_of(wk), i = it.i0 + row_q;
            const bool row_ok = row_in(it);
            const int vhi = row_ok ? i - wk.lo + wk.sp : -1;
            const int64_t vl = int64_t(vhi) - a.window + 1;
            const int vlo = vl > wk.sp ? int(vl) : wk.sp;
            const float lse2 = lse * kLog2e;
            float Di = 0.f;
            float2 ds_sum2 = make_float2(0.f, 0.f);
            for (int j = 0; j < n_kv; ++j, ++step) {
                const uint32_t par = step & 1u;
                float2 pr[16];
                bool ok = !aborted && row_wait(s_full, par, abort_flag, a.err_word);
                if (ok) {
                    ptx::tc_fence_after_sync();
                    uint32_t sv[32], pk[16];
                    ptx::tmem_ld32(tS, sv);
                    ptx::tmem_wait_ld();
                    const int v0 = j * BT + col0;    // this thread's first place
                    if (__any_sync(0xffffffffu, v0 < vlo || v0 + 31 > vhi)) {
                        const uint32_t seen = window_bits(v0, vlo, vhi, a.sinks);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(seen & (1u << e)))
                                sv[e] = __float_as_uint(-INFINITY);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 x = __ffma2_rn(make_float2(__uint_as_float(sv[2 * e]),
                                                                __uint_as_float(sv[2 * e + 1])),
                                                    make_float2(sl, sl), make_float2(-lse2, -lse2));
                        pr[e] = make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
                        pk[e] = ptx::pack_bf16x2(pr[e].x, pr[e].y);
                    }
                    ptx::tmem_st16(tS, pk);          // P of this row's 32 keys, packed
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        ptx::mbar_arrive(p_full);
                }
                if (j == 0) {
                    ok = ok &&
                         row_wait(&full[ring.hold], phases >> ring.hold & 1u, abort_flag, a.err_word) &&
                         row_wait(&o_in[k % C::kOBufs], uint32_t(k / C::kOBufs) & 1u, abort_flag,
                                  a.err_word);
                    float part = 0.f;                // of D_i = dO_i . O_i
                    if (ok) {
                        const uint8_t *tile_do = stage_ptr(ring.hold) + C::kTileBytes;
                        const uint8_t *tile_o = smem + C::kOffO + uint32_t(k % C::kOBufs) * C::kTileBytes;
#pragma unroll
                        for (int ul = 0; ul < D / 32; ++ul) {
                            const uint4 o = unit(tile_o, ul), gr = unit(tile_do, ul);
                            const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
                            const uint32_t gw[4] = {gr.x, gr.y, gr.z, gr.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                part = fmaf(__uint_as_float(ow[e] << 16),
                                            __uint_as_float(gw[e] << 16), part);
                                part = fmaf(__uint_as_float(ow[e] & 0xffff0000u),
                                            __uint_as_float(gw[e] & 0xffff0000u), part);
                            }
                        }
                    }
                    Di = exchange(part);
                }
                if (!ok || !row_wait(&dp_full[step % C::kDPs], (step / C::kDPs) & 1u, abort_flag,
                                     a.err_word)) {
                    aborted = true;
                    break;
                }
                ptx::tc_fence_after_sync();
                uint32_t dv[32], pk[16];
                ptx::tmem_ld32(tS + C::col_dp(step), dv);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 y = __fmul2_rn(
                        pr[e], __fadd2_rn(make_float2(__uint_as_float(dv[2 * e]),
                                                      __uint_as_float(dv[2 * e + 1])),
                                          make_float2(-Di, -Di)));
                    pk[e] = ptx::pack_bf16x2(y.x, y.y);
                }
                ptx::tmem_st16(tS + C::col_dp(step), pk);     // dS of this row's 32 keys, packed
                ptx::tmem_wait_st();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(ds_full);
                // (dS as the product has it)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    ds_sum2 = __fadd2_rn(ds_sum2, make_float2(__uint_as_float(pk[e] << 16),
                                                              __uint_as_float(pk[e] & 0xffff0000u)));
            }
            // (each stage's fills in this item: one of Q and dO, then steps in turn)
            phases ^= 1u << ring.hold | uint32_t((n_kv + 1) >> 1 & 1) << ring.a |
                      uint32_t(n_kv >> 1 & 1) << ring.b;
            ring.next(n_kv);
            prepare(k + 1);
            // the sum of the row's dS over its threads.  (Where D and the sums share a place:
            // with two steps or more, dP_1 came behind every row's dS_0 and so behind its
            // reading D.)
            if (C::kOffSum == C::kOffXch && n_kv == 1)
                asm volatile("bar.sync 1, %0;" ::"n"(kRows) : "memory");
            xsum[g * BT + r] = ds_sum2.x + ds_sum2.y;
            if (ptx::bar_red_or(2, kRows, aborted))
                break;
            const float ri = (xsum[r] + xsum[BT + r]) + (xsum[2 * BT + r] + xsum[3 * BT + r]);
            if (g == 0 && row_ok)
                p.D[stat_of(it)] = Di + ri;
            // 32 columns of each row's dQ a thread: a whole tile by one copy, a cut one row by
            // row
            const bool whole = it.i1 - it.i0 == p.P;
            if (!row_wait(acc_full, uint32_t(k) & 1u, abort_flag, a.err_word)) {
                aborted = true;
                continue;
            }
            ptx::tc_fence_after_sync();
            if (g < D / 32) {
                const int64_t row_h = it.hk * p.G + r - row_q * p.G;
                store_row<true>(tmem + lane_bits + kColAcc, a.scale,
                                row_ok ? p.dQ + (it.q0 + i) * p.dq_stride + row_h * D : nullptr,
                                whole ? smem + C::kOffOut : nullptr, r, g, g + 1, -ri,
                                tmem + lane_bits + kColPK);
                ptx::fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(out_full);
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    if (warp == kWarpMma)
        ptx::tmem_dealloc(tmem, kTmemCols);
}

// =============================================================================
// dK, dV
// =============================================================================
// Per 128-query step S^T = K Q_j^T in columns [0, 128) and dP^T = V dO_j^T in [128, 256)
// (a key per lane), P^T and dS^T packed into them; dV from 256, dK behind it.  The MMA
// warp issues dV += P^T_j dO_j, S^T_{j+1}, dK += dS^T_j Q_j, dP^T_{j+1}: sixteen row warps
// (four threads a row, 32 columns each) form P^T while dK and dP^T run, and dS^T while dV
// and S^T do.  (2 x 4096 queries, 32 heads on 8, d = 128, window 1024: 232 us, tensor cores
// 64 % busy; steps of 64 queries in two buffers took 304 us where these took 263.)
template <int D>
struct CfgK {
    static constexpr int kChunks = D / 64;
    static constexpr uint32_t kTileBytes = BT * D * 2;
    // [K][V][three Q][two dO][statistics: two of (-lse log2 e, -D) x 128][barriers]: Q_j is
    // read by S^T_j and, a step later, dK; dO_j by dP^T_j and dV soon after it
    static constexpr int kQ = 3, kDO = 2;
    static constexpr uint32_t kOffQ = 2 * kTileBytes;
    static constexpr uint32_t kOffDO = kOffQ + kQ * kTileBytes;
    static constexpr uint32_t kOffStat = kOffDO + kDO * kTileBytes;
    static constexpr uint32_t kOffBar = kOffStat + 2 * 2 * BT * 4;
    static constexpr int kBars = 1 + 2 * kQ + 2 * kDO + 2 + 6;
    static constexpr uint32_t kSmemBytes = kOffBar + 8 * kBars + 16;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// 128-query tiles of a sequence that have a key of tile kt in their window: [kt,
// near_end); those behind it see the tile's sinks alone.
__device__ __forceinline__ int near_end(int kt, int window, int L)
{
    const int n = (L + BT - 1) / BT;
    const int64_t e = (int64_t(kt) * BT + BT - 1 + window + BT - 1) / BT;
    return e < n ? int(e) : n;
}

// A sink tile's parts: [place][kv head][sink tile], a place being a slot of a sequence, slot
// 0 its window's.
__device__ __forceinline__ int64_t part_offset(const Params &p, int b, int hk, int kt, int slot,
                                               int64_t q0)
{
    const int64_t place = (p.part_cut.div > 0 ? p.part_cut.at(q0, b) : int64_t(b) * p.slots) + slot;
    return (place * p.a.Hkv + hk) * p.sink_tiles + kt;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_window_dkdv_kernel(const __grid_constant__ Params p)
{
    using C = CfgK<D>;
    // aligned as the tiles need it, with no room to align it here
    extern __shared__ __align__(1024) uint8_t smem_aligned[];
    uint8_t *smem = smem_aligned;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *a_full = bars, *q_full = bars + 1, *q_empty = q_full + C::kQ;
    uint64_t *do_full = q_empty + C::kQ, *do_empty = do_full + C::kDO, *st_full = do_empty + C::kDO;
    uint64_t *s_full = st_full + 2, *dp_full = s_full + 1, *p_full = s_full + 2,
             *ds_full = s_full + 3, *o_full = s_full + 4, *drain = s_full + 5;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffBar + 8 * C::kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    if (threadIdx.x == 32) {
        ptx::prefetch_tmap(&p.tm_k);
        ptx::prefetch_tmap(&p.tm_v);
        ptx::prefetch_tmap(&p.tm_q);
        ptx::prefetch_tmap(&p.tm_do);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // work item: the far pieces of the sinks' tiles first, then every key tile's window
    const WindowArgs &a = p.a;
    int b, hk, kt, slot = 0;
    const unsigned far = unsigned(p.far_items);
    if (blockIdx.x < far) {
        // (kt, place, kv head): a place is a (sequence, slot)
        const unsigned q = blockIdx.x / unsigned(p.sink_tiles);
        kt = int(blockIdx.x - q * unsigned(p.sink_tiles));
        hk = int(q % unsigned(a.Hkv));
        const int place = int(q / unsigned(a.Hkv));
        if (p.part_cut.div > 0) {
            int64_t number;
            b = window_find(a.cu_seqlens_q, a.B, p.part_cut, place, number);
            slot = int(number);
        } else {
            b = place / p.slots;
            slot = place - b * p.slots;
        }
        if (slot <= 0)
            return;                            // (the window's own part has its place, too)
    } else if (!window_item(a, p.grid, blockIdx.x - far, b, hk, kt)) {
        return;
    }
    WindowSeq sq;
    if (!window_seq(a, b, sq) || kt * BT >= sq.L)   // (a bad one is flagged by the dQ kernel)
        return;
    const int L = sq.L;
    const int n_qt = (L + BT - 1) / BT;
    const int near = near_end(kt, a.window, L);
    const bool in_parts = kt < p.sink_tiles && near < n_qt;   // several CTAs form this tile's sums
    int s0 = kt, s1 = near;                                   // 128-query tiles
    if (slot > 0) {
        s0 = near + (slot - 1) * p.piece;
        s1 = min(s0 + p.piece, n_qt);
        if (s0 >= s1)
            return;
    }
    const int n_i = s1 - s0, n_q = n_i * p.G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    uint8_t *tile_k = smem, *tile_v = smem + C::kTileBytes;
    float *stats = reinterpret_cast<float *>(smem + C::kOffStat);
    if (warp == kWarpLoad) {
        // the barriers, and the first copies while the others set up
        if (lane == 0) {
            ptx::mbar_init(a_full, 1);
            for (int s = 0; s < C::kQ; ++s) {
                ptx::mbar_init(&q_full[s], 1);
                ptx::mbar_init(&q_empty[s], 1);
            }
            for (int s = 0; s < C::kDO; ++s) {
                ptx::mbar_init(&do_full[s], 1);
                ptx::mbar_init(&do_empty[s], 1);
                ptx::mbar_init(&st_full[s], 32);     // the load warp's lanes
            }
            ptx::mbar_init(s_full, 1);
            ptx::mbar_init(dp_full, 1);
            ptx::mbar_init(p_full, kRowWarps);
            ptx::mbar_init(ds_full, kRowWarps);
            ptx::mbar_init(o_full, 1);
            ptx::mbar_init(drain, 1);
            *abort_flag = 0;
            ptx::fence_barrier_init();
            const int k_row = int(sq.k0 + int64_t(kt) * BT), q_row = int(sq.q0 + int64_t(s0) * BT);
            ptx::mbar_arrive_expect_tx(a_full, 2 * C::kTileBytes);
            ptx::mbar_arrive_expect_tx(&q_full[0], C::kTileBytes);
            ptx::mbar_arrive_expect_tx(&do_full[0], C::kTileBytes);
            ptx::tma_load_5d(tile_k, &p.tm_k, a_full, 0, 0, k_row, 0, hk);
            ptx::tma_load_5d(smem + C::kOffQ, &p.tm_q, &q_full[0], 0, 0, q_row, 0, hk * p.G);
            ptx::tma_load_5d(tile_v, &p.tm_v, a_full, 0, 0, k_row, 0, hk);
            ptx::tma_load_5d(smem + C::kOffDO, &p.tm_do, &do_full[0], 0, 0, q_row, 0, hk * p.G);
        }
        __syncwarp();
    }
    if (warp == kWarpMma) {
        ptx::tmem_alloc(tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool aborted = false;
    if (warp == kWarpLoad) {
        // ======================= TMA producer (whole warp) ===================
        // Per step j: Q_j (its place is free once dK_{j-3} is through), dO_j (dV_{j-2}),
        // and the queries' statistics (dK_{j-2}: the rows are done with step j - 2).
        int q_issued = 1, do_issued = 1;
        int h = hk * p.G, i = s0;
        // a step's statistics, on their way a step ahead
        float ls[BT / 32], ds[BT / 32];
        auto load_stats = [&](int h, int i) {
            const int64_t stat0 = stat_row(a, b, h, sq.q0);
#pragma unroll
            for (int u = 0; u < BT / 32; ++u) {
                const int q = i * BT + u * 32 + lane;
                ls[u] = q < L ? a.lse[stat0 + q] : 0.f;
                ds[u] = q < L ? p.D[stat0 + q] : 0.f;
            }
        };
        load_stats(h, i);
        for (int j = 0; j < n_q; ++j) {
            const int row = int(sq.q0 + int64_t(i) * BT);
            auto load = [&](uint8_t *dst, const CUtensorMap *tm, uint64_t *full) {
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(full, C::kTileBytes);
                    ptx::tma_load_5d(dst, tm, full, 0, 0, row, 0, h);
                }
                __syncwarp();
            };
            const int qs = j % C::kQ, os = j % C::kDO;
            if (j > 0) {
                if (!ptx::mbar_wait_warp(&q_empty[qs], (uint32_t(j / C::kQ) & 1u) ^ 1u, abort_flag,
                                         a.err_word))
                    break;
                load(smem + C::kOffQ + qs * C::kTileBytes, &p.tm_q, &q_full[qs]);
                q_issued = j + 1;
                if (!ptx::mbar_wait_warp(&do_empty[os], (uint32_t(j / C::kDO) & 1u) ^ 1u, abort_flag,
                                         a.err_word))
                    break;
                load(smem + C::kOffDO + os * C::kTileBytes, &p.tm_do, &do_full[os]);
                do_issued = j + 1;
            }
            if (j >= 2 && !ptx::mbar_wait_warp(&q_empty[(j - 2) % C::kQ],
                                               uint32_t((j - 2) / C::kQ) & 1u, abort_flag,
                                               a.err_word))
                break;
            float *st = stats + os * (2 * BT);
#pragma unroll
            for (int u = 0; u < BT / 32; ++u) {
                st[u * 32 + lane] = -ls[u] * kLog2e;
                st[BT + u * 32 + lane] = -ds[u];
            }
            ptx::mbar_arrive(&st_full[os]);          // all lanes, after their writes
            if (++i == s1) {
                i = s0;
                ++h;
            }
            if (j + 1 < n_q)
                load_stats(h, i);
        }
        if (lane == 0 && *abort_flag) {
            ptx::drain_wait(a_full, 0);
            for (int j = q_issued > C::kQ ? q_issued - C::kQ : 0; j < q_issued; ++j)
                ptx::drain_wait(&q_full[j % C::kQ], uint32_t(j / C::kQ) & 1u);
            for (int j = do_issued > C::kDO ? do_issued - C::kDO : 0; j < do_issued; ++j)
                ptx::drain_wait(&do_full[j % C::kDO], uint32_t(j / C::kDO) & 1u);
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        // ======================= MMA issuer (whole warp) =====================
        constexpr uint32_t idesc_ss = ptx::idesc_bf16_f32(BT, BT, false);
        constexpr uint32_t idesc_ts = ptx::idesc_bf16_f32(BT, D, true);
        constexpr uint64_t desc_kmajor = ptx::smem_desc_base(16, 1024);
        constexpr uint64_t desc_mnmajor = ptx::smem_desc_base(kChunkBytes, 1024);
        const uint64_t dk = ptx::smem_desc(desc_kmajor, ptx::smem_u32(tile_k));
        const uint64_t dvk = ptx::smem_desc(desc_kmajor, ptx::smem_u32(tile_v));
        const uint32_t q_addr = ptx::smem_u32(smem + C::kOffQ);
        const uint32_t do_addr = ptx::smem_u32(smem + C::kOffDO);
        int i = s0;
        auto q_tile = [&](int j) { return uint32_t(j % C::kQ) * C::kTileBytes; };
        auto do_tile = [&](int j) { return uint32_t(j % C::kDO) * C::kTileBytes; };
        // waits for step j's Q, for its dO; rows behind the sequence's end are cleared
        auto tail = [&](uint8_t *tile, int i) {
            if ((i + 1) * BT > L) {
                clear_rows<C::kChunks>(tile, L - i * BT, BT, kChunkBytes);
                ptx::fence_proxy_async_smem();
                __syncwarp();
            }
            ptx::tc_fence_after_sync();
        };
        auto q_ready = [&](int j) -> bool {
            if (!ptx::mbar_wait_warp(&q_full[j % C::kQ], uint32_t(j / C::kQ) & 1u, abort_flag,
                                     a.err_word))
                return false;
            tail(smem + C::kOffQ + q_tile(j), i);
            return true;
        };
        auto do_ready = [&](int j) -> bool {
            if (!ptx::mbar_wait_warp(&do_full[j % C::kDO], uint32_t(j / C::kDO) & 1u, abort_flag,
                                     a.err_word))
                return false;
            tail(smem + C::kOffDO + do_tile(j), i);
            if (++i == s1)
                i = s0;
            return true;
        };
        // S^T = K Q^T, dP^T = V dO^T
        auto issue = [&](uint32_t to, uint64_t da, uint32_t addr, uint64_t *bar) {
            const uint64_t db = ptx::smem_desc(desc_kmajor, addr);
            if (ptx::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    ptx::mma_ss(tmem + to, da + kmajor_off(kk, kChunkBytes),
                                db + kmajor_off(kk, kChunkBytes), idesc_ss, kk > 0 ? 1u : 0u);
                ptx::mma_commit(bar);
            }
            __syncwarp();
        };
        // dV += P^T dO, dK += dS^T Q
        auto add = [&](uint32_t to, uint32_t from, uint32_t addr, bool first, uint64_t *bar) {
            const uint64_t db = ptx::smem_desc(desc_mnmajor, addr);
            if (ptx::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < BT / 16; ++kk)
                    ptx::mma_ts(tmem + to, tmem + from + packed_col(kk),
                                db + uint64_t((kk * 16 * 128) >> 4), idesc_ts,
                                (!first || kk > 0) ? 1u : 0u);
                ptx::mma_commit(bar);
            }
            __syncwarp();
        };
        do {
            if (!ptx::mbar_wait_warp(a_full, 0, abort_flag, a.err_word) || !q_ready(0)) {
                aborted = true;
                break;
            }
            issue(0, dk, q_addr, s_full);
            if (!do_ready(0)) {
                aborted = true;
                break;
            }
            issue(kColDP, dvk, do_addr, dp_full);
            int j = 0;
            for (; j < n_q; ++j) {
                const bool more = j + 1 < n_q;
                if (!ptx::mbar_wait_warp(p_full, uint32_t(j) & 1u, abort_flag, a.err_word))
                    break;
                ptx::tc_fence_after_sync();
                add(kColAcc, 0, do_addr + do_tile(j), j == 0, &do_empty[j % C::kDO]);
                if (more) {                         // S^T_{j+1} overwrites P^T_j, which dV has read
                    if (!q_ready(j + 1))
                        break;
                    issue(0, dk, q_addr + q_tile(j + 1), s_full);
                }
                if (!ptx::mbar_wait_warp(ds_full, uint32_t(j) & 1u, abort_flag, a.err_word))
                    break;
                ptx::tc_fence_after_sync();
                add(kColAcc + D, kColDP, q_addr + q_tile(j), j == 0, &q_empty[j % C::kQ]);
                if (more) {
                    if (!do_ready(j + 1))
                        break;
                    issue(kColDP, dvk, do_addr + do_tile(j + 1), dp_full);
                }
            }
            aborted = j < n_q;
        } while (false);
        if (ptx::elect_one()) {
            if (!aborted)
                ptx::mma_commit(o_full);
            ptx::mma_commit(drain);
            ptx::drain_wait(drain, 0);
        }
        __syncwarp();
    } else {
        // ======================= key rows ==================================
        const int r = (warp & 3) * 32 + lane;        // key of the tile = TMEM lane
        const int g = warp >> 2, col0 = 32 * g;      // of the row's four threads; its columns
        const int k = kt * BT + r;
        const uint32_t lane_bits = uint32_t((warp & 3) * 32) << 16;
        const float sl = p.scale_log2;
        // queries that see the key: k .. last
        const int64_t end = k < a.sinks ? int64_t(L) : int64_t(k) + a.window;
        const int last = int(end < L ? end : L) - 1;
        const uint32_t tS = tmem + lane_bits + uint32_t(col0);
        int i = s0;
        for (int j = 0; j < n_q; ++j) {
            const uint32_t par = uint32_t(j) & 1u;
            const int q0 = i * BT + col0;            // this thread's first query
            if (++i == s1)
                i = s0;
            if (!row_wait(&st_full[j & 1], uint32_t(j >> 1) & 1u, abort_flag, a.err_word) ||
                !row_wait(s_full, par, abort_flag, a.err_word)) {
                aborted = true;
                break;
            }
            ptx::tc_fence_after_sync();
            const float *stat = stats + (j & 1) * (2 * BT) + col0;
            uint32_t sv[32], pk[16];
            ptx::tmem_ld32(tS, sv);
            ptx::tmem_wait_ld();
            const int lo = k - q0, hi = last - q0;   // seen columns
            if (__any_sync(0xffffffffu, lo > 0 || hi < 31)) {
                const uint32_t seen = low_bits(hi + 1) & ~low_bits(lo);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (!(seen & (1u << e)))
                        sv[e] = __float_as_uint(-INFINITY);
            }
            float2 pr[16];
#pragma unroll
            for (int e4 = 0; e4 < 8; ++e4) {
                const float4 l4 = *reinterpret_cast<const float4 *>(stat + 4 * e4);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int e = 4 * e4 + 2 * half;
                    const float2 x = __ffma2_rn(
                        make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])),
                        make_float2(sl, sl),
                        half ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y));
                    pr[e / 2] = make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
                    pk[e / 2] = ptx::pack_bf16x2(pr[e / 2].x, pr[e / 2].y);
                }
            }
            ptx::tmem_st16(tS, pk);                  // P^T of this block, packed
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(p_full);
            if (!row_wait(dp_full, par, abort_flag, a.err_word)) {
                aborted = true;
                break;
            }
            ptx::tc_fence_after_sync();
            uint32_t dv[32];
            ptx::tmem_ld32(tS + kColDP, dv);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e4 = 0; e4 < 8; ++e4) {
                const float4 d4 = *reinterpret_cast<const float4 *>(stat + BT + 4 * e4);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int e = 4 * e4 + 2 * half;
                    const float2 y = __fmul2_rn(
                        pr[e / 2],
                        __fadd2_rn(make_float2(__uint_as_float(dv[e]), __uint_as_float(dv[e + 1])),
                                   half ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y)));
                    pk[e / 2] = ptx::pack_bf16x2(y.x, y.y);
                }
            }
            ptx::tmem_st16(tS + kColDP, pk);         // dS^T of this block, packed
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(ds_full);
        }
        // groups 0 and 1 have dV, 2 and 3 dK, half of the columns each: a whole tile by way of
        // V's and K's places (all products are through) and a copy each, a cut one row by row
        const int of = g >> 1, c0 = (g & 1) * (D / 64), c1 = c0 + D / 64;
        const uint32_t acc = tmem + lane_bits + kColAcc + uint32_t(of * D);
        const float mul = of == 0 ? 1.f : a.scale;
        const bool key_ok = k < L, whole = !in_parts && kt * BT + BT <= L;
        const bool ok = !aborted && ptx::mbar_wait(o_full, 0, abort_flag, a.err_word);
        if (ok) {
            ptx::tc_fence_after_sync();
            if (in_parts) {
                float *part = p.parts + part_offset(p, b, hk, kt, slot, sq.q0) * (2 * BT * D) +
                              of * (BT * D) + r * D;
#pragma unroll 1
                for (int c = c0; c < c1; ++c) {
                    uint32_t o[32];
                    ptx::tmem_ld32(acc + c * 32, o);
                    ptx::tmem_wait_ld();
                    if (key_ok)
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            *reinterpret_cast<float4 *>(part + c * 32 + 4 * q) =
                                make_float4(__uint_as_float(o[4 * q]) * mul,
                                            __uint_as_float(o[4 * q + 1]) * mul,
                                            __uint_as_float(o[4 * q + 2]) * mul,
                                            __uint_as_float(o[4 * q + 3]) * mul);
                }
            } else {
                __nv_bfloat16 *dst = of == 0 ? p.dV + (sq.k0 + k) * p.dv_stride
                                             : p.dK + (sq.k0 + k) * p.dk_stride;
                store_row(acc, mul, key_ok ? dst + int64_t(hk) * D : nullptr,
                          whole ? (of == 0 ? tile_v : tile_k) : nullptr, r, c0, c1);
            }
        }
        if (whole) {
            ptx::fence_proxy_async_smem();
            if (!ptx::bar_red_or(1, 32 * kRowWarps, !ok) && threadIdx.x == 0) {
                const int k_row = int(sq.k0 + int64_t(kt) * BT);
                ptx::tma_store_5d(&p.tm_d0, tile_v, 0, 0, k_row, 0, hk);
                ptx::tma_store_5d(&p.tm_d1, tile_k, 0, 0, k_row, 0, hk);
                ptx::bulk_commit_and_wait_read();
            }
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    if (warp == kWarpMma)
        ptx::tmem_dealloc(tmem, kTmemCols);
}

// A sink tile's parts added in order: a warp a row of dV or dK.
template <int D>
__global__ void __launch_bounds__(256) attn_window_join_kernel(const __grid_constant__ Params p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const WindowArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    const int64_t item = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int r = int(item % BT);
    const int g = int(item / BT % 2), kt = int(item / (2 * BT) % p.sink_tiles);
    const int bh = int(item / (2 * BT) / p.sink_tiles);
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    WindowSeq sq;
    if (!window_seq(a, b, sq) || kt * BT + r >= sq.L)
        return;
    const int n_qt = (sq.L + BT - 1) / BT, near = near_end(kt, a.window, sq.L);
    if (near >= n_qt)
        return;
    const int n = 1 + (n_qt - near + p.piece - 1) / p.piece;
    const float *part = p.parts + part_offset(p, b, hk, kt, 0, sq.q0) * (2 * BT * D) + g * (BT * D) +
                        r * D + lane * (D / 32);
    const int64_t next = int64_t(a.Hkv) * p.sink_tiles * (2 * BT * D);
    float v[D / 32] = {};
    for (int s = 0; s < n; ++s, part += next)
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            v[e] += part[e];
    const int64_t row = sq.k0 + kt * BT + r;
    __nv_bfloat16 *dst = (g == 0 ? p.dV + row * p.dv_stride : p.dK + row * p.dk_stride) +
                         int64_t(hk) * D + lane * (D / 32);
#pragma unroll
    for (int e = 0; e < D / 32; e += 2)
        *reinterpret_cast<uint32_t *>(dst + e) = ptx::pack_bf16x2(v[e], v[e + 1]);
}

template <int D>
int launch_d(const Params &pq, const Params &pk, int64_t dq_blocks, int64_t kv_blocks,
             int64_t join_blocks, cudaStream_t stream)
{
    auto kq = attn_window_dq_kernel<D>;
    auto kk = attn_window_dkdv_kernel<D>;
    static PerDeviceOnce once_q, once_k;
    constexpr int smem_q = int(CfgQ<D>::kSmemBytes), smem_k = int(CfgK<D>::kSmemBytes);
    if (!set_max_dynamic_smem(once_q, reinterpret_cast<const void *>(kq), smem_q) ||
        !set_max_dynamic_smem(once_k, reinterpret_cast<const void *>(kk), smem_k) ||
        launch_early(kq, dim3(unsigned(dq_blocks)), kThreads, smem_q, stream, pq) != cudaSuccess ||
        launch_early(kk, dim3(unsigned(kv_blocks)), kThreads, smem_k, stream, pk) != cudaSuccess)
        return FA_ERR_CUDA;
    if (join_blocks > 0 && launch_early(attn_window_join_kernel<D>, dim3(unsigned(join_blocks)), 256, 0,
                                        stream, pk) != cudaSuccess)
        return FA_ERR_CUDA;
    return FA_OK;
}

}  // namespace

int launch_attention_window_bwd(const WindowBwdArgs &w, cudaStream_t stream)
{
    const WindowArgs &a = w.a;
    const WindowBwdLayout lay = window_bwd_layout(a.B, a.Nq, a.total_q, a.H, a.Hkv, a.d, a.window,
                                                  a.sinks);
    Params pq{};
    pq.a = a;
    uint8_t *ws = static_cast<uint8_t *>(w.workspace);
    pq.D = reinterpret_cast<float *>(ws + lay.D);
    pq.parts = reinterpret_cast<float *>(ws + lay.parts);
    pq.dQ = static_cast<__nv_bfloat16 *>(w.dQ);
    pq.dK = static_cast<__nv_bfloat16 *>(w.dK);
    pq.dV = static_cast<__nv_bfloat16 *>(w.dV);
    pq.dq_stride = w.dq_stride;
    pq.dk_stride = w.dk_stride;
    pq.dv_stride = w.dv_stride;
    pq.G = a.H / a.Hkv;
    pq.P = BT / pq.G;
    pq.q_chunks = tmap_heads_chunks(pq.G, a.d, pq.P);
    pq.div_g = uint32_t(65536 / pq.G + 1);
    pq.grid = window_grid(a, pq.P);
    pq.sink_tiles = lay.sink_tiles;
    pq.slots = lay.slots;
    pq.part_cut = lay.cut_div > 0 ? WindowCut{3, lay.cut_div, 0} : WindowCut{0, 0, 0};
    pq.piece = lay.piece;
    pq.scale_log2 = float(double(a.scale) * 1.4426950408889634);
    Params pk = pq;
    pk.grid = window_grid(a, BT);
    const int64_t bh = int64_t(a.B) * a.Hkv;
    const int64_t dq_blocks = window_items(a, pq.grid);
    const int64_t far_blocks = lay.places * lay.sink_tiles * a.Hkv;
    const int64_t kv_blocks = window_items(a, pk.grid) + far_blocks;
    const int64_t join_blocks = lay.slots > 1 ? bh * lay.sink_tiles * (2 * BT / 8) : 0;
    if (dq_blocks > 0x7fffffffLL || kv_blocks > 0x7fffffffLL || join_blocks > 0x7fffffffLL)
        return FA_ERR_TOO_LARGE;
    pk.far_items = int(far_blocks);
    const int64_t row = int64_t(a.H) * a.d;
    if (!make_tmap_heads(&pq.tm_q, a.Q, a.total_q, a.Hkv, pq.G, a.d, a.q_stride, pq.P) ||
        !make_tmap_heads(&pq.tm_do, w.dO, a.total_q, a.Hkv, pq.G, a.d, row, pq.P) ||
        !make_tmap_heads(&pq.tm_o, a.O, a.total_q, a.Hkv, pq.G, a.d, row, pq.P) ||
        !make_tmap_heads(&pq.tm_k, a.K, a.total_k, a.Hkv, 1, a.d, a.k_stride, BT) ||
        !make_tmap_heads(&pq.tm_v, a.V, a.total_k, a.Hkv, 1, a.d, a.v_stride, BT) ||
        !make_tmap_heads(&pq.tm_k32, a.K, a.total_k, a.Hkv, 1, a.d, a.k_stride, kPad) ||
        !make_tmap_heads(&pq.tm_v32, a.V, a.total_k, a.Hkv, 1, a.d, a.v_stride, kPad) ||
        !make_tmap_heads(&pk.tm_q, a.Q, a.total_q, a.H, 1, a.d, a.q_stride, BT) ||
        !make_tmap_heads(&pk.tm_do, w.dO, a.total_q, a.H, 1, a.d, row, BT))
        return FA_ERR_CUDA;
    if (!make_tmap_heads(&pq.tm_d0, w.dQ, a.total_q, a.Hkv, pq.G, a.d, w.dq_stride, pq.P) ||
        !make_tmap_heads(&pk.tm_d0, w.dV, a.total_k, a.Hkv, 1, a.d, w.dv_stride, BT) ||
        !make_tmap_heads(&pk.tm_d1, w.dK, a.total_k, a.Hkv, 1, a.d, w.dk_stride, BT))
        return FA_ERR_CUDA;
    pk.tm_k = pq.tm_k;
    pk.tm_v = pq.tm_v;
    return a.d == 64 ? launch_d<64>(pq, pk, dq_blocks, kv_blocks, join_blocks, stream)
                     : launch_d<128>(pq, pk, dq_blocks, kv_blocks, join_blocks, stream);
}

}  // namespace fa
