// attn_window.cu -- attention with a sliding window and sinks, forward, for many
// queries (chunks of prompts, training), on the sm_103a tensor cores.
//
// What it computes: O = softmax(scale Q K^T | seen keys) V and the row logsumexp,
// with the online softmax over tiles of 128 keys, as attn_bf16.cu does.  What the
// window changes:
//   * a CTA's keys are the window of its queries and the sinks, laid one behind
//     the other (window.cuh), so that few sinks share a tile with the window's
//     first keys instead of taking a tile of their own; the window starts at any
//     row, tiles need no alignment to multiples of 128;
//   * the tiles are few (window 1024: nine), so rows that do not see the same keys
//     cost: the rows of a tile are the queries of the G query heads that share a kv
//     head, row r = query r / G, head r % G, and the two tiles of a CTA follow one
//     another in the sequence: 256 rows span 256 / G positions and see window + 256
//     / G keys at most;
//   * a row's mask is two ranges of columns, formed as bits 32 columns at a time.
// Roles, tensor memory and the order of the products are those of attn_bf16.cu: a
// CTA per SM; warps 0-3 and 4-7 the softmax of Q0 and Q1, a thread per row; warp 8
// TMA, warp 9 tcgen05.  S0 [0, 128), S1 [128, 256), O0 and O1 from 256 (with a narrow
// window one tile a CTA, two CTAs an SM: S0, then O0 from 128); P in bf16 over the upper
// half of S: probabilities relative to a reference that at most 2^8
// below the row's maximum, each off by 2^-9 relative, and the sum that divides O
// is corrected by the error of the tile's largest.
// Where the items (two tiles of a kv head) are few, a cluster of 2 to 8 CTAs takes one, a
// range of its steps each; the rows' unnormalised O, maxima and sums meet through
// distributed shared memory, where each CTA joins a share of the rows.
// Rows of V behind a sequence's keys (the room of a cache, the next sequence) are
// zeroed in shared memory before the product reads them: their P is 0, but they may
// hold NaN.  Every wait is bounded; a timed-out one leaves the CTA's rows unwritten.
//
// Bound by the chain product, softmax, product, of which a CTA has two in turn: 2 x 4096
// queries, 32 heads on 8, d = 128, window 1024, 128 us (121 GFLOP at the keys seen, 940
// TFLOP/s; tensor cores 48 % busy, where the start and end of a CTA, 3.5 us of its 18, leave
// them idle).  1 x 32768, 16 heads on 4, window 2048: 427 us, 1250 TFLOP/s.  4 chunks of 512
// queries at most, 32 heads on 8, window 4096: 84 to 86 us, 890 to 912 TFLOP/s, in two waves of
// CTAs.
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

constexpr int BM = 128, BN = 128;
constexpr int kPad = 32;               // sinks fill whole pieces of a tile
constexpr uint32_t kColPinS = 64;
constexpr uint32_t kChunkBytes = BM * 128;   // 128 rows of 64 bf16
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kRescaleLog2 = 8.f;

__device__ __forceinline__ uint32_t col_s(int t) { return uint32_t(t) * 128u; }

// TILES query tiles a CTA: two, one CTA an SM; or one, two CTAs an SM.
template <int D, int TILES>
struct Cfg {
    static constexpr int kThreads = 128 * TILES + 64;
    static constexpr int kWarpLoad = 4 * TILES, kWarpMma = kWarpLoad + 1;
    static constexpr uint32_t kTmemCols = 256 * TILES, kColO = 128 * TILES;
    static constexpr int kChunks = D / 64;
    static constexpr uint32_t kTileBytes = BM * D * 2;
    static constexpr int kStages = (D == 128 ? 2 : 4) * TILES;
    static constexpr uint32_t kOffRing = TILES * kTileBytes;   // [Q0][Q1][ring][barriers]
    static constexpr uint32_t kOffBar = kOffRing + kStages * kTileBytes;
    static constexpr uint32_t kBars = 2 + 2 * kStages + 2 + 2 + 2 + 1 + 1;
    static constexpr uint32_t kSmemBytes = kOffBar + 8 * kBars + 16 + 1024;
    static_assert(kSmemBytes <= (TILES == 2 ? 227 : 113) * 1024, "shared memory");
};

struct Params {
    CUtensorMap tm_q, tm_o;            // P rows of G heads, q_chunks chunks a copy
    CUtensorMap tm_k, tm_v;            // 128 rows of a head
    CUtensorMap tm_k32, tm_v32;        // 32 rows, a chunk a copy: the tile where the sinks end
    WindowArgs a;
    int G, P, q_chunks;                // heads of a kv head; queries of a tile
    uint32_t div_g;                    // r / G = r * div_g >> 16 for r < 128
    WindowGrid grid;                   // of TILES * P queries
    int split;
    float scale_log2;
};

template <int D, bool SPLIT, int TILES>
__global__ void __launch_bounds__(Cfg<D, TILES>::kThreads, TILES == 2 ? 1 : 2)
    attn_window_kernel(const __grid_constant__ Params p)
{
    using C = Cfg<D, TILES>;
    static_assert(!SPLIT || TILES == 2, "a join has two tiles' threads");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *q_full = bars, *kv_full = bars + 2, *kv_empty = kv_full + C::kStages;
    uint64_t *s_full = kv_empty + C::kStages, *p_full = s_full + 2, *o_full = s_full + 4;
    uint64_t *drain = s_full + 6, *never = s_full + 7;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    if (threadIdx.x == 32) {
        ptx::prefetch_tmap(&p.tm_q);
        ptx::prefetch_tmap(&p.tm_k);
        ptx::prefetch_tmap(&p.tm_v);
        ptx::prefetch_tmap(&p.tm_k32);
        ptx::prefetch_tmap(&p.tm_v32);
        ptx::prefetch_tmap(&p.tm_o);
    }
    // nothing that a kernel before may still be writing is read ahead of this
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- work item: the last pairs of a sequence first (early ones see less) ------
    const WindowArgs &a = p.a;
    const int n_split = SPLIT ? p.split : 1;
    const int part = SPLIT ? int(blockIdx.x % unsigned(n_split)) : 0;
    const int item = SPLIT ? int(blockIdx.x / unsigned(n_split)) : int(blockIdx.x);
    int b, hk, pair;
    window_check(a, p.grid, blockIdx.x);
    if (!window_item(a, p.grid, unsigned(item), b, hk, pair))
        return;
    WindowSeq sq;
    if (!window_seq(a, b, sq)) {
        if (threadIdx.x == 0 && pair == 0 && hk == 0 && part == 0)
            record_device_error(a.err_word, FA_DEVERR_BAD_SEQLENS);
        return;
    }
    const int i0 = pair * TILES * p.P;         // first query of the pair
    if (i0 >= sq.n)
        return;
    const int off = sq.L - sq.n;
    const bool has_q1 = TILES == 2 && i0 + p.P < sq.n;
    const int i1 = min(i0 + p.P, sq.n), i2 = min(i0 + TILES * p.P, sq.n);
    const WindowKeys w = window_keys(a.window, a.sinks, i0, i2, off, kPad);
    // tile t takes steps [first_t, last_t) of the places' tiles: Q0 those that its
    // own last query reaches, Q1 all but leading ones that are behind its window
    const int all_steps = (w.places + BN - 1) / BN;
    const int reach0 = w.places - (i2 - i1);
    // this CTA's steps are [step0, step1)
    const int step0 = SPLIT ? int(int64_t(all_steps) * part / n_split) : 0;
    const int step1 = SPLIT ? int(int64_t(all_steps) * (part + 1) / n_split) : all_steps;
    const int first0 = step0;
    const int last0 = min(reach0 > w.sp ? (reach0 + BN - 1) / BN : 0, step1);
    const int first1 = max(a.sinks == 0 && w.lo > 0 ? p.P / BN : 0, step0);
    const int last1 = has_q1 ? step1 : 0;
    const int n_steps = step1 - step0;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int t = 0; t < TILES; ++t) {
            ptx::mbar_init(&q_full[t], 1);
            ptx::mbar_init(&s_full[t], 1);
            ptx::mbar_init(&p_full[t], 128);
            ptx::mbar_init(&o_full[t], 1);
        }
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(&kv_full[s], 1);
            ptx::mbar_init(&kv_empty[s], 1);
        }
        ptx::mbar_init(drain, 1);
        ptx::mbar_init(never, 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == C::kWarpMma) {
        ptx::tmem_alloc(tmem_slot, C::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool aborted = false;
    uint8_t *ring = smem + C::kOffRing;

    if (warp == C::kWarpLoad) {
        // ======================= TMA producer (whole warp) ===================
        int last_phase[C::kStages];
        for (int s = 0; s < C::kStages; ++s)
            last_phase[s] = -1;
        bool q_issued[2] = {false, false};
        auto load_q = [&](int t) {
            q_issued[t] = true;
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(&q_full[t], C::kChunks * p.P * p.G * 128);
                for (int c = 0; c < C::kChunks; c += p.q_chunks)
                    ptx::tma_load_5d(smem + t * C::kTileBytes + c * kChunkBytes, &p.tm_q,
                                     &q_full[t], 0, 0, int(sq.q0 + (t ? i1 : i0)), c, hk);
            }
            __syncwarp();
        };
        if (last0 > first0)
            load_q(0);
        int stage = 0;
        uint32_t phase = 0;
        for (int j = step0; j < step1 && !aborted; ++j) {
            for (int kv = 0; kv < 2; ++kv) {
                if (!ptx::mbar_wait_warp(&kv_empty[stage], phase ^ 1u, abort_flag, a.err_word)) {
                    aborted = true;
                    break;
                }
                if (lane == 0)
                    ptx::mbar_arrive_expect_tx(&kv_full[stage], C::kTileBytes);
                __syncwarp();
                uint8_t *dst = ring + stage * C::kTileBytes;
                const int v0 = j * BN;
                if (v0 < w.sp && v0 + BN > w.sp) {
                    // pieces of 32 rows, a lane each
                    const int c = lane / (BN / kPad), q = lane % (BN / kPad), v = v0 + q * kPad;
                    if (c < C::kChunks)
                        ptx::tma_load_5d(dst + c * kChunkBytes + q * kPad * 128,
                                         kv ? &p.tm_v32 : &p.tm_k32, &kv_full[stage], 0, 0,
                                         int(sq.k0 + (v < w.sp ? v : w.lo + v - w.sp)), c, hk);
                } else if (lane == 0) {
                    ptx::tma_load_5d(dst, kv ? &p.tm_v : &p.tm_k, &kv_full[stage], 0, 0,
                                     int(sq.k0 + (v0 < w.sp ? v0 : w.lo + v0 - w.sp)), 0, hk);
                }
                __syncwarp();
                last_phase[stage] = int(phase);
                if (++stage == C::kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (j == step0 && kv == 0 && last1 > first1)
                    load_q(1);
            }
        }
        if (lane == 0 && (aborted || *abort_flag)) {
            // copies already issued land before the CTA goes away
            for (int t = 0; t < TILES; ++t)
                if (q_issued[t])
                    ptx::drain_wait(&q_full[t], 0);
            for (int s = 0; s < C::kStages; ++s)
                if (last_phase[s] >= 0)
                    ptx::drain_wait(&kv_full[s], uint32_t(last_phase[s]));
        }
        __syncwarp();
    } else if (warp == C::kWarpMma) {
        // ======================= MMA issuer (whole warp) =====================
        constexpr uint32_t idesc_qk = ptx::idesc_bf16_f32(BM, BN, false);
        constexpr uint32_t idesc_pv = ptx::idesc_bf16_f32(BM, D, true);
        constexpr uint64_t desc_kmajor = ptx::smem_desc_base(16, 1024);
        constexpr uint64_t desc_mnmajor = ptx::smem_desc_base(kChunkBytes, 1024);
        const uint32_t ring_addr = ptx::smem_u32(ring), q_addr = ptx::smem_u32(smem);
        auto issue_qk = [&](int t, int st) {
            const uint64_t dq = ptx::smem_desc(desc_kmajor, q_addr + t * C::kTileBytes);
            const uint64_t dk = ptx::smem_desc(desc_kmajor, ring_addr + st * C::kTileBytes);
            if (ptx::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t o = ((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4;
                    ptx::mma_ss(tmem + col_s(t), dq + o, dk + o, idesc_qk, kk > 0 ? 1u : 0u);
                }
                ptx::mma_commit(&s_full[t]);
            }
            __syncwarp();
        };
        auto issue_pv = [&](int t, int st, bool accumulate, bool last) {
            const uint64_t dv = ptx::smem_desc(desc_mnmajor, ring_addr + st * C::kTileBytes);
            if (ptx::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                    ptx::mma_ts(tmem + C::kColO + uint32_t(t) * D, tmem + col_s(t) + kColPinS + kk * 8,
                                dv + uint64_t((kk * 16 * 128) >> 4), idesc_pv,
                                (accumulate || kk > 0) ? 1u : 0u);
                if (last)
                    ptx::mma_commit(&o_full[t]);
            }
            __syncwarp();
        };
        auto release = [&](int st) {
            if (ptx::elect_one())
                ptx::mma_commit(&kv_empty[st]);
            __syncwarp();
        };
        int stage = 0;
        uint32_t phase = 0;
        // waits for the next ring stage and returns it (-1: gave up)
        auto next_stage = [&]() -> int {
            if (!ptx::mbar_wait_warp(&kv_full[stage], phase, abort_flag, a.err_word))
                return -1;
            const int st = stage;
            if (++stage == C::kStages) {
                stage = 0;
                phase ^= 1u;
            }
            return st;
        };
        // V's rows of step j behind the sequence's keys are cleared
        const int end_place = w.sp + (sq.L - w.lo);
        auto clear_tail = [&](int j, int st) {
            const int r0 = end_place - j * BN;
            if (r0 >= BN)
                return;
            uint8_t *v = ring + st * C::kTileBytes;
            for (int r = max(r0, 0) + (lane >> 3); r < BN; r += 4)
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c)
                    *reinterpret_cast<uint4 *>(v + c * kChunkBytes + r * 128 + (lane & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
            ptx::fence_proxy_async_smem();
            __syncwarp();
        };
        if (a.expire_wait_ns != 0u &&
            !__all_sync(0xffffffffu, ptx::mbar_wait_limited(never, 0, abort_flag, a.err_word,
                                                            a.expire_wait_ns)))
            aborted = true;
        auto has = [&](int t, int j) {
            return t ? TILES == 2 && j >= first1 && j < last1 : j >= first0 && j < last0;
        };
        bool q_ready[2] = {false, false};
        auto wait_q = [&](int t) -> bool {
            if (!q_ready[t])
                q_ready[t] = ptx::mbar_wait_warp(&q_full[t], 0, abort_flag, a.err_word);
            return q_ready[t];
        };
        do {
            if (aborted || n_steps == 0)
                break;
            aborted = true;                        // until the loop is through
            int k_st = next_stage();
            if (k_st < 0)
                break;
            if (has(0, step0) && !wait_q(0))
                break;
            ptx::tc_fence_after_sync();
            if (has(0, step0))
                issue_qk(0, k_st);
            if (has(1, step0)) {
                if (!wait_q(1))
                    break;
                ptx::tc_fence_after_sync();
                issue_qk(1, k_st);
            }
            release(k_st);
            int j = step0;
            for (; j < step1; ++j) {
                const int v_st = next_stage();
                if (v_st < 0)
                    break;
                clear_tail(j, v_st);
                if (has(0, j)) {
                    if (!ptx::mbar_wait_warp(&p_full[0], uint32_t(j - first0) & 1u, abort_flag,
                                             a.err_word))
                        break;
                    ptx::tc_fence_after_sync();
                    issue_pv(0, v_st, j > first0, j == last0 - 1);
                }
                const bool more = j + 1 < step1;
                if (more) {
                    if ((k_st = next_stage()) < 0)
                        break;
                    ptx::tc_fence_after_sync();
                    if (has(0, j + 1))
                        issue_qk(0, k_st);
                }
                if (has(1, j)) {
                    if (!ptx::mbar_wait_warp(&p_full[1], uint32_t(j - first1) & 1u, abort_flag,
                                             a.err_word))
                        break;
                    ptx::tc_fence_after_sync();
                    issue_pv(1, v_st, j > first1, j == last1 - 1);
                }
                release(v_st);
                if (more) {
                    if (has(1, j + 1)) {
                        if (!wait_q(1))
                            break;
                        ptx::tc_fence_after_sync();
                        issue_qk(1, k_st);
                    }
                    release(k_st);
                }
            }
            aborted = j < step1;
        } while (false);
        // every product issued above is through once this commit arrives
        if (ptx::elect_one()) {
            ptx::mma_commit(drain);
            ptx::drain_wait(drain, 0);
        }
        __syncwarp();
    } else {
        // ======================= softmax warpgroups ========================
        const int t = TILES == 1 ? 0 : warp >> 2;
        const int r = threadIdx.x & 127;               // row of the tile = TMEM lane
        const int j0 = t ? first1 : first0, j1 = t ? last1 : last0;
        const int qi = int(r * p.div_g >> 16), i = (t ? i1 : i0) + qi;
        const int h = hk * p.G + r - qi * p.G;            // query, head
        const bool row_ok = qi < p.P && i < (t ? i2 : i1);
        const uint32_t lane_bits = uint32_t((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_bits + col_s(t);
        const uint32_t tO = tmem + lane_bits + C::kColO + uint32_t(t) * D;
        const int vhi = row_ok ? i + off - w.lo + w.sp : -1;
        const int64_t vl = int64_t(vhi) - a.window + 1;
        const int vlo = vl > w.sp ? int(vl) : w.sp;
        const float sl = p.scale_log2;
        float m = -INFINITY;                           // reference, log2 units
        float l = 0.f;                                 // running sum (lse)
        float l_o = 0.f;                               // the sum that divides O (see above)

        for (int j = j0; j < j1; ++j) {
            if (!ptx::mbar_wait(&s_full[t], uint32_t(j - j0) & 1u, abort_flag, a.err_word)) {
                aborted = true;
                break;
            }
            ptx::tc_fence_after_sync();
            uint32_t sr[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                ptx::tmem_ld32(tS + c * 32, sr[c]);
            ptx::tmem_wait_ld();
            const int v0 = j * BN;
            if (__any_sync(0xffffffffu, v0 < vlo || v0 + BN - 1 > vhi)) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t seen = window_bits(v0 + 32 * c, vlo, vhi, a.sinks);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(seen & (1u << e)))
                            sr[c][e] = __float_as_uint(-INFINITY);
                }
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int q = 0; q < 16; ++q)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = q * 8 + 2 * k;
                    m4[k] = ptx::max3(m4[k], __uint_as_float(sr[c >> 5][c & 31]),
                                      __uint_as_float(sr[(c + 1) >> 5][(c + 1) & 31]));
                }
            const float mx = fmaxf(ptx::max3(m4[0], m4[1], m4[2]), m4[3]);
            const float mt = mx * sl;
            const bool grew = mt > m + kRescaleLog2;
            const float m_new = grew ? mt : m;
            const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
            const float corr = grew ? ptx::ex2(m - m_use) : 1.f;

            const uint32_t tP = tS + kColPinS;
            const float2 sl2 = make_float2(sl, sl);
            const float2 nm2 = make_float2(-m_use, -m_use);
            float2 rowsum2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const int col = half * 64 + 2 * e;
                    const float2 sv = make_float2(__uint_as_float(sr[col >> 5][col & 31]),
                                                  __uint_as_float(sr[(col + 1) >> 5][(col + 1) & 31]));
                    const float2 arg = __ffma2_rn(sv, sl2, nm2);
                    const float p0 = ptx::ex2(arg.x), p1 = ptx::ex2(arg.y);
                    rowsum2 = __fadd2_rn(rowsum2, make_float2(p0, p1));
                    pk[e] = ptx::pack_bf16x2(p0, p1);
                }
                ptx::tmem_st32(tP + half * 32, pk);
            }
            // O's row moves to the new reference (never in the first step: its product
            // overwrites O); a warp goes together
            if (j > j0 && __any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    ptx::tmem_ld32(tO + c * 32, o);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                    ptx::tmem_st32(tO + c * 32, o);
                }
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            ptx::mbar_arrive(&p_full[t]);

            const float tile_sum = rowsum2.x + rowsum2.y;
            l = l * corr + tile_sum;
            // the tile's largest probability as the loop formed it, and in bf16
            const float p_top = ptx::ex2(fmaf(mx, sl, -m_use));
            const float p_top_bf16 = __uint_as_float(ptx::pack_bf16x2(p_top, 0.f) << 16);
            l_o = l_o * corr + (tile_sum + (p_top_bf16 - p_top));
            m = m_new;
        }

        // ---- epilogue ------------------------------------------------------------
        if constexpr (SPLIT) {
            // this CTA's part of its row; every CTA of the cluster is through with its ring
            bool ok = !aborted && (j1 <= j0 || ptx::mbar_wait(&o_full[t], 0, abort_flag, a.err_word));
            ptx::tc_fence_after_sync();
            ptx::cluster_sync();
            // Rows [owner * per, + per) are joined by CTA `owner`: it gets (m, l, l_o) and O
            // of each from every CTA.  A part's O lies by units of four values, the rows of
            // a unit one behind the other, so that a warp's stores fill whole lines (rows
            // one behind the other took twice as long).
            const int per = 2 * BM / n_split;
            constexpr uint32_t kOffParts = 2 * BM * 16;
            static_assert(kOffParts + 2 * BM * D * 4 <= C::kOffBar, "shared memory");
            {
                const int row = t * BM + r;
                const uint32_t to = ptx::cluster_addr(ptx::smem_u32(smem), uint32_t(row / per));
                const uint32_t at = to + kOffParts +
                                    uint32_t(part * per * (D / 4) + row % per) * 16;
                ptx::st_cluster4(to + uint32_t(part * per + row % per) * 16,
                            make_float4(m, l, l_o, ok ? 0.f : 1.f));
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (j1 > j0) {
                        ptx::tmem_ld32(tO + c * 32, o);
                        ptx::tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            o[q] = 0u;
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        ptx::st_cluster4(at + uint32_t((c * 8 + q) * per) * 16,
                                    make_float4(__uint_as_float(o[4 * q]),
                                                __uint_as_float(o[4 * q + 1]),
                                                __uint_as_float(o[4 * q + 2]),
                                                __uint_as_float(o[4 * q + 3])));
                }
            }
            ptx::cluster_sync();
            // eight rows and four units a warp at once: whole 32-byte sectors of O
            const float4 *st = reinterpret_cast<const float4 *>(smem);
            const int groups = per / 8;                    // of rows: 16, 8 or 4
            const int share = groups < 8 ? 8 / groups : 1; // warps of a group
            for (int rg = warp % (8 / share); rg < groups; rg += 8) {
                const int jr = rg * 8 + (lane & 7);
                const int gt = (part * per + jr) / BM, gr = (part * per + jr) % BM;
                const int gq = int(gr * p.div_g >> 16), gi = (gt ? i1 : i0) + gq;
                const int gh = hk * p.G + gr - gq * p.G;
                float M = -INFINITY, bad = 0.f, sum = 0.f, sum_o = 0.f;
                float f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < n_split) {
                        const float4 x = st[k * per + jr];
                        M = fmaxf(M, x.x);
                        bad += x.w;
                    }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    f[k] = 0.f;
                    if (k < n_split) {
                        const float4 x = st[k * per + jr];
                        f[k] = x.x == -INFINITY ? 1.f : ptx::ex2(x.x - M);   // (zeros, or NaN)
                        sum = fmaf(f[k], x.y, sum);
                        sum_o = fmaf(f[k], x.z, sum_o);
                    }
                }
                // (bad: a CTA's wait ran out)
                if (gq >= p.P || gi >= (gt ? i2 : i1) || bad != 0.f)
                    continue;
                const float inv = 1.f / sum_o;
                __nv_bfloat16 *orow = static_cast<__nv_bfloat16 *>(a.O) +
                                      ((sq.q0 + gi) * a.H + gh) * D;
                const float4 *parts = reinterpret_cast<const float4 *>(smem + kOffParts) + jr;
                for (int u = warp / (8 / share) * 4 + (lane >> 3); u < D / 4; u += 4 * share) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < n_split) {
                            const float4 y = parts[(k * (D / 4) + u) * per];
                            v.x = fmaf(f[k], y.x, v.x);
                            v.y = fmaf(f[k], y.y, v.y);
                            v.z = fmaf(f[k], y.z, v.z);
                            v.w = fmaf(f[k], y.w, v.w);
                        }
                    *reinterpret_cast<uint2 *>(orow + u * 4) =
                        sum == 0.f ? make_uint2(0, 0)
                                   : make_uint2(ptx::pack_bf16x2(v.x * inv, v.y * inv),
                                                ptx::pack_bf16x2(v.z * inv, v.w * inv));
                    if (u == 0)
                        a.lse[a.cu_seqlens_q != nullptr
                                  ? int64_t(gh) * a.total_q + sq.q0 + gi
                                  : (int64_t(b) * a.H + gh) * a.Nq + gi] =
                            sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
                }
            }
        }
        const int rows_t = t ? i2 - i1 : i1 - i0;      // queries of the tile
        if (!SPLIT && rows_t > 0) {
            const bool full_tile = rows_t == p.P;
            const bool work = j1 > j0;                 // else O was never formed: zeros
            const bool ok = !aborted &&
                            (!work || ptx::mbar_wait(&o_full[t], 0, abort_flag, a.err_word));
            uint8_t *o_stage = smem + t * C::kTileBytes;
            if (ok) {
                ptx::tc_fence_after_sync();
                // a row that sees no key: zeros (a NaN keeps its way)
                const float inv = l == 0.f ? 0.f : 1.f / l_o;
                __nv_bfloat16 *orow = static_cast<__nv_bfloat16 *>(a.O) +
                                      ((sq.q0 + i) * a.H + h) * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (work) {
                        ptx::tmem_ld32(tO + c * 32, o);
                        ptx::tmem_wait_ld();
                    }
                    uint4 v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t u[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            u[e] = work && l != 0.f
                                       ? ptx::pack_bf16x2(__uint_as_float(o[8 * q + 2 * e]) * inv,
                                                          __uint_as_float(o[8 * q + 2 * e + 1]) * inv)
                                       : 0u;
                        v[q] = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                    if (full_tile) {
                        uint8_t *rowp = o_stage + (c >> 1) * kChunkBytes + r * 128;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int u = (c & 1) * 4 + q;
                            *reinterpret_cast<uint4 *>(rowp + ((u ^ (r & 7)) << 4)) = v[q];
                        }
                    } else if (row_ok) {
                        uint4 *dst = reinterpret_cast<uint4 *>(orow + c * 32);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            dst[q] = v[q];
                    }
                }
                if (row_ok) {
                    const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                    a.lse[a.cu_seqlens_q != nullptr ? int64_t(h) * a.total_q + sq.q0 + i
                                                    : (int64_t(b) * a.H + h) * a.Nq + i] = lse;
                }
            }
            if (full_tile) {
                ptx::fence_proxy_async_smem();
                // the store goes out only if all 128 threads are through
                if (!ptx::bar_red_or(1 + t, 128, !ok) && r == 0) {
                    for (int c = 0; c < C::kChunks; c += p.q_chunks)
                        ptx::tma_store_5d(&p.tm_o, o_stage + c * kChunkBytes, 0, 0,
                                          int(sq.q0 + (t ? i1 : i0)), c, hk);
                    ptx::bulk_commit_and_wait_read();
                }
            }
        }
    }

    if (SPLIT && warp >= C::kWarpLoad) {              // the rows' warps wait twice above
        ptx::cluster_sync();
        ptx::cluster_sync();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    if (warp == C::kWarpMma)
        ptx::tmem_dealloc(tmem, C::kTmemCols);
}

template <int D, bool SPLIT, int TILES>
int launch_d(const Params &p, int64_t blocks, cudaStream_t stream)
{
    auto kern = attn_window_kernel<D, SPLIT, TILES>;
    static PerDeviceOnce once;
    constexpr int smem = int(Cfg<D, TILES>::kSmemBytes), kThreads = Cfg<D, TILES>::kThreads;
    if (!set_max_dynamic_smem(once, reinterpret_cast<const void *>(kern), smem))
        return FA_ERR_CUDA;
    const cudaError_t e =
        SPLIT ? launch_early_clusters(kern, dim3(unsigned(blocks)), kThreads, smem, p.split, stream, p)
              : launch_early(kern, dim3(unsigned(blocks)), kThreads, smem, stream, p);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// CTAs of an item.  They run one an SM, so what counts is waves of the SMs that clusters
// find (of 152; eight neighbours are not free everywhere), a step of an item taking some
// 1.5 us, its start and end 3.5, a join 8.5 more.  1 x 512 queries on a window of 4096, 64
// items: 56 us with one, 38 with two, 51 with four; 1 x 64, 8 items: 56, 37, 25, 19 with eight.
int choose_split(const WindowArgs &a, int P)
{
    const int64_t pairs = (a.total_q + 2 * P - 1) / (2 * P), most = (a.Nq + 2 * P - 1) / (2 * P);
    // packed sequences may all be short: at least the pairs that the rows need
    const int64_t items = (a.cu_seqlens_q != nullptr ? pairs : most * a.B) * a.Hkv;
    int64_t keys = int64_t(a.window) + a.sinks + 2 * P;
    keys = keys < a.Nk ? keys : a.Nk;
    const int64_t steps = (keys + BN - 1) / BN;
    int best = 1;
    double least = 0;
    for (int s = 1; s <= 8; s *= 2) {
        const int64_t sms = s <= 2 ? 152 : s == 4 ? 144 : 112;
        const double t = double((items * s + sms - 1) / sms) *
                         (1.5 * double((steps + s - 1) / s) + 3.5 + (s > 1 ? 8.5 : 0.));
        if (s == 1 || t < least) {
            best = s;
            least = t;
        }
    }
    return best;
}

// Tiles of a CTA.  With a narrow window a CTA has few steps, and its start and end (loads
// without a product, the way of O) weigh more than that two tiles share K and V: one tile
// then, two CTAs an SM (2 x 4096 tokens, d = 64, 16 heads: window 64 26 us against 34, 256
// 39 against 46, 512 49 against 54, 1024 65 and 66, 4096 113 against 109; 4 x 4096: 1024 117
// against 126, 4096 202 against 195; d = 128, 32 heads on 8: 64 51 against 64, 256 75 and 76,
// 512 95 and 95, 1024 133 against 128).
int choose_tiles(const WindowArgs &a)
{
    return a.window <= (a.d == 64 ? 1024 : 256) ? 1 : 2;
}

}  // namespace

int launch_attention_window(const WindowArgs &a, cudaStream_t stream)
{
    Params p;
    p.a = a;
    p.G = a.H / a.Hkv;
    p.P = BM / p.G;
    p.q_chunks = tmap_heads_chunks(p.G, a.d, p.P);
    p.div_g = uint32_t(65536 / p.G + 1);
    p.split = choose_split(a, p.P);
    const int tiles = p.split > 1 ? 2 : choose_tiles(a);
    p.grid = window_grid(a, tiles * p.P);
    p.scale_log2 = float(double(a.scale) * 1.4426950408889634);
    const int64_t blocks = window_items(a, p.grid) * p.split;
    const int64_t k_rows = a.total_k > 0 ? a.total_k : 1;      // (a map has a row at least)
    if (blocks > 0x7fffffffLL)
        return FA_ERR_TOO_LARGE;
    if (!make_tmap_heads(&p.tm_q, a.Q, a.total_q, a.Hkv, p.G, a.d, a.q_stride, p.P) ||
        !make_tmap_heads(&p.tm_o, a.O, a.total_q, a.Hkv, p.G, a.d, int64_t(a.H) * a.d, p.P) ||
        !make_tmap_heads(&p.tm_k, a.K, k_rows, a.Hkv, 1, a.d, a.k_stride, BN) ||
        !make_tmap_heads(&p.tm_v, a.V, k_rows, a.Hkv, 1, a.d, a.v_stride, BN) ||
        !make_tmap_heads(&p.tm_k32, a.K, k_rows, a.Hkv, 1, a.d, a.k_stride, kPad) ||
        !make_tmap_heads(&p.tm_v32, a.V, k_rows, a.Hkv, 1, a.d, a.v_stride, kPad))
        return FA_ERR_CUDA;
    if (p.split > 1)
        return a.d == 64 ? launch_d<64, true, 2>(p, blocks, stream)
                         : launch_d<128, true, 2>(p, blocks, stream);
    if (tiles == 1)
        return a.d == 64 ? launch_d<64, false, 1>(p, blocks, stream)
                         : launch_d<128, false, 1>(p, blocks, stream);
    return a.d == 64 ? launch_d<64, false, 2>(p, blocks, stream)
                     : launch_d<128, false, 2>(p, blocks, stream);
}

}  // namespace fa
