// attn_kv4_many.cu -- attention over the 4-bit paged cache for many query rows a kv
// head (chunks of prompts), on the tcgen05 tensor cores.
//
// attn_kv4.cu expands the codes anew for every 16 query rows and is bound by that;
// with hundreds of rows a kv head the products are what costs.  Here the cache's
// values are written out once, as fp16, and a kernel of the shape of attn_bf16.cu
// (two 128-row Q tiles a CTA, K and V tiles of 128 keys through a TMA ring, S, P
// and O in tensor memory) reads them: 4 sequences x 256 to 512 queries on 2k to 16k
// keys, 32 heads on 8, take 843 us with the one and 214 with the other, 44 of them
// for the copy (5.2 TB/s) and 15 for the join; with 1024 queries each on 16384 keys
// the whole takes 0.80 ms, 1.33 PFLOP/s, 0.71 of the measured cuBLAS rate.
//
// fp16 has 11 bits where min + scale * code needs up to 16: each value is rounded
// once, by 2^-11 of itself at most, after the power of two that brings the largest
// value of its tile (128 tokens of a head) into [2^13, 2^14).  Q is scaled per row
// likewise (8 bits: exact down to 2^-28 of the row's largest).  The tile's factors act
// on the scores and, for V, on P: with V = V^ 2^f and the reference m of
// S log2e + f, P^ = 2^(S log2e + f - m) <= 2^8 goes into P V^ as fp16 (times 2^7) and
// P = P^ 2^-f into the sum.
//
// A P of 0 does not keep a NaN of V from the sums: a group of a token whose V is not
// finite is written as 0, and each tile says which of its tokens is the first such one
// of each group.  A row sees a prefix of the keys, so that the epilogue knows from these
// whether the group's columns are NaN.
//
// The rows of a kv head are (query, head of the group) pairs, query by query, so
// that the heads of a group share K and V tiles; a row's mask goes by its query.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/fa.h"
#include "fa_error.cuh"
#include "kv4.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace fa {
namespace {

using kv4::bf16_hi;
using kv4::bf16_lo;
using kv4::pow2;

constexpr int BM = 128;              // query rows of a Q tile
constexpr int BN = 128;              // keys of a K/V tile
constexpr int kThreads = 320;
constexpr int kWarpLoad = 8;
constexpr int kWarpMma = 9;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColPinS = 64;    // P_t starts 64 columns into S_t
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kRescaleLog2 = 8.f;  // the reference lags by up to 2^8
// P^ goes to fp16 times 2^7, up to 2^15: a key keeps all bits down to 2^-21 of the row's
// largest P 2^f, where tiles with values far larger than its own would take them.
constexpr float kUp = 7.f, kDown = 0x1p-7f;
constexpr uint32_t kChunkBytes = BM * 128;
constexpr int kExpandThreads = 256;
constexpr int kNoNan = 255;          // of a tile's group

// e with 2^-e x in [2^13, 2^14), `least` at least.  For V -84: a sum of 2^31 P = P^ 2^-e
// <= 2^92 stays finite.  For Q and K -110: their factors stay normal numbers, and any
// bf16 number is 2^-16 at least.
constexpr int kLeastOfV = -84, kLeastOfQK = -110;
__device__ __forceinline__ int exponent_of(float x, int least)
{
    return x > 0.f ? max(least, min(114, int(__float_as_uint(x) >> 23) - 140)) : least;
}

// Sequence b's first query row, queries and keys; false (with the error recorded
// if `tell`) where they are not allowed.
struct Seq {
    int q0, nq, L;
};
__device__ __forceinline__ bool seq_of(const Kv4AttnArgs &a, int b, bool tell, Seq &s)
{
    s.q0 = b * a.Nq;
    s.nq = a.Nq;
    if (a.cu_seqlens_q != nullptr) {
        s.q0 = a.cu_seqlens_q[b];
        s.nq = a.cu_seqlens_q[b + 1] - s.q0;
    }
    s.L = a.seqlens[b];
    if (s.nq < 0 || s.nq > a.Nq || s.q0 < 0 || int64_t(s.q0) + s.nq > a.total_q || s.L < 0 ||
        s.L > a.Nk) {
        if (tell)
            record_device_error(a.err_word, FA_DEVERR_BAD_SEQLENS);
        return false;
    }
    return true;
}

// The values of 8 codes as fp16, rounded once: nibbles i and i + 4 as the pair
// 1024 + code, exact, less 1024, times scale plus min.
__device__ __forceinline__ uint4 values_of(uint32_t code, __half2 s, __half2 m)
{
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = ((code >> (4 * i)) & 0x000f000fu) | 0x64006400u;
        const __half2 c = __hsub2(*reinterpret_cast<const __half2 *>(&u), __float2half2_rn(1024.f));
        const __half2 y = __hfma2(s, c, m);
        v[i] = *reinterpret_cast<const uint32_t *>(&y);
    }
    return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                      __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

// Grid (tiles of the longest sequence, Hkv, B + some): block (j, h, b) writes the K
// and V tile of keys 128 j .. of head h of sequence b, zeros behind its end; the
// blocks with z >= B the queries.
template <int D, int G>
__global__ void __launch_bounds__(kExpandThreads, 4)
    kv4_expand_kernel(const Kv4AttnArgs a, const Kv4ManyBuffers w)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kCell = kv4::cell_bytes(D, G), NG = D / G, kN = D / 32, kLanes = D / 16;
    const int tid = threadIdx.x, lane = tid & 31, grp = a.H / a.Hkv;
    if (blockIdx.z >= unsigned(a.B)) {
        // queries: a warp a row of a head
        constexpr int kPer = D / 32;
        constexpr int kRows = kExpandThreads / 32;
        const int64_t all = a.total_q * a.H;
        const int64_t step = int64_t(gridDim.x) * gridDim.y * (gridDim.z - a.B) * kRows;
        const int64_t block = (int64_t(blockIdx.z - a.B) * gridDim.y + blockIdx.y) * gridDim.x +
                              blockIdx.x;
        for (int64_t x = block * kRows + tid / 32; x < all; x += step) {
            const int64_t tok = x / a.H;
            const int head = int(x - tok * a.H);
            const auto *src = static_cast<const __nv_bfloat16 *>(a.Q) + tok * a.q_stride +
                              int64_t(head) * D + lane * kPer;
            float q[kPer], big = 0.f;
#pragma unroll
            for (int e = 0; e < kPer; e += 2) {
                const uint32_t z = *reinterpret_cast<const uint32_t *>(src + e);
                q[e] = bf16_lo(z);
                q[e + 1] = bf16_hi(z);
                big = ptx::max3(big, fabsf(q[e]), fabsf(q[e + 1]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            const int e2 = big > 0.f ? exponent_of(big, kLeastOfQK) : 0;
            const float up = a.scale < 0.f ? -pow2(-e2) : pow2(-e2);   // q_mul is positive
            const int64_t row = ((head / grp) * a.total_q + tok) * grp + head % grp;
            auto *dst = reinterpret_cast<__half2 *>(w.Q + row * D + lane * kPer);
#pragma unroll
            for (int e = 0; e < kPer; e += 2)
                dst[e / 2] = __floats2half2_rn(q[e] * up, q[e + 1] * up);
            if (lane == 0)
                w.q_mul[row] = fabsf(a.scale) * kLog2e * pow2(e2);
        }
        return;
    }
    const int b = blockIdx.z, h = blockIdx.y, tok0 = blockIdx.x * BN;
    Seq seq;
    if (!seq_of(a, b, tid == 0 && h == 0 && blockIdx.x == 0, seq) || tok0 >= seq.L || seq.nq == 0)
        return;
    const int n = min(BN, seq.L - tok0);
    __shared__ const uint8_t *s_cell[BN / kv4::kCellTokens];
    __shared__ float s_big[2][kExpandThreads / 32];
    __shared__ int s_nan[4];           // a group's first token whose V is not finite
    if (tid < 4)
        s_nan[tid] = kNoNan;
    if (tid < BN / kv4::kCellTokens) {
        const int tok = tok0 + tid * kv4::kCellTokens;
        const uint8_t *cell = nullptr;
        if (tok < seq.L) {
            const int page = a.page_table[int64_t(b) * a.max_pages + tok / a.page_size];
            if (page >= 0 && page < a.num_pages)
                cell = static_cast<const uint8_t *>(a.cache) +
                       ((int64_t(page) * a.Hkv + h) * (a.page_size / kv4::kCellTokens) +
                        tok % a.page_size / kv4::kCellTokens) * kCell;
            else
                record_device_error(a.err_word, FA_DEVERR_BAD_PAGE);
        }
        s_cell[tid] = cell;
    }
    __syncthreads();
    // Everything that the thread converts is loaded first (the layout of
    // kv4_cache.cu: 16 values a thread, K then V), so that the largest magnitude
    // that the tile's parameters allow comes from registers.
    constexpr int kRounds = BN * kLanes / kExpandThreads;          // of K, and as many of V
    constexpr int kPairs = G == 32 ? 2 : 1;
    uint32_t code[2][kRounds][2], pair[2][kRounds][kPairs];
    float big[2] = {0.f, 0.f};
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int x = 0; x < kRounds; ++x) {
            const int l = tid % kLanes, t = tid / kLanes + x * (kExpandThreads / kLanes);
            const int jj = l / 4, c = l % 4;
            const uint8_t *cell = t < n ? s_cell[t / 16] : nullptr;
            code[kv][x][0] = code[kv][x][1] = 0;
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                pair[kv][x][i] = 0;
            if (cell == nullptr)
                continue;
            if (kv) {
                const uint8_t *from =
                    cell + kv4::v_off(D) + kv4::v_swizzle(t % 16 * (D / 2) + c * (kN * 4) + jj * 4);
                code[kv][x][0] = *reinterpret_cast<const uint32_t *>(from);
                code[kv][x][1] = *reinterpret_cast<const uint32_t *>(from + kN * 2);
            } else {
                const uint2 z = *reinterpret_cast<const uint2 *>(cell + t % 16 * (D / 2) +
                                                                 (c * kN + 2 * jj) * 4);
                code[kv][x][0] = z.x;
                code[kv][x][1] = z.y;
            }
            const auto *par = reinterpret_cast<const uint32_t *>(
                                  cell + (kv ? kv4::v_par_off(D, G) : kv4::k_par_off(D))) +
                              t % 16 * NG + (G == 32 ? 2 * jj : G == 64 ? jj : 0);
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                pair[kv][x][i] = par[i];
        }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
        for (int x = 0; x < kRounds; ++x)
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const uint32_t p = pair[kv][x][i];
                const float m = bf16_hi(p), top = fmaf(15.f, bf16_lo(p), m);
                if (fabsf(m) < INFINITY && bf16_lo(p) < INFINITY) {
                    // (the last of a group near the end of fp32's range may lie beyond it)
                    big[kv] = ptx::max3(big[kv], fabsf(m), fminf(fabsf(top), 3.4e38f));
                } else if (kv) {
                    const int jj = tid % kLanes / 4;
                    atomicMin(&s_nan[G == 32 ? 2 * jj + i : G == 64 ? jj : 0],
                              tid / kLanes + x * (kExpandThreads / kLanes));
                    pair[kv][x][i] = 0;
                }
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            big[kv] = fmaxf(big[kv], __shfl_xor_sync(0xffffffffu, big[kv], o));
        if (lane == 0)
            s_big[kv][tid / 32] = big[kv];
    }
    __syncthreads();
    const int64_t bh = int64_t(b) * a.Hkv + h;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        float top = s_big[kv][0];
#pragma unroll
        for (int i = 1; i < kExpandThreads / 32; ++i)
            top = fmaxf(top, s_big[kv][i]);
        const int e = exponent_of(top, kv ? kLeastOfV : kLeastOfQK);
        if (tid == 0) {
            uint2 &f = w.tile[bh * w.n_tiles + blockIdx.x];
            if (kv)
                f.y = __float_as_uint(float(e)) | uint32_t(s_nan[2] | s_nan[3] << 8);
            else
                f.x = __float_as_uint(pow2(e)) | uint32_t(s_nan[0] | s_nan[1] << 8);
        }
        const float up = pow2(-e);
#pragma unroll
        for (int x = 0; x < kRounds; ++x) {
            const int l = tid % kLanes, t = tid / kLanes + x * (kExpandThreads / kLanes);
            uint4 y[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t z = code[kv][x][i], other = code[kv][x][i ^ 1];
                // V: the halves of two stored words
                const uint32_t u = !kv ? z : i == 0 ? __byte_perm(z, other, 0x5410)
                                                    : __byte_perm(other, z, 0x7632);
                const uint32_t p = pair[kv][x][kPairs == 2 ? i : 0];
                y[i] = values_of(u, __float2half2_rn(bf16_lo(p) * up), __float2half2_rn(bf16_hi(p) * up));
            }
            __half *dst = (kv ? w.V : w.K) + (bh * w.n_tiles * BN + tok0 + t) * D +
                          (8 * (l / 4) + l % 4) * 8;
            *reinterpret_cast<uint4 *>(dst) = y[0];
            *reinterpret_cast<uint4 *>(dst + 32) = y[1];
        }
    }
}

template <int D>
struct Cfg {
    static constexpr int kChunks = D / 64;                           // 128-byte column chunks
    static constexpr uint32_t kTileBytes = BM * D * 2;               // a Q, K or V tile
    static constexpr int kStages = D == 128 ? 4 : 8;                 // K/V ring depth
    static constexpr uint32_t kOffRing = 2 * kTileBytes;
    static constexpr uint32_t kOffBar = kOffRing + kStages * kTileBytes;
    static constexpr uint32_t kBarBytes = 8 * (2 + 2 * kStages + 2 + 2 + 2 + 1 + 1);
    static constexpr uint32_t kSmemBytes = kOffBar + kBarBytes + 16 + 1024;  // +1024 align slack
};

struct ManyParams {
    CUtensorMap tm_q, tm_k, tm_v;    // fp16 rows of d values, box {64, 1, 128}
    Kv4AttnArgs a;
    Kv4ManyBuffers w;
    int n_pairs;                     // pairs of Q tiles of the longest run of queries
};

__device__ __forceinline__ uint32_t col_s(int t) { return uint32_t(t) * 128u; }
template <int D>
__device__ __forceinline__ uint32_t col_o(int t) { return 256u + uint32_t(t) * D; }

// fp16 operands: format code 0 where bf16 has 1
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, bool b_mn_major)
{
    return ptx::idesc_bf16_f32(M, N, b_mn_major) & ~((1u << 7) | (1u << 10));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Bounded wait while draining after an abort: ignores the abort flag.
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t it = 0; it < kWaitMaxPolls; ++it) {
        if (ptx::mbar_try_wait(bar, parity))
            return;
        if ((it & 255u) == 255u && ptx::globaltimer() - t0 > kWaitTimeoutNs)
            return;
    }
}

// The x-th longest sequence of up to 32 (of more, the x-th): the CTAs with the most
// work come first (32 x 256 queries on 300 to 8000 keys 456 us, in the order of the
// batch 490; equal lengths lose half a per cent).
__device__ __forceinline__ int by_length(const Kv4AttnArgs &a, int x)
{
    if (a.B == 1 || a.B > 32)
        return x;
    const int lane = threadIdx.x & 31, mine = lane < a.B ? a.seqlens[lane] : -1;
    int rank = 0;
    for (int i = 0; i < a.B; ++i) {
        const int other = __shfl_sync(0xffffffffu, mine, i);
        rank += other > mine || (other == mine && i < lane);
    }
    return __ffs(__ballot_sync(0xffffffffu, lane < a.B && rank == x)) - 1;
}

// The roles, the order of the products and the layout of tensor memory are those
// of attn_bf16.cu.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kv4_many_kernel(const __grid_constant__ ManyParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *q_full = bars, *kv_full = bars + 2, *kv_empty = kv_full + C::kStages,
             *s_full = kv_empty + C::kStages, *p_full = s_full + 2, *o_full = p_full + 2,
             *drain = o_full + 2,
             *never = drain + 1;      // nothing arrives: the failure-detection test waits here
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + (C::kBarBytes / 8));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    // ---- work item: (sequence, kv head, range of p.w.chunk key tiles, pair of Q
    //      tiles), the pairs side by side: they read the same K and V tiles (with the
    //      pairs apart, 4 x 512 queries on 16k keys took 240 us, so 214) --------------
    const Kv4AttnArgs &a = p.a;
    const int grp = a.H / a.Hkv;
    const int rest = int(blockIdx.x) / p.n_pairs, px = int(blockIdx.x) % p.n_pairs;
    const int pair = p.n_pairs - 1 - px;   // the heaviest of a causal run first
    const int split = rest % p.w.splits, h = rest / p.w.splits % a.Hkv;
    const int b = by_length(a, rest / p.w.splits / a.Hkv), bh = b * a.Hkv + h;
    Seq seq;
    if (!seq_of(a, b, false, seq))
        return;                                // the expanding kernel has told
    const int rows = seq.nq * grp, qt0 = 2 * pair;
    if (qt0 * BM >= rows)
        return;
    const int n_kv = (seq.L + BN - 1) / BN;
    // keys that row x sees lie at or below last_key(x)
    auto last_key = [&](int x) {
        return a.causal ? min(seq.L, seq.L - seq.nq + x / grp + 1) - 1 : seq.L - 1;
    };
    auto tiles_seen = [&](int qt) {
        if (qt * BM >= rows)
            return 0;
        const int last = last_key(min(rows, (qt + 1) * BM) - 1);
        return last < 0 ? 0 : min(n_kv, last / BN + 1);
    };
    const int all0 = tiles_seen(qt0), all1 = tiles_seen(qt0 + 1);
    const int all = all0 > all1 ? all0 : all1, j0 = split * p.w.chunk;
    if (split > 0 && j0 >= all)
        return;
    const bool parts = all > p.w.chunk;        // the item has further ranges
    const int n0 = max(0, min(all0 - j0, p.w.chunk)), n1 = max(0, min(all1 - j0, p.w.chunk));
    const int n_max = n0 > n1 ? n0 : n1;

    auto store_lse = [&](int x, float lse) {
        const int i = x / grp, head = h * grp + x % grp;
        a.lse[a.cu_seqlens_q ? int64_t(head) * a.total_q + seq.q0 + i
                             : (int64_t(b) * a.H + head) * a.Nq + i] = lse;
    };
    auto out_row = [&](int x) {
        return static_cast<__nv_bfloat16 *>(a.O) +
               (int64_t(seq.q0 + x / grp) * a.H + h * grp + x % grp) * D;
    };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        ptx::mbar_init(&q_full[0], 1);
        ptx::mbar_init(&q_full[1], 1);
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(&kv_full[s], 1);
            ptx::mbar_init(&kv_empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(&s_full[t], 1);
            ptx::mbar_init(&p_full[t], 128);
            ptx::mbar_init(&o_full[t], 1);
        }
        ptx::mbar_init(drain, 1);
        ptx::mbar_init(never, 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
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
    uint8_t *q_smem[2] = {smem, smem + C::kTileBytes}, *ring = smem + C::kOffRing;

    if (warp == kWarpLoad) {
        // ======================= TMA producer ==============================
        if (lane == 0 && n_max > 0) {
            int last_phase[C::kStages];
            for (int s = 0; s < C::kStages; ++s)
                last_phase[s] = -1;
            bool q_issued[2] = {false, false};
            const int q_row = int((int64_t(h) * a.total_q + seq.q0) * grp);
            const int k_row = (bh * p.w.n_tiles + j0) * BN;
            auto load_q = [&](int t) {
                q_issued[t] = true;
                ptx::mbar_arrive_expect_tx(&q_full[t], C::kTileBytes);
                for (int c = 0; c < C::kChunks; ++c)
                    ptx::tma_load_3d(q_smem[t] + c * kChunkBytes, &p.tm_q, &q_full[t], c * 64, 0,
                                     q_row + (qt0 + t) * BM);
            };
            if (n0 > 0)
                load_q(0);
            int stage = 0;
            uint32_t phase = 0;
            for (int j = 0; j < n_max && !aborted; ++j) {
                for (int kv = 0; kv < 2; ++kv) {
                    if (!ptx::mbar_wait(&kv_empty[stage], phase ^ 1u, abort_flag, a.err_word)) {
                        aborted = true;
                        break;
                    }
                    ptx::mbar_arrive_expect_tx(&kv_full[stage], C::kTileBytes);
                    for (int c = 0; c < C::kChunks; ++c)
                        ptx::tma_load_3d(ring + stage * C::kTileBytes + c * kChunkBytes,
                                         kv ? &p.tm_v : &p.tm_k, &kv_full[stage], c * 64, 0,
                                         k_row + j * BN);
                    last_phase[stage] = int(phase);
                    if (++stage == C::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (j == 0 && kv == 0 && n1 > 0)
                        load_q(1);
                }
            }
            // Every copy issued lands before the CTA goes away, also where another
            // warp gives up after this one is through.
            for (int t = 0; t < 2; ++t)
                if (q_issued[t])
                    drain_wait(&q_full[t], 0);
            for (int s = 0; s < C::kStages; ++s)
                if (last_phase[s] >= 0)
                    drain_wait(&kv_full[s], uint32_t(last_phase[s]));
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        // ======================= MMA issuer (whole warp) =====================
        constexpr uint32_t idesc_qk = idesc_f16(BM, BN, false), idesc_pv = idesc_f16(BM, D, true);
        constexpr uint64_t desc_kmajor = ptx::smem_desc_base(16, 1024);
        constexpr uint64_t desc_mnmajor = ptx::smem_desc_base(kChunkBytes, 1024);
        const uint64_t dq[2] = {ptx::smem_desc(desc_kmajor, ptx::smem_u32(q_smem[0])),
                                ptx::smem_desc(desc_kmajor, ptx::smem_u32(q_smem[1]))};
        const uint32_t ring_addr = ptx::smem_u32(ring);
        auto issue_qk = [&](int t, uint64_t dk) {
            const uint32_t ts = tmem + col_s(t);
            if (ptx::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t off = ((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4;
                    ptx::mma_ss(ts, (t == 0 ? dq[0] : dq[1]) + off, dk + off, idesc_qk,
                                kk > 0 ? 1u : 0u);
                }
                ptx::mma_commit(&s_full[t]);
            }
            __syncwarp();
        };
        auto issue_pv = [&](int t, uint64_t dv, bool accumulate) {
            const uint32_t to = tmem + col_o<D>(t), tp = tmem + col_s(t) + kColPinS;
            if (ptx::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                    ptx::mma_ts(to, tp + kk * 8, dv + uint64_t((kk * 16 * 128) >> 4), idesc_pv,
                                (accumulate || kk > 0) ? 1u : 0u);
            }
            __syncwarp();
        };
        auto commit = [&](uint64_t *bar) {
            if (ptx::elect_one())
                ptx::mma_commit(bar);
            __syncwarp();
        };
        int stage = 0;
        uint32_t phase = 0;
        auto next_stage = [&](uint64_t &dk, uint64_t &dv) -> bool {
            if (!ptx::mbar_wait_warp(&kv_full[stage], phase, abort_flag, a.err_word))
                return false;
            const uint32_t addr = ring_addr + stage * C::kTileBytes;
            dk = ptx::smem_desc(desc_kmajor, addr);
            dv = ptx::smem_desc(desc_mnmajor, addr);
            return true;
        };
        auto advance = [&]() {
            if (++stage == C::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        };
        auto p_ready = [&](int t, int j) {
            const bool ok = ptx::mbar_wait_warp(&p_full[t], uint32_t(j) & 1u, abort_flag, a.err_word);
            if (ok)
                ptx::tc_fence_after_sync();
            return ok;
        };
        // Failure-detection test: in the first CTA of the longest sequence's first head a
        // wait on a barrier that nothing arrives at runs out.
        if (a.expire_wait_ns != 0u && rest == 0 && pair == 0)
            aborted = !__all_sync(0xffffffffu, ptx::mbar_wait_limited(never, 0, abort_flag, a.err_word,
                                                                      a.expire_wait_ns));
        if (n_max > 0 && !aborted) do {
            uint64_t k_desc, v_desc, unused;
            if (!next_stage(k_desc, unused))
                break;
            int k_stage = stage;
            advance();
            bool ok = true;
            for (int t = 0; t < 2 && ok; ++t) {
                if ((t == 0 ? n0 : n1) == 0)
                    continue;
                ok = ptx::mbar_wait_warp(&q_full[t], 0, abort_flag, a.err_word);
                if (ok) {
                    ptx::tc_fence_after_sync();
                    issue_qk(t, k_desc);
                }
            }
            if (!ok)
                break;
            commit(&kv_empty[k_stage]);
            for (int j = 0; j < n_max; ++j) {
                if (!next_stage(unused, v_desc))
                    break;
                const int v_stage = stage;
                advance();
                if (j < n0) {
                    if (!p_ready(0, j))
                        break;
                    issue_pv(0, v_desc, j > 0);
                    if (j == n0 - 1)
                        commit(&o_full[0]);
                }
                const bool more = j + 1 < n_max;
                if (more) {
                    if (!next_stage(k_desc, unused))
                        break;
                    k_stage = stage;
                    advance();
                    ptx::tc_fence_after_sync();
                    if (j + 1 < n0)
                        issue_qk(0, k_desc);
                }
                if (j < n1) {
                    if (!p_ready(1, j))
                        break;
                    issue_pv(1, v_desc, j > 0);
                    if (j == n1 - 1)
                        commit(&o_full[1]);
                }
                commit(&kv_empty[v_stage]);
                if (more) {
                    if (j + 1 < n1)
                        issue_qk(1, k_desc);
                    commit(&kv_empty[k_stage]);
                }
            }
        } while (false);
        // every MMA issued has completed once this last commit arrives
        if (ptx::elect_one()) {
            ptx::mma_commit(drain);
            drain_wait(drain, 0);
        }
        __syncwarp();
    } else {
        // ======================= softmax warpgroups ========================
        const int t = warp >> 2, r = threadIdx.x & 127;
        const int n_t = t == 0 ? n0 : n1, qt = qt0 + t, x = qt * BM + r;
        const bool row_ok = x < rows;
        const uint32_t lane_bits = uint32_t((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_bits + col_s(t), tO = tmem + lane_bits + col_o<D>(t);
        const int tile0 = bh * p.w.n_tiles + j0;
        const float sl = row_ok
            ? p.w.q_mul[(int64_t(h) * a.total_q + seq.q0) * grp + x] : 0.f;
        // relative to the range's first key
        const int last = last_key(x) - j0 * BN, last_first = last_key(qt * BM) - j0 * BN;
        float m = -INFINITY, l = 0.f;

        for (int j = 0; j < n_t; ++j) {
            // (a factor of 0 would make NaN of the mask's -inf, one of inf of a score of 0)
            const uint2 both = p.w.tile[tile0 + j];
            const float2 factor = make_float2(bf16_hi(both.x), bf16_hi(both.y));
            const float slj = fminf(fmaxf(sl * factor.x, 1.2e-38f), 3e38f);
            float f = factor.y;
            // |raw scores| are below 2^28 d: scores beyond 2^18 are possible
            const bool large = slj > 0x1p-10f / D;
            const bool any_large = __any_sync(0xffffffffu, large);
            // (the warp gives up as one: votes and aligned loads follow)
            if (!ptx::mbar_wait_warp(&s_full[t], uint32_t(j) & 1u, abort_flag, a.err_word)) {
                aborted = true;
                break;
            }
            ptx::tc_fence_after_sync();
            uint32_t sr[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                ptx::tmem_ld32(tS + c * 32, sr[c]);
            ptx::tmem_wait_ld();
            if (any_large || j * BN + BN - 1 > last_first) {
                const int lim = last - j * BN;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e > lim)
                            sr[c][e] = __float_as_uint(-INFINITY);
                if (any_large) {
                    // The rounding of the reference would show in P, and from 2^40 on make
                    // infinities: such a row's scores go by their distance to the largest.
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            top = fmaxf(top, __uint_as_float(sr[c][e]));
                    top = large && fabsf(top) < INFINITY ? top : 0.f;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            sr[c][e] = __float_as_uint(__uint_as_float(sr[c][e]) - top);
                    f = fmaf(top, slj, f);
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
            const float mt = fmaf(mx, slj, f);
            const bool grew = mt > m + kRescaleLog2;
            const float m_new = grew ? mt : m;
            const float m_use = m_new == -INFINITY ? 0.f : m_new;
            const float corr = grew ? ptx::ex2(m - m_use) : 1.f;   // 0 on the first tile
            const uint32_t tP = tS + kColPinS;
            const float2 sl2 = make_float2(slj, slj), nm2 = make_float2(f - m_use + kUp, f - m_use + kUp);
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
                    pk[e] = pack_f16x2(p0, p1);
                }
                ptx::tmem_st32(tP + half * 32, pk);
            }
            if (j > 0 && __any_sync(0xffffffffu, grew)) {
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
            l = l * corr + (rowsum2.x + rowsum2.y) * ptx::ex2(-factor.y - kUp);
            m = m_new;
        }

        // Each group's first key whose V is not finite, relative to the range's first key:
        // the columns of a row that sees it are NaN.
        int first_nan[4] = {INT_MAX, INT_MAX, INT_MAX, INT_MAX};
        for (int j = lane; j < n_t; j += 32) {
            const uint2 both = p.w.tile[tile0 + j];
            const uint32_t z = __byte_perm(both.x, both.y, 0x5410);
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if ((z >> (8 * y) & 255u) != kNoNan)
                    first_nan[y] = min(first_nan[y], j * BN + int(z >> (8 * y) & 255u));
        }
        float keep[D / 32];                // of 32 columns: 1 or NaN
#pragma unroll
        for (int y = 0; y < 4; ++y)
            first_nan[y] = __reduce_min_sync(0xffffffffu, first_nan[y]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const int y = c * 32 / a.group;
            const int at = y == 0 ? first_nan[0] : y == 1 ? first_nan[1]
                           : y == 2 ? first_nan[2] : first_nan[3];
            keep[c] = at <= last ? NAN : 1.f;
        }

        // ---- epilogue: O = O~ / l (bf16), lse = (m + log2 l) ln 2 --------------------
        const int64_t part = int64_t(split) * a.total_q * a.H +
                             (int64_t(h) * a.total_q + seq.q0) * grp + x;
        if (n_t == 0) {
            if (row_ok && parts) {
                p.w.ml[part] = make_float2(-INFINITY, 0.f);
            } else if (row_ok) {
                uint4 *dst = reinterpret_cast<uint4 *>(out_row(x));
#pragma unroll
                for (int q = 0; q < D / 8; ++q)
                    dst[q] = make_uint4(0, 0, 0, 0);
                store_lse(x, -INFINITY);
            }
        } else if (!aborted && ptx::mbar_wait_warp(&o_full[t], 0, abort_flag, a.err_word)) {
            ptx::tc_fence_after_sync();
            const bool any = l > 0.f || l != l;
            const float all_inv = any ? kDown / l : 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const float inv = all_inv * keep[c];
                uint32_t o[32];
                ptx::tmem_ld32(tO + c * 32, o);
                ptx::tmem_wait_ld();
                if (!row_ok)
                    continue;
                if (parts) {
                    float4 *dst = reinterpret_cast<float4 *>(p.w.O_part + part * D + c * 32);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        dst[q] = make_float4(__uint_as_float(o[4 * q + 0]) * keep[c],
                                             __uint_as_float(o[4 * q + 1]) * keep[c],
                                             __uint_as_float(o[4 * q + 2]) * keep[c],
                                             __uint_as_float(o[4 * q + 3]) * keep[c]);
                    continue;
                }
                uint4 *dst = reinterpret_cast<uint4 *>(out_row(x) + c * 32);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint4 y;
                    y.x = ptx::pack_bf16x2(__uint_as_float(o[8 * q + 0]) * inv,
                                           __uint_as_float(o[8 * q + 1]) * inv);
                    y.y = ptx::pack_bf16x2(__uint_as_float(o[8 * q + 2]) * inv,
                                           __uint_as_float(o[8 * q + 3]) * inv);
                    y.z = ptx::pack_bf16x2(__uint_as_float(o[8 * q + 4]) * inv,
                                           __uint_as_float(o[8 * q + 5]) * inv);
                    y.w = ptx::pack_bf16x2(__uint_as_float(o[8 * q + 6]) * inv,
                                           __uint_as_float(o[8 * q + 7]) * inv);
                    dst[q] = y;
                }
            }
            if (row_ok && parts)
                p.w.ml[part] = make_float2(m, l);
            else if (row_ok)
                store_lse(x, any ? (m + log2f(l)) * kLn2 : -INFINITY);
        } else if (row_ok && parts) {
            p.w.ml[part] = make_float2(0.f, -1.f);     // a wait ran out: no such part
        }
    }

    // ---- teardown ------------------------------------------------------------
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    if (warp == kWarpMma)
        ptx::tmem_dealloc(tmem, kTmemCols);
}

// Joins the ranges of the items that have several, in their order: block (x, y)
// takes every eighth eight rows of item x, a warp a row.  Rows that lack a part (its
// sum is negative: a wait ran out) stay as they were.
template <int D>
__global__ void __launch_bounds__(kExpandThreads) kv4_many_join_kernel(const ManyParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Kv4AttnArgs &a = p.a;
    const int grp = a.H / a.Hkv, bh = int(blockIdx.x) % (a.B * a.Hkv), b = bh / a.Hkv, h = bh % a.Hkv;
    Seq seq;
    if (!seq_of(a, b, false, seq))
        return;
    const int rows = seq.nq * grp, x0 = int(blockIdx.x) / (a.B * a.Hkv) * 2 * BM;
    const int x1 = min(rows, x0 + 2 * BM), lane = threadIdx.x & 31;
    if (x0 >= x1)
        return;
    const int last = a.causal ? min(seq.L, seq.L - seq.nq + (x1 - 1) / grp + 1) : seq.L;
    const int n = (((last + BN - 1) / BN) + p.w.chunk - 1) / p.w.chunk;
    if (last <= 0 || n <= 1)
        return;
    constexpr int kPer = D / 32;
    for (int x = x0 + int(blockIdx.y * kExpandThreads + threadIdx.x) / 32; x < x1;
         x += int(gridDim.y) * (kExpandThreads / 32)) {
        const int64_t row = (int64_t(h) * a.total_q + seq.q0) * grp + x, step = a.total_q * a.H;
        float m = -INFINITY, l = 0.f, y[kPer];
        bool lacks = false;
        for (int s = 0; s < n; ++s) {
            const float2 ml = p.w.ml[s * step + row];
            m = fmaxf(m, ml.x);
            lacks = lacks || ml.y < 0.f;
        }
        if (lacks)
            continue;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            y[e] = 0.f;
        for (int s = 0; s < n; ++s) {
            const float2 ml = p.w.ml[s * step + row];
            if (ml.y == 0.f)                   // nothing seen
                continue;
            const float f = ptx::ex2(ml.x - m);
            l = fmaf(ml.y, f, l);
            const float *src = p.w.O_part + (s * step + row) * D + lane * kPer;
#pragma unroll
            for (int e = 0; e < kPer; e += 2) {
                const float2 z = *reinterpret_cast<const float2 *>(src + e);
                y[e] = fmaf(z.x, f, y[e]);
                y[e + 1] = fmaf(z.y, f, y[e + 1]);
            }
        }
        const bool any = l > 0.f || l != l;
        const float inv = any ? kDown / l : 0.f;
        const int i = x / grp, head = h * grp + x % grp;
        auto *dst = static_cast<__nv_bfloat16 *>(a.O) + (int64_t(seq.q0 + i) * a.H + head) * D +
                    lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; e += 2)
            *reinterpret_cast<uint32_t *>(dst + e) = ptx::pack_bf16x2(y[e] * inv, y[e + 1] * inv);
        if (lane == 0)
            a.lse[a.cu_seqlens_q ? int64_t(head) * a.total_q + seq.q0 + i
                                 : (int64_t(b) * a.H + head) * a.Nq + i] =
                any ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
}

template <int D, int G>
int launch(const Kv4AttnArgs &a, cudaStream_t stream)
{
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const Kv4ManyLayout at = kv4_many_layout(a.B, a.total_q, a.Nk, a.H, a.Hkv, D);
    ManyParams p;
    p.a = a;
    p.w.Q = reinterpret_cast<__half *>(ws + at.q);
    p.w.K = reinterpret_cast<__half *>(ws + at.k);
    p.w.V = reinterpret_cast<__half *>(ws + at.v);
    p.w.q_mul = reinterpret_cast<float *>(ws + at.q_mul);
    p.w.tile = reinterpret_cast<uint2 *>(ws + at.tile);
    p.w.O_part = reinterpret_cast<float *>(ws + at.O_part);
    p.w.ml = reinterpret_cast<float2 *>(ws + at.ml);
    p.w.n_tiles = at.n_tiles;
    p.w.splits = at.splits;
    p.w.chunk = at.chunk;
    const int64_t k_rows = int64_t(a.B) * a.Hkv * at.n_tiles * BN;
    if (!make_tmap_bf16(&p.tm_q, p.w.Q, a.total_q * a.H, 1, D) ||
        !make_tmap_bf16(&p.tm_k, p.w.K, k_rows, 1, D) || !make_tmap_bf16(&p.tm_v, p.w.V, k_rows, 1, D))
        return FA_ERR_CUDA;
    const int64_t rows = int64_t(a.Nq) * (a.H / a.Hkv);
    p.n_pairs = int((rows + 2 * BM - 1) / (2 * BM));
    const int64_t items = int64_t(p.n_pairs) * a.B * a.Hkv, blocks = items * at.splits;
    if (blocks > 0x7fffffffLL)
        return FA_ERR_TOO_LARGE;
    // about four rows of Q a warp
    const int64_t per_layer = int64_t(at.n_tiles) * a.Hkv * (kExpandThreads / 32) * 4;
    const int64_t layers = (a.total_q * a.H + per_layer - 1) / per_layer;
    const dim3 grid(at.n_tiles, a.Hkv, unsigned(a.B + (layers < 1024 ? layers : 1024)));
    if (launch_early(kv4_expand_kernel<D, G>, grid, kExpandThreads, 0, stream, a, p.w) != cudaSuccess)
        return FA_ERR_CUDA;
    auto kern = attn_kv4_many_kernel<D>;
    static PerDeviceOnce once;
    if (!set_max_dynamic_smem(once, reinterpret_cast<const void *>(kern), int(Cfg<D>::kSmemBytes)))
        return FA_ERR_CUDA;
    cudaError_t e = launch_early(kern, dim3(unsigned(blocks)), kThreads, int(Cfg<D>::kSmemBytes),
                                 stream, p);
    if (e == cudaSuccess && at.splits > 1)
        e = launch_early(kv4_many_join_kernel<D>, dim3(unsigned(items), 8), kExpandThreads, 0, stream,
                         p);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

int launch_attention_kv4_many(const Kv4AttnArgs &a, cudaStream_t stream)
{
    if (a.d == 64)
        return a.group == 32 ? launch<64, 32>(a, stream) : launch<64, 64>(a, stream);
    return a.group == 32   ? launch<128, 32>(a, stream)
           : a.group == 64 ? launch<128, 64>(a, stream)
                           : launch<128, 128>(a, stream);
}

}  // namespace fa
