// attn_kv4.cu -- attention over the 4-bit paged cache (kv4.cuh, include/fa.h).
//
// With k_j = mK_j + sK_j u_j and v_j = mV_j + sV_j w_j (u, w the codes 0..15, s
// and m per token and group of the head dimension):
//     S_ij = scale * sum_g ( sK_jg * sum_{k in g} q_ik u_jk + mK_jg * Qbar_ig ),
//     Qbar_ig = sum_{k in g} q_ik,
//     O_ik = sum_j (P_ij sV_jg) w_jk + sum_j P_ij mV_jg        (k in group g),
// so the codes go into the matrix products as they are and the scales act on
// the small results: nothing is dequantised.
//
// A code as an fp16 number costs one logical operation for two values: the
// nibble u at the low end of a half-word IS the subnormal u * 2^-24, and the
// nibble above it 16 u * 2^-24 (fp16 is linear up to 2^11 units of 2^-24).  The
// matrix instructions take subnormals exactly; 2^24 and the 16 go into Q and
// the epilogue.  Q is scaled per row by a power of two into fp16's range, so
// its 8 bits are exact down to 2^-26 of the row's largest value.  P s is
// rounded to fp16 (2^-11), against 2^-8 for bf16.
//
// Layout: keys are the rows (M = 16 tokens), query rows (query, head of the
// group) the columns (N = 8) of mma.m16n8k16, S^T = K Q^T and O^T = V^T P^T, so
// that a decode step with up to 8 heads a kv head wastes nothing.  tcgen05 has
// M = 64 at least and takes its operands from shared or tensor memory: the
// codes would be expanded fourfold into shared memory first, which costs more
// than the products.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/fa.h"
#include "kv4.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlock = kWarps * kv4::kCellTokens;   // tokens of a block: a cell each warp
constexpr float kNoRef = -1e30f;   // reference of a row that has seen no key: exp2(-inf - kNoRef) = 0
// A row's reference is max(S + log2 w), w the weight of a key's V parameters, so
// that P s <= 1 in fp16 whatever the scales are; it may lag by a factor of 16.
// w >= 2^-92 keeps P <= 2^96 and the sum of 2^31 of them finite.
constexpr float kLag = 16.f;
constexpr float kLeastWeight = 0x1p-92f;

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same on a zero accumulator.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float max3(float x, float y, float z)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// N words of shared memory at address `at` + OFF.  Volatile: the ring's contents
// change, and the queries' fragments are read again each time rather than held.
template <int OFF, int N>
__device__ __forceinline__ void load_shared(uint32_t (&w)[N], uint32_t at)
{
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at), "n"(OFF));
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];"
                     : "=r"(w[0]), "=r"(w[1])
                     : "r"(at), "n"(OFF));
    else
        asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(w[0]) : "r"(at), "n"(OFF));
}

// Lane `mine` of the warp: arrives at the cell's barrier and starts its copy; with
// no source it only arrives.
template <int BYTES>
__device__ __forceinline__ void copy_cell(uint32_t bar, uint32_t to, const uint8_t *src, bool mine)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b32 n;\n\t"
                 "setp.ne.u32 p, %3, 0;\n\t"
                 "setp.ne.and.u64 q, %2, 0, p;\n\t"
                 "selp.b32 n, %4, 0, q;\n\t"
                 "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], n;\n\t"
                 "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%2], "
                 "%4, [%0];\n\t}"
                 ::"r"(bar), "r"(to), "l"(src), "r"(uint32_t(mine)), "n"(BYTES)
                 : "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Cells on their way or in use: each warp keeps a ring of its own, one bulk copy
// a cell, no barrier between warps.  Two CTAs an SM with 4 cells of 2304 bytes a
// warp have up to 147 KB in flight, against the 36 KB that cover HBM's latency at
// full rate.
constexpr int kStages = 4;

// A work item is (sequence, kv head, tile of R query rows); its keys are cut
// into blocks of kBlock tokens.  All items' blocks, sequence by sequence, form
// one line that is cut into equal ranges, one a CTA: ragged batches and single
// long sequences fill the GPU alike, and nothing of it needs the host.
struct Desc {          // of an item that begins in this CTA's range and does not end there
    int parts;         // CTAs that hold a part (0: no such item)
    int b, kvh, tile;
};

// Workspace: Desc[kMaxCtas], then (reference, sum) [2 kMaxCtas][R], then
// the unnormalised O [2 kMaxCtas][R][d] fp32.  A CTA's slot 0 holds the part of
// an item that began before its range, slot 1 that of one that goes on after.
struct Parts {
    Desc *desc;
    float2 *ml;
    float *O;
};

template <int R>
__host__ __device__ inline Parts parts_of(void *ws)
{
    Parts p;
    p.desc = static_cast<Desc *>(ws);
    p.ml = reinterpret_cast<float2 *>(p.desc + kKv4MaxCtas);
    p.O = reinterpret_cast<float *>(p.ml + 2 * kKv4MaxCtas * R);
    return p;
}

// Blocks of a sequence: its items have one at least, so that a row without a
// key is written too.
__device__ __forceinline__ int blocks_of(int L) { return L <= 0 ? 1 : (L + kBlock - 1) / kBlock; }

// Sequence b's first query row and query count, or a count of 0 (with the
// error recorded) where its lengths are not allowed.
__device__ __forceinline__ int2 queries_of(const Kv4AttnArgs &a, int b)
{
    if (a.cu_seqlens_q == nullptr)
        return make_int2(b * a.Nq, a.Nq);
    const int c0 = a.cu_seqlens_q[b], n = a.cu_seqlens_q[b + 1] - c0;
    return make_int2(c0, n);
}

// A tile's queries in shared memory.
template <int D, int G, int NT>
struct alignas(16) QueryTile {
    uint4 frag[NT][D / 32][32];    // B fragments of two k-steps, lane by lane
    float bar[D / G][8 * NT];      // scale log2e * (sum of the row's values in the group)
    float mul[8 * NT];             // scale log2e * 2^24 / (the row's power of two)
    int end[8 * NT];               // the keys that the row sees lie below this
};

template <int D, int G, int NT>
struct Shared {
    static constexpr int R = 8 * NT;
    static constexpr int ring = 0;                                   // [kWarps][kStages] cells
    static constexpr int q = ring + kWarps * kStages * kv4::cell_bytes(D, G);  // [2] QueryTile
    static constexpr int O = q + 2 * int(sizeof(QueryTile<D, G, NT>));  // [kWarps / 2][8][D + 4]
    static constexpr int full = O + kWarps / 2 * 8 * (D + 4) * 4;    // [kWarps][kStages] barriers
    static constexpr int pre = full + kWarps * kStages * 8;          // [B + 1] blocks before b
    static constexpr int len = pre + (kKv4MaxSeqs + 4) * 4;          // [B] keys
    static constexpr int ref = len + kKv4MaxSeqs * 4;                // [kWarps][R]
    static constexpr int sum = ref + kWarps * R * 4;                 // [kWarps][R]
    static constexpr int bytes = sum + kWarps * R * 4;
};

// Where block x of the line is.
struct Item {
    int b, q0, nq, L;      // sequence, its first query row, queries, keys
    int kvh, tile;
    uint32_t first;        // the item's first block
    int nb;                // its blocks
};

__device__ __forceinline__ Item item_at(const Kv4AttnArgs &a, const uint32_t *s_pre,
                                        const int *s_len, int grp, int R, uint32_t x)
{
    int lo = 0, hi = a.B;                  // s_pre[lo] <= x < s_pre[lo + 1]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pre[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    Item it;
    const int2 q = queries_of(a, lo);
    it.b = lo;
    it.q0 = q.x;
    it.nq = q.y;
    it.L = s_len[lo];
    it.nb = blocks_of(it.L);
    const uint32_t tiles = uint32_t(q.y * grp + R - 1) / R, at = x - s_pre[lo];
    const uint32_t i = at / uint32_t(it.nb);
    it.kvh = int(i / tiles);
    it.tile = int(i % tiles);
    it.first = s_pre[lo] + i * it.nb;
    return it;
}

// The keys that query i of the item's sequence sees lie below this.
__device__ __forceinline__ int key_end(const Kv4AttnArgs &a, const Item &it, int i)
{
    return a.causal ? min(it.L, it.L - it.nq + i + 1) : it.L;
}

// The 8 query rows of n-tile nt as B fragments, by one warp.
template <int D, int G, int NT>
__device__ __forceinline__ void load_queries(const Kv4AttnArgs &a, const Item &it, int grp, int nt,
                                             QueryTile<D, G, NT> &to)
{
    constexpr int R = 8 * NT, NJ = D / 32, NG = D / G;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, r = nt * 8 + g;
    const int at = it.tile * R + r, i = at / grp;
    uint4 w[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        w[j] = make_uint4(0, 0, 0, 0);
    if (at < it.nq * grp) {
        const auto *src = static_cast<const __nv_bfloat16 *>(a.Q) +
                          int64_t(it.q0 + i) * a.q_stride +
                          int64_t(it.kvh * grp + at % grp) * D + 8 * c;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            w[j] = __ldg(reinterpret_cast<const uint4 *>(src + 32 * j));
    }
    float big = 0.f, sum[NG];
#pragma unroll
    for (int x = 0; x < NG; ++x)
        sum[x] = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const uint32_t v[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            big = max3(big, fabsf(bf16_lo(v[e])), fabsf(bf16_hi(v[e])));
            sum[32 * j / G] += bf16_lo(v[e]) + bf16_hi(v[e]);
        }
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // a power of two that brings the row's largest value into [2^12, 2^13)
    const int ex = big > 0.f ? max(-100, min(100, 139 - int(__float_as_uint(big) >> 23))) : 0;
    const float up = __uint_as_float(uint32_t(127 + ex) << 23);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const float x0 = bf16_lo(w[j].x) * up, x1 = bf16_hi(w[j].x) * up,
                    x2 = bf16_lo(w[j].y) * up, x3 = bf16_hi(w[j].y) * up,
                    x4 = bf16_lo(w[j].z) * up, x5 = bf16_hi(w[j].z) * up,
                    x6 = bf16_lo(w[j].w) * up, x7 = bf16_hi(w[j].w) * up;
        // nibbles i and i + 4 of a word are a half-word apart; the upper nibble
        // of a byte counts 16 times
        to.frag[nt][j][lane] =
            make_uint4(pack_f16(x0, x4), pack_f16(x1 * 0.0625f, x5 * 0.0625f), pack_f16(x2, x6),
                       pack_f16(x3 * 0.0625f, x7 * 0.0625f));
    }
    const float sc = a.scale * kLog2e;
#pragma unroll
    for (int x = 0; x < NG; ++x) {
        sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
        sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
        if (c == 0)
            to.bar[x][r] = sum[x] * sc;
    }
    if (c == 0) {
        to.mul[r] = sc * __uint_as_float(uint32_t(127 + 24 - ex) << 23);
        to.end[r] = key_end(a, it, i);
    }
}

template <int D, int G, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) attn_kv4_kernel(const Kv4AttnArgs a)
{
    constexpr int R = 8 * NT;              // query rows of a tile
    constexpr int NG = D / G;              // groups of the head dimension
    constexpr int NJ = D / 32;             // words a lane holds of a K row
    constexpr int kCell = kv4::cell_bytes(D, G);
    constexpr int kRow = D + 4;            // padded fp32 row of the merge buffer
    using Smem = Shared<D, G, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    auto *s_q = reinterpret_cast<QueryTile<D, G, NT> *>(smem + Smem::q);
    float *s_O = reinterpret_cast<float *>(smem + Smem::O);
    uint32_t *s_pre = reinterpret_cast<uint32_t *>(smem + Smem::pre);
    int *s_len = reinterpret_cast<int *>(smem + Smem::len);
    float *s_ref = reinterpret_cast<float *>(smem + Smem::ref);
    float *s_sum = reinterpret_cast<float *>(smem + Smem::sum);
    __shared__ int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int grp = a.H / a.Hkv;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Smem::full) + warp * kStages;
    uint8_t *ring = smem + Smem::ring + warp * kStages * kCell;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i)
            ptx::mbar_init(full + i, 1);
        ptx::fence_barrier_init();
    }
    if (tid == 0)
        s_abort = 0;

    // ---- the line of blocks ------------------------------------------------
    const int per = (a.B + kThreads - 1) / kThreads;
    uint32_t mine = 0;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= a.B)
            break;
        const int2 q = queries_of(a, b);
        const int L = a.seqlens[b];
        uint32_t n = 0;
        if (q.y < 0 || q.y > a.Nq || q.x < 0 || int64_t(q.x) + q.y > a.total_q || L < 0 ||
            L > a.Nk)
            record_device_error(a.err_word, FA_DEVERR_BAD_SEQLENS);
        else
            n = uint32_t((q.y * grp + R - 1) / R) * a.Hkv * blocks_of(L);
        s_len[b] = L;
        s_pre[b + 1] = n;
        mine += n;
    }
    // exclusive scan over the threads, then over each thread's sequences
    uint32_t incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += t;
    }
    uint32_t *s_w = reinterpret_cast<uint32_t *>(s_ref);
    if (lane == 31)
        s_w[warp] = incl;
    __syncthreads();
    uint32_t base = incl - mine;
    for (int w = 0; w < warp; ++w)
        base += s_w[w];
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= a.B)
            break;
        base += s_pre[b + 1];
        s_pre[b + 1] = base;
    }
    if (tid == 0)
        s_pre[0] = 0;
    __syncthreads();
    const uint64_t T = s_pre[a.B];
    const uint32_t n_ctas = uint32_t(T < gridDim.x ? T : gridDim.x);
    const Parts parts = parts_of<R>(a.workspace);
    if (blockIdx.x >= n_ctas) {
        if (tid == 0)
            parts.desc[blockIdx.x].parts = 0;
        return;
    }
    const uint32_t begin = uint32_t(T * blockIdx.x / n_ctas);
    const uint32_t end = uint32_t(T * (blockIdx.x + 1) / n_ctas);
    Desc desc{0, 0, 0, 0};

    // ---- copies ---------------------------------------------------------------
    // Lane i finds where this warp's cell of every 32nd block begins, so that the
    // search and the page table's latency are paid once for 32 cells; it then
    // issues that cell's copy itself.  `have`: which of the batch's cells are read.
    const uint32_t n_cells = end - begin;
    const uint8_t *src = nullptr;
    uint32_t have = 0, have_before = 0;
    bool bad_pages = false;
    auto find = [&](uint32_t k0) {
        src = nullptr;
        const uint32_t x = begin + k0 + lane;
        bool bad = false;
        if (x < end) {
            const Item it = item_at(a, s_pre, s_len, grp, R, x);
            const int tok = int(x - it.first) * kBlock + warp * kv4::kCellTokens;
            if (tok < key_end(a, it, (min(it.nq * grp, (it.tile + 1) * R) - 1) / grp)) {
                const int page = a.page_table[int64_t(it.b) * a.max_pages + tok / a.page_size];
                if (page >= 0 && page < a.num_pages)
                    src = static_cast<const uint8_t *>(a.cache) +
                          ((int64_t(page) * a.Hkv + it.kvh) * (a.page_size / kv4::kCellTokens) +
                           tok % a.page_size / kv4::kCellTokens) * kCell;
                else
                    bad = true;
            }
        }
        if (bad)
            record_device_error(a.err_word, FA_DEVERR_BAD_PAGE);
        bad_pages |= __any_sync(0xffffffffu, bad) != 0;
        have_before = have;
        have = __ballot_sync(0xffffffffu, src != nullptr);
    };
    const uint32_t ring_at = ptx::smem_u32(ring), full_at = ptx::smem_u32(full);
    auto issue = [&](uint32_t k) {         // all lanes of the warp
        if ((k & 31) == 0 && k < n_cells)
            find(k);
        if (k < n_cells)
            copy_cell<kCell>(full_at + (k % kStages) * 8, ring_at + (k % kStages) * kCell, src,
                             lane == int(k & 31));
    };
    for (uint32_t k = 0; k < kStages; ++k)
        issue(k);
    uint32_t done = 0;                     // cells read
    // whether cell k was left out; the batch that cell k + kStages - 1 is in, the
    // last one issued, may be the next one already
    auto skipped = [&](uint32_t k) {
        const uint32_t ahead = min(k + kStages, n_cells) - 1;
        return !((ahead / 32 == k / 32 ? have : have_before) >> (k & 31) & 1);
    };

    // this lane's places in a cell
    const uint32_t at_K = ring_at + lane * (4 * NJ);
    const uint32_t at_par = ring_at + kv4::k_par_off(D) + g * (4 * NG);
    uint32_t at_V[4];                      // of tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9
#pragma unroll
    for (int x = 0; x < 4; ++x)
        at_V[x] = ring_at + kv4::v_off(D) +
                  kv4::v_swizzle((2 * c + (x & 1) + 8 * (x >> 1)) * (D / 2) + g * (D / 16));

    Item it = item_at(a, s_pre, s_len, grp, R, begin);
    if (warp < NT)
        load_queries<D, G, NT>(a, it, grp, warp, s_q[0]);
    __syncthreads();
    int buf = 0;
    for (uint32_t cur = begin; cur < end;) {
        const uint32_t stop = min(end, it.first + it.nb);
        const int rows = min(R, it.nq * grp - it.tile * R);         // rows of this tile
        const QueryTile<D, G, NT> &qt = s_q[buf];
        const uint32_t at_Q = ptx::smem_u32(&qt.frag[0][0][lane]);
        float mul[NT][2], qbar[NT][NG][2];     // of rows 2 c, 2 c + 1 of n-tile nt
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = nt * 8 + 2 * c + e;
                mul[nt][e] = qt.mul[r];
#pragma unroll
                for (int x = 0; x < NG; ++x)
                    qbar[nt][x][e] = qt.bar[x][r];
            }

        // ---- the keys ----------------------------------------------------------
        float O[NT][D / 16][4], ref[NT][2], sum[NT][2], pm[NT][NG][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
                O[nt][x][0] = O[nt][x][1] = O[nt][x][2] = O[nt][x][3] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ref[nt][e] = kNoRef;
                sum[nt][e] = 0.f;
#pragma unroll
                for (int x = 0; x < NG; ++x)
                    pm[nt][x][e] = 0.f;
            }
        }
        // One cell's keys.  kMasked: some query row of the tile does not see all
        // of them, or the sequence ends inside the cell.
        auto cell_step = [&](uint32_t slot, int tok, auto masked_tag) {
            constexpr bool kMasked = decltype(masked_tag)::value;
            constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;
            // S^T = K Q^T: lane (g, c) holds tokens g, g + 8
            uint32_t k0[NJ], k1[NJ];
            load_shared<0>(k0, at_K + slot);
            load_shared<8 * (D / 2)>(k1, at_K + slot);
            // (scale, min) pairs of tokens g and g + 8
            uint32_t pk[2][NG], pv[2][NG];
            constexpr int kV = 64 * NG, kUp = 32 * NG;
            load_shared<0>(pk[0], at_par + slot);
            load_shared<kUp>(pk[1], at_par + slot);
            load_shared<kV>(pv[0], at_par + slot);
            load_shared<kV + kUp>(pv[1], at_par + slot);
            if constexpr (kMasked) {
                // behind the sequence's end they may be anything, and count as 0
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (tok + g + 8 * t >= it.L)
#pragma unroll
                        for (int x = 0; x < NG; ++x)
                            pk[t][x] = pv[t][x] = 0;
            }
            float acc[NT][NG][4];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const uint32_t y0 = k0[j] >> 8, y1 = k1[j] >> 8;
                const uint32_t a0[4] = {k0[j] & kLo, k1[j] & kLo, k0[j] & kHi, k1[j] & kHi};
                const uint32_t a1[4] = {y0 & kLo, y1 & kLo, y0 & kHi, y1 & kHi};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t q[4];
                    load_shared<0>(q, at_Q + (nt * NJ + j) * 512);
                    if (32 * j % G == 0)
                        mma_first(acc[nt][32 * j / G], a0, q[0], q[1]);
                    else
                        mma(acc[nt][32 * j / G], a0, q[0], q[1]);
                    mma(acc[nt][32 * j / G], a1, q[2], q[3]);
                }
            }
            float w[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float s_big = bf16_lo(pv[t][0]), m_big = fabsf(bf16_hi(pv[t][0]));
#pragma unroll
                for (int x = 1; x < NG; ++x) {
                    s_big = fmaxf(s_big, bf16_lo(pv[t][x]));
                    m_big = fmaxf(m_big, fabsf(bf16_hi(pv[t][x])));
                }
                // |m| counts too (a constant group has s = 0), so that P m stays
                // finite in fp32
                w[t] = max3(s_big, m_big * 0x1p-12f, kLeastWeight);
            }
            uint32_t pf[NT][NG][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // S - `from`, [token g, g + 8][row 2 c, 2 c + 1]
                bool seen[2][2];
                auto score = [&](int t, int e, float from) {
                    float x = bf16_lo(pk[t][0]) * acc[nt][0][2 * t + e], y = -from;
#pragma unroll
                    for (int gr = 1; gr < NG; ++gr)
                        x = fmaf(bf16_lo(pk[t][gr]), acc[nt][gr][2 * t + e], x);
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr)
                        y = fmaf(bf16_hi(pk[t][gr]), qbar[nt][gr][e], y);
                    return seen[t][e] ? fmaf(x, mul[nt][e], y) : -INFINITY;
                };
                float P[2][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int last = kMasked ? qt.end[nt * 8 + 2 * c + e] : 0;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        seen[t][e] = !kMasked || tok + g + 8 * t < last;
                        P[t][e] = ptx::ex2(score(t, e, ref[nt][e]));
                    }
                }
                const float over = fmaxf(max3(P[0][0] * w[0], P[0][1] * w[0], P[1][0] * w[1]),
                                         P[1][1] * w[1]);
                if (__any_sync(0xffffffffu, over > kLag)) {
                    // a row outgrew its reference: every row's becomes the largest
                    // S + log2 w seen
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float S0 = score(0, e, 0.f), S1 = score(1, e, 0.f);
                        float m = fmaxf(S0 + __log2f(w[0]), S1 + __log2f(w[1]));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        m = fmaxf(m, ref[nt][e]);
                        const float f = ptx::ex2(ref[nt][e] - m);
                        ref[nt][e] = m;
                        sum[nt][e] *= f;
#pragma unroll
                        for (int x = 0; x < NG; ++x)
                            pm[nt][x][e] *= f;
#pragma unroll
                        for (int x = 0; x < D / 16; ++x) {
                            O[nt][x][e] *= f;
                            O[nt][x][2 + e] *= f;
                        }
                        P[0][e] = ptx::ex2(S0 - m);
                        P[1][e] = ptx::ex2(S1 - m);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    sum[nt][e] += P[0][e] + P[1][e];
#pragma unroll
                for (int x = 0; x < NG; ++x)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        float y[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            // a key that the row does not see adds nothing,
                            // whatever its parameters are
                            y[e] = P[t][e] * bf16_lo(pv[t][x]);
                            const float z = fmaf(P[t][e], bf16_hi(pv[t][x]), pm[nt][x][e]);
                            if (kMasked && !seen[t][e])
                                y[e] = 0.f;
                            else
                                pm[nt][x][e] = z;
                        }
                        pf[nt][x][t] = transpose8x8(pack_f16(y[0], y[1]));
                    }
            }

            // O^T += V^T P^T: lane (g, c) holds its halves of tokens 2 c, 2 c + 1,
            // 2 c + 8, 2 c + 9; a half-word pair of two tokens is one A register
            uint32_t v[4][D / 64];
#pragma unroll
            for (int x = 0; x < 4; ++x)
                load_shared<0>(v[x], at_V[x] + slot);
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                const uint32_t sel = (q & 1) ? 0x7632 : 0x5410;
                const uint32_t x = __byte_perm(v[0][q / 2], v[1][q / 2], sel);
                const uint32_t y = __byte_perm(v[2][q / 2], v[3][q / 2], sel);
                const uint32_t x8 = x >> 8, y8 = y >> 8;
                const uint32_t a0[4] = {x & kLo, x & kHi, y & kLo, y & kHi};
                const uint32_t a1[4] = {x8 & kLo, x8 & kHi, y8 & kLo, y8 & kHi};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma(O[nt][2 * q], a0, pf[nt][32 * q / G][0], pf[nt][32 * q / G][1]);
                    mma(O[nt][2 * q + 1], a1, pf[nt][32 * q / G][0], pf[nt][32 * q / G][1]);
                }
            }
        };

        // keys that some row of the tile sees, and that all rows see
        const int tok_end = key_end(a, it, (it.tile * R + rows - 1) / grp);
        const int all_end = key_end(a, it, it.tile * R / grp);
        int tok = int(cur - it.first) * kBlock + warp * kv4::kCellTokens;
        for (uint32_t k = cur - begin; k < stop - begin; ++k, tok += kBlock) {
            if (!ptx::mbar_wait_warp(full + k % kStages, k / kStages & 1, &s_abort, a.err_word))
                break;                     // the error is recorded, nothing is written
            done = k + 1;
            if (tok < tok_end && !(bad_pages && skipped(k))) {
                const uint32_t slot = k % kStages * kCell;
                if (tok + kv4::kCellTokens <= all_end)
                    cell_step(slot, tok, std::false_type{});
                else
                    cell_step(slot, tok, std::true_type{});
            }
            __syncwarp();                  // every lane has read the cell
            issue(k + kStages);
        }

        // ---- the warps' parts joined, and written ----------------------------
        const bool whole = cur == it.first && stop == it.first + it.nb;
        const int slot = 2 * int(blockIdx.x) + (cur == it.first ? 1 : 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float s = sum[nt][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
                for (int x = 0; x < NG; ++x)
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1)
                        pm[nt][x][e] += __shfl_xor_sync(0xffffffffu, pm[nt][x][e], o);
                if (g == 0) {
                    s_ref[warp * R + nt * 8 + 2 * c + e] = ref[nt][e];
                    s_sum[warp * R + nt * 8 + 2 * c + e] = s;
                }
            }
        __syncthreads();
        const Item next = stop < end ? item_at(a, s_pre, s_len, grp, R, stop) : it;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // the upper warps' rows through shared memory into the lower warps'
            // registers, then the lower warps' rows for all to sum
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (warp / (kWarps / 2) == 1 - half) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = nt * 8 + 2 * c + e;
                        float m = s_ref[r];
#pragma unroll
                        for (int w = 1; w < kWarps; ++w)
                            m = fmaxf(m, s_ref[w * R + r]);
                        const float f = ptx::ex2(ref[nt][e] - m);
                        float *row = s_O + (warp % (kWarps / 2) * 8 + 2 * c + e) * kRow + 4 * g;
#pragma unroll
                        for (int q = 0; q < D / 32; ++q) {
                            const float p = pm[nt][32 * q / G][e];
                            float4 y = make_float4(fmaf(O[nt][2 * q][e], 0x1p24f, p) * f,
                                                   fmaf(O[nt][2 * q][2 + e], 0x1p20f, p) * f,
                                                   fmaf(O[nt][2 * q + 1][e], 0x1p24f, p) * f,
                                                   fmaf(O[nt][2 * q + 1][2 + e], 0x1p20f, p) * f);
                            float4 *at = reinterpret_cast<float4 *>(row + 32 * q);
                            if (half == 1) {
                                const float4 z = *at;
                                y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
                            }
                            *at = y;
                        }
                    }
                } else if (half == 0 && nt == 0 && warp < NT && stop < end) {
                    // meanwhile the next item's queries
                    load_queries<D, G, NT>(a, next, grp, warp, s_q[buf ^ 1]);
                }
                __syncthreads();
            }
            // 8 rows x D values over the threads, four consecutive values each
            for (int x = tid; x < 8 * (D / 4); x += kThreads) {
                const int rr = x / (D / 4), d4 = x % (D / 4) * 4, r = nt * 8 + rr;
                float4 y = *reinterpret_cast<const float4 *>(s_O + rr * kRow + d4);
                float m = s_ref[r];
#pragma unroll
                for (int w = 1; w < kWarps / 2; ++w) {
                    const float4 z =
                        *reinterpret_cast<const float4 *>(s_O + (w * 8 + rr) * kRow + d4);
                    y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
                }
#pragma unroll
                for (int w = 1; w < kWarps; ++w)
                    m = fmaxf(m, s_ref[w * R + r]);
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    s = fmaf(s_sum[w * R + r], ptx::ex2(s_ref[w * R + r] - m), s);
                if (r >= rows || s_abort)
                    continue;
                if (whole) {
                    const int at = it.tile * R + r, i = at / grp, h = it.kvh * grp + at % grp;
                    const bool any = s > 0.f || s != s;
                    const float inv = any ? 1.f / s : 0.f;
                    const uint2 o = make_uint2(ptx::pack_bf16x2(y.x * inv, y.y * inv),
                                               ptx::pack_bf16x2(y.z * inv, y.w * inv));
                    auto *dst = static_cast<__nv_bfloat16 *>(a.O) +
                                (int64_t(it.q0 + i) * a.H + h) * D + d4;
                    *reinterpret_cast<uint2 *>(dst) = o;
                    if (d4 == 0)
                        a.lse[a.cu_seqlens_q ? int64_t(h) * a.total_q + it.q0 + i
                                             : (int64_t(it.b) * a.H + h) * a.Nq + i] =
                            any ? (m + log2f(s)) * kLn2 : -INFINITY;
                } else {
                    *reinterpret_cast<float4 *>(parts.O + (int64_t(slot) * R + r) * D + d4) = y;
                    if (d4 == 0)
                        parts.ml[slot * R + r] = make_float2(m, s);
                }
            }
            __syncthreads();
        }
        if (cur == it.first && !whole) {
            // CTAs that hold a part: up to the one whose range has the last block
            const uint64_t x = uint64_t(it.first) + it.nb;      // ceil(x n / T) - 1
            const int last_cta = int((x * n_ctas + T - 1) / T) - 1;
            desc = Desc{last_cta - int(blockIdx.x) + 1, it.b, it.kvh, it.tile};
        }
        cur = stop;
        it = next;
        buf ^= 1;
    }
    if (s_abort) {
        // a wait ran out: copies still on their way must land before the CTA ends
        desc.parts = 0;
        volatile int go_on = 0;
        for (uint32_t k = done; k < min(done + kStages, n_cells); ++k)
            ptx::mbar_wait_limited(full + k % kStages, k / kStages & 1, &go_on, a.err_word,
                                   kWaitTimeoutNs);
    }
    if (tid == 0)
        parts.desc[blockIdx.x] = desc;
}

// Joins the parts of the items that span CTAs: block (x, y) takes row y of the
// item that begins in CTA x's range.  Parts are added in the order of the CTAs.
template <int D, int R>
__global__ void __launch_bounds__(D) attn_kv4_join_kernel(const Kv4AttnArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Parts parts = parts_of<R>(a.workspace);
    const Desc desc = parts.desc[blockIdx.x];
    if (desc.parts == 0)
        return;
    const int2 qb = queries_of(a, desc.b);
    const int grp = a.H / a.Hkv, r = blockIdx.y, at = desc.tile * R + r;
    if (at >= qb.y * grp)
        return;
    const int x = threadIdx.x;
    float m = kNoRef;
    for (int p = 0; p < desc.parts; ++p) {
        const int slot = 2 * (blockIdx.x + p) + (p == 0);
        m = fmaxf(m, parts.ml[slot * R + r].x);
    }
    float s = 0.f, y = 0.f;
    for (int p = 0; p < desc.parts; ++p) {
        const int slot = 2 * (blockIdx.x + p) + (p == 0);
        const float2 ml = parts.ml[slot * R + r];
        const float f = ptx::ex2(ml.x - m);
        s = fmaf(ml.y, f, s);
        y = fmaf(parts.O[(int64_t(slot) * R + r) * D + x], f, y);
    }
    const int i = at / grp, h = desc.kvh * grp + at % grp;
    const bool any = s > 0.f || s != s;
    static_cast<__nv_bfloat16 *>(a.O)[(int64_t(qb.x + i) * a.H + h) * D + x] =
        __float2bfloat16_rn(any ? y / s : 0.f);
    if (x == 0)
        a.lse[a.cu_seqlens_q ? int64_t(h) * a.total_q + qb.x + i
                             : (int64_t(desc.b) * a.H + h) * a.Nq + i] =
            any ? (m + log2f(s)) * kLn2 : -INFINITY;
}

template <int D, int G, int NT>
int launch(const Kv4AttnArgs &a, cudaStream_t stream)
{
    constexpr int R = 8 * NT;
    constexpr int smem = Shared<D, G, NT>::bytes;
    static PerDeviceOnce once;
    if (!set_max_dynamic_smem(once, reinterpret_cast<const void *>(attn_kv4_kernel<D, G, NT>), smem))
        return FA_ERR_CUDA;
    // one CTA of the widest tile fits an SM (registers), two of the others
    const int ctas = NT == 4 ? kKv4MaxCtas / 2 : kKv4MaxCtas;
    attn_kv4_kernel<D, G, NT><<<ctas, kThreads, smem, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess)
        return FA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, R);
    cfg.blockDim = dim3(D);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_kv4_join_kernel<D, R>, a);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, int G>
int launch_rows(const Kv4AttnArgs &a, cudaStream_t stream)
{
    switch (kv4_attention_rows(a.Nq, a.H, a.Hkv)) {
    case 8: return launch<D, G, 1>(a, stream);
    case 16: return launch<D, G, 2>(a, stream);
    default: return launch<D, G, 4>(a, stream);
    }
}

}  // namespace

int launch_attention_kv4(const Kv4AttnArgs &a, cudaStream_t stream)
{
    if (a.d == 64)
        return a.group == 32 ? launch_rows<64, 32>(a, stream) : launch_rows<64, 64>(a, stream);
    return a.group == 32   ? launch_rows<128, 32>(a, stream)
           : a.group == 64 ? launch_rows<128, 64>(a, stream)
                           : launch_rows<128, 128>(a, stream);
}

}  // namespace fa
