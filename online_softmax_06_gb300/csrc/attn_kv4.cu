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
// rounded to fp16 (2^-11, against 2^-8 for bf16), after a power of two for each row
// and group.
//
// Layout: keys are the rows (M = 16 tokens), query rows (query, head of the
// group) the columns (N = 8) of mma.m16n8k16, S^T = K Q^T and O^T = V^T P^T, so
// that a decode step with up to 8 heads a kv head wastes nothing.  tcgen05 has
// M = 64 at least and takes its operands from shared or tensor memory: the
// codes would be expanded fourfold into shared memory first, which costs more
// than the products (attn_kv4_many.cu does it where there are rows enough).
//
// What bounds it: a cell of 16 tokens (2304 bytes with d = 128, group 64) costs a
// warp 236 instructions with 4 rows, 274 with 8, of which half are logical
// operations at two a cycle and SM, 88 of them the expansion; HBM leaves 100 cycles a
// cell.  64 sequences of 300 to 16000 keys (32 heads on 8) take 102 us, 5.9 TB/s, 0.87
// of the measured copy rate: the start (lengths, page table, first cells: three memory
// latencies) takes 7 of them, the crews' ends 5, the join 4.  One MMA of 16 x 8 x 16
// takes two cycles of an SM (605 TFLOP/s), a quarter of the time.
//
// One CTA an SM, of crews of four warps that share nothing but the layout of the
// work.  As CTAs of their own, three an SM, the crews were served in the order in
// which they came and ended 25 us apart (84, 95 and 110 us; so 99, 100 and 101).
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

using kv4::bf16_hi;
using kv4::bf16_lo;
using kv4::pow2;
using ptx::max3;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kWarps = 4;            // of a crew
constexpr int kThreads = kWarps * 32;
constexpr int kPair = 2 * kv4::kCellTokens;         // tokens that a warp copies and takes at once
constexpr int kBlock = kWarps * kPair;              // tokens of a block: two cells each warp
// Reference of a row that has seen no key: exp2(-inf - kNoRef) = 0, and a score above it
// by 2^7 or more makes a P that moves it.
constexpr float kNoRef = -0x1p126f;
// A row's reference stands kRefAbove above its largest S and may lag until a P exceeds
// kMostP, so that the fp32 sums of P and P m stay finite for values up to 2^110.  P s
// goes to fp16 after a power of two of the row and group (`up`) that brings the largest
// into [2^7, 2^8), up to kMostPs as it lags: a group of small scales keeps its bits
// beside one of large scales, and a key of 2^-21 of the largest weight its share.  (With
// one reference for all groups, P s <= 1 for a key's largest scale, a group of scales
// 2^-20 of its neighbour's was off by three of its own steps.)  It costs 0 to 1 % with
// 4 rows (64 x 8k keys 101.7 us) and one to five with 8 and 16 and groups of 32 or 64 (32
// x 2 queries on 2k to 9k keys, groups of 64, 48.8 us, so 47.7; of 32 56.3 and 55.1).
constexpr float kRefAbove = 10.f, kMostP = 0x1p-2f, kMostPs = 0x1p15f;
constexpr int kMostUp = 120;       // log2 of `up` at the most, and of 1 / `up`
// 1 / x of such a power of two
__device__ __forceinline__ float inverse(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }

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

// The same value in every lane, as the compiler cannot know: what follows from it
// (addresses, loop control) then runs on the uniform datapath.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Keeps a lane's address in its register instead of computing it anew at each use.
__device__ __forceinline__ void keep(uint32_t &x) { asm volatile("" : "+r"(x)); }

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

// Of NC cells the words at address `at` + OFF and, for token g + 8, UP on.
template <int NC, int CELL, int OFF, int UP, int N>
__device__ __forceinline__ void load_tokens(uint32_t (&w)[NC][2][N], uint32_t at)
{
    load_shared<OFF>(w[0][0], at);
    load_shared<OFF + UP>(w[0][1], at);
    if constexpr (NC == 2) {
        load_shared<CELL + OFF>(w[1][0], at);
        load_shared<CELL + OFF + UP>(w[1][1], at);
    }
}

// The words of token number i of a lane's four.
template <int NC, int CELL, int OFF, int N>
__device__ __forceinline__ void load_values(uint32_t (&v)[NC][4][N], int i, uint32_t at)
{
    load_shared<OFF>(v[0][i], at);
    if constexpr (NC == 2)
        load_shared<CELL + OFF>(v[1][i], at);
}

// Pairs of cells on their way or in use: each warp has a ring of its own and
// fills a place again as soon as it has read it; no barrier between warps.  12
// warps an SM with one pair of 4608 bytes each on its way are 55 KB in flight,
// against the 36 KB that cover HBM's latency at full rate; three pairs a ring
// measured the same (64 x 8k keys 104 us with either).
constexpr int kStages = 2;
constexpr int kJoinWarps = 8;

// A work item is (sequence, kv head, tile of R query rows); its keys are cut
// into blocks of kBlock tokens.  All items' blocks, sequence by sequence, form
// one line that is cut into equal ranges, one a crew: ragged batches and single
// long sequences fill the GPU alike, and nothing of it needs the host.
//
// An item costs a crew some time beside its blocks' (queries, the four warps'
// join): the line is cut as if each item had kItemCost blocks more.  Without it
// the crews whose range holds the short sequences of a batch ended last (32
// sequences of 1 to 8191 keys, 16 kv heads, d = 64: 74 us, against 46 with 4096
// each).
constexpr uint32_t kItemCost = 3;

struct Desc {          // of a range
    uint32_t begin;    // first block of its range
    uint32_t item_end; // end of the item that begins in it and goes on after it; 0: none
    int b, kvh, tile;  // that item
    int aborted;       // a wait ran out: parts of the range's items may be missing
    int unused[2];
};

// Workspace: Desc[ranges], then (reference, sum) [2 ranges][R], then the
// unnormalised O [2 ranges][R][d] fp32.  A range's slot 0 holds the part of an item
// that began before its range, slot 1 that of one that goes on after.
struct Parts {
    Desc *desc;
    float2 *ml;
    float *O;
};

template <int D, int R>
__host__ __device__ inline Parts parts_of(void *ws)
{
    Parts p;
    p.desc = static_cast<Desc *>(ws);
    p.ml = reinterpret_cast<float2 *>(p.desc + kv4_attention_ranges(R, D));
    p.O = reinterpret_cast<float *>(p.ml + 2 * kv4_attention_ranges(R, D) * R);
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

// A crew's shared memory, and at its end what the CTA's crews have in common.
template <int D, int G, int NT>
struct Shared {
    static constexpr int R = 8 * NT;                                 // columns
    static constexpr int ring = 0;                                   // [kWarps][kStages] pairs
    static constexpr int q = ring + kWarps * kStages * 2 * kv4::cell_bytes(D, G);  // QueryTile
    static constexpr int O = q + int(sizeof(QueryTile<D, G, NT>));   // [kWarps / 2][8][D + 4]
    static constexpr int full = O + kWarps / 2 * 8 * (D + 4) * 4;    // [kWarps][kStages] barriers
    static constexpr int ref = full + kWarps * kStages * 8;          // [kWarps][R]
    static constexpr int sum = ref + kWarps * R * 4;                 // [kWarps][R]
    static constexpr int abort = sum + kWarps * R * 4;               // a wait ran out
    static constexpr int limit = abort + 4;                          // of its waits, ns
    static constexpr int bytes = (limit + 4 + 127) / 128 * 128;

    static constexpr int crews = kv4_attention_crews(R, D);
    static constexpr int pre = 0;                                    // [B + 1] blocks before b
    // [B + 1] their costs.  Not in a ring: a barrier does not order these stores before
    // the copies, which another proxy makes
    static constexpr int cost = pre + (kKv4MaxSeqs + 4) * 4;
    static constexpr int scan = cost + (kKv4MaxSeqs + 4) * 4;        // a uint2 of each warp
    static constexpr int own = (scan + crews * kWarps * 8 + 127) / 128 * 128;
    static constexpr int all = own + crews * bytes;
};

// Where block x of the line is.
struct Item {
    int b, q0, nq, L;      // sequence, its first query row, queries, keys
    int kvh, tile;
    uint32_t first;        // the item's first block
    int nb;                // its blocks
};

__device__ __forceinline__ Item item_at(const Kv4AttnArgs &a, const uint32_t *s_pre, int grp, int R,
                                        uint32_t x)
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
    it.L = a.seqlens[lo];
    it.nb = blocks_of(it.L);
    const uint32_t tiles = uint32_t(q.y * grp + R - 1) / R, at = x - s_pre[lo];
    const uint32_t i = at / uint32_t(it.nb);
    it.kvh = int(i / tiles);
    it.tile = int(i % tiles);
    it.first = s_pre[lo] + i * it.nb;
    return it;
}

__device__ __forceinline__ Item uniform(Item it)
{
    it.b = uniform(it.b);
    it.q0 = uniform(it.q0);
    it.nq = uniform(it.nq);
    it.L = uniform(it.L);
    it.kvh = uniform(it.kvh);
    it.tile = uniform(it.tile);
    it.first = uint32_t(uniform(int(it.first)));
    it.nb = uniform(it.nb);
    return it;
}

// The item after `it`.
__device__ __forceinline__ Item next_item(const Kv4AttnArgs &a, const uint32_t *s_pre, int grp,
                                          int R, Item it)
{
    it.first += it.nb;
    if (++it.tile * R < it.nq * grp)
        return it;
    it.tile = 0;
    if (++it.kvh < a.Hkv)
        return it;
    it.kvh = 0;
    do                                     // sequences without blocks are passed over
        ++it.b;
    while (it.b + 1 < a.B && s_pre[it.b + 1] == s_pre[it.b]);
    if (it.b < a.B) {
        const int2 q = queries_of(a, it.b);
        it.q0 = q.x;
        it.nq = q.y;
        it.L = a.seqlens[it.b];
        it.nb = blocks_of(it.L);
    }
    return uniform(it);
}

// The keys that query i of the item's sequence sees lie below this.
__device__ __forceinline__ int key_end(const Kv4AttnArgs &a, const Item &it, int i)
{
    return a.causal ? min(it.L, it.L - it.nq + i + 1) : it.L;
}

// The block at place x of the line of costs: an item's kItemCost come first.
__device__ __forceinline__ uint32_t block_of(const Kv4AttnArgs &a, const uint32_t *s_pre,
                                             const uint32_t *s_cost, uint32_t x)
{
    if (x >= s_cost[a.B])
        return s_pre[a.B];
    int lo = 0, hi = a.B;                  // s_cost[lo] <= x < s_cost[lo + 1]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cost[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    const uint32_t nb = blocks_of(a.seqlens[lo]), at = x - s_cost[lo], i = at / (nb + kItemCost);
    const uint32_t o = at - i * (nb + kItemCost);
    return s_pre[lo] + i * nb + (o > kItemCost ? o - kItemCost : 0);
}

// The first item that begins at block x or after it.
__device__ __forceinline__ uint32_t item_from(const Kv4AttnArgs &a, const uint32_t *s_pre, int grp,
                                              int R, uint32_t x, uint32_t T)
{
    if (x >= T)
        return T;
    const Item it = item_at(a, s_pre, grp, R, x);
    return it.first == x ? x : it.first + it.nb;
}

// The tile row at column col of the products.  With E = 1 (4 rows and fewer) a lane's
// second column stays empty, and what it would cost is left out.
template <int E>
__host__ __device__ constexpr int row_of(int col) { return E == 1 ? col / 2 : col; }

// A lane's share of the 8 columns of n-tile nt: column g, values 32 j + 8 c ...
template <int D, int NT, int E>
__device__ __forceinline__ void fetch_queries(const Kv4AttnArgs &a, const Item &it, int grp, int nt,
                                              uint4 (&w)[D / 32])
{
    constexpr int R = 4 * NT * E, NJ = D / 32;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int at = it.tile * R + row_of<E>(nt * 8 + g), i = at / grp;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        w[j] = make_uint4(0, 0, 0, 0);
    if (at < it.nq * grp && (E == 2 || g % 2 == 0)) {
        const auto *src = static_cast<const __nv_bfloat16 *>(a.Q) +
                          int64_t(it.q0 + i) * a.q_stride +
                          int64_t(it.kvh * grp + at % grp) * D + 8 * c;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            w[j] = *reinterpret_cast<const uint4 *>(src + 32 * j);
    }
}

// They as B fragments, by the warp.
template <int D, int G, int NT, int E>
__device__ __forceinline__ void place_queries(const Kv4AttnArgs &a, const Item &it, int grp, int nt,
                                              const uint4 (&w)[D / 32], QueryTile<D, G, NT> &to)
{
    constexpr int R = 4 * NT * E, NJ = D / 32, NG = D / G;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, r = nt * 8 + g;
    const int i = (it.tile * R + row_of<E>(r)) / grp;
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
    // a power of two that brings the row's largest value into [2^12, 2^13) (below 2^16 up
    // to 2^116, so that the factor of the scores stays finite; none too small is left out)
    const int ex = big > 0.f ? max(-100, min(127, 139 - int(__float_as_uint(big) >> 23))) : 0;
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

// A warp's wait for a pair of cells; behind the abort flag stands its limit in ns.
__device__ __noinline__ bool wait_pair_slow(uint64_t *bar, uint32_t parity, volatile int *abort,
                                            int *err_word)
{
    return ptx::mbar_wait_limited(bar, parity, abort, err_word, uint32_t(abort[1]));
}
__device__ __forceinline__ bool wait_pair(uint64_t *bar, uint32_t parity, volatile int *abort,
                                          int *err_word)
{
    return __all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity) ||
                                       wait_pair_slow(bar, parity, abort, err_word)) != 0;
}

// One copy: `bytes` from `src`; 0: none; -n: n bytes of a page that there is not.
struct Copy {
    const uint8_t *src;
    int bytes;
};

// What lane `half` of two has to copy of the pair of cells from token `tok0` of
// block x on: the cells of a page of a multiple of 32 tokens are one piece of
// memory, which the first lane copies; otherwise each lane copies a cell.
__device__ __noinline__ Copy find_copy(const Kv4AttnArgs &a, const uint32_t *s_pre, int grp, int R,
                                       int cell_bytes, uint32_t x, int tok0, int half)
{
    Copy c{nullptr, 0};
    const Item it = item_at(a, s_pre, grp, R, x);
    const bool one = a.page_size % kPair == 0;
    const int tok = int(x - it.first) * kBlock + tok0 + half * kv4::kCellTokens;
    const int stop = key_end(a, it, (min(it.nq * grp, (it.tile + 1) * R) - 1) / grp);
    if (tok >= stop || (one && half == 1))
        return c;
    c.bytes = one && tok + kv4::kCellTokens < stop ? 2 * cell_bytes : cell_bytes;
    const int col = tok / a.page_size;
    const int page = a.page_table[int64_t(it.b) * a.max_pages + col];
    if (page < 0 || page >= a.num_pages) {
        record_device_error(a.err_word, FA_DEVERR_BAD_PAGE);
        c.bytes = -c.bytes;
        return c;
    }
    c.src = static_cast<const uint8_t *>(a.cache) +
            ((int64_t(page) * a.Hkv + it.kvh) * (a.page_size / kv4::kCellTokens) +
             (tok - col * a.page_size) / kv4::kCellTokens) * cell_bytes;
    return c;
}

template <int D, int G, int NT, int E>
__global__ void __launch_bounds__(kThreads *kv4_attention_crews(8 * NT, D), 1)
    attn_kv4_kernel(const Kv4AttnArgs a)
{
    constexpr int R = 4 * NT * E;          // query rows of a tile
    constexpr int kCols = 8 * NT;          // columns of the products
    constexpr int NG = D / G;              // groups of the head dimension
    constexpr int NJ = D / 32;             // words a lane holds of a K row
    constexpr int kCell = kv4::cell_bytes(D, G);
    constexpr int kRow = D + 4;            // padded fp32 row of the merge buffer
    constexpr int kVBases = D == 128 ? 2 : 4;   // d = 128: 8 tokens are 512 bytes on
    // Cells taken at once: two overlap, but with four groups a head their
    // parameters do not fit the registers.
    constexpr int kCells = NG == 4 ? 1 : 2;
    using Smem = Shared<D, G, NT>;
    extern __shared__ __align__(128) uint8_t smem_cta[];
    const int crew = uniform(int(threadIdx.x) / kThreads);
    const int id = crew * kv4_attention_sms + int(blockIdx.x);       // of the crew's range
    uint8_t *smem = smem_cta + Smem::own + crew * Smem::bytes;
    auto &s_q = *reinterpret_cast<QueryTile<D, G, NT> *>(smem + Smem::q);
    float *s_O = reinterpret_cast<float *>(smem + Smem::O);
    uint32_t *s_pre = reinterpret_cast<uint32_t *>(smem_cta + Smem::pre);
    float *s_ref = reinterpret_cast<float *>(smem + Smem::ref);
    float *s_sum = reinterpret_cast<float *>(smem + Smem::sum);
    volatile int &s_abort = *reinterpret_cast<volatile int *>(smem + Smem::abort);
    volatile uint32_t &s_limit = *reinterpret_cast<volatile uint32_t *>(smem + Smem::limit);
    const int tid = threadIdx.x % kThreads, warp = uniform(tid >> 5), lane = tid & 31, g = lane >> 2,
              c = lane & 3;
    auto sync_crew = [&] { asm volatile("bar.sync %0, 128;" ::"r"(crew + 1) : "memory"); };
    const int grp = a.H / a.Hkv;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Smem::full) + warp * kStages;
    uint8_t *ring = smem + Smem::ring + warp * (kStages * 2 * kCell);
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i)
            ptx::mbar_init(full + i, 2);   // a pair's two lanes
        ptx::fence_barrier_init();
    }
    if (tid == 0) {
        s_abort = 0;
        s_limit = uint32_t(kWaitTimeoutNs);
    }
    // the kernels before have ended; the join's launch may overlap this kernel, whose
    // end it waits for
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the line of blocks ------------------------------------------------
    constexpr int kAll = kThreads * Smem::crews;
    const int per = (a.B + kAll - 1) / kAll;
    uint32_t *s_cost = reinterpret_cast<uint32_t *>(smem_cta + Smem::cost);
    uint32_t mine = 0, mine_cost = 0;
    bool falls = false;                    // cu_seqlens_q does, somewhere
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b >= a.B)
            break;
        const int2 q = queries_of(a, b);
        const int L = a.seqlens[b];
        uint32_t items = 0;
        falls = falls || q.y < 0;
        if (q.y < 0 || q.y > a.Nq || q.x < 0 || int64_t(q.x) + q.y > a.total_q || L < 0 ||
            L > a.Nk)
            record_device_error(a.err_word, FA_DEVERR_BAD_SEQLENS);
        else
            items = uint32_t((q.y * grp + R - 1) / R) * a.Hkv;
        s_pre[b + 1] = items * blocks_of(L);
        s_cost[b + 1] = items * (blocks_of(L) + kItemCost);
        mine += s_pre[b + 1];
        mine_cost += s_cost[b + 1];
    }
    // exclusive scans over the threads, then over each thread's sequences
    uint32_t incl = mine, incl_cost = mine_cost;
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
        const uint32_t t_cost = __shfl_up_sync(0xffffffffu, incl_cost, o);
        if (lane >= o) {
            incl += t;
            incl_cost += t_cost;
        }
    }
    uint2 *s_w = reinterpret_cast<uint2 *>(smem_cta + Smem::scan);
    if (lane == 31)
        s_w[crew * kWarps + warp] = make_uint2(incl, incl_cost);
    // Where cu_seqlens_q falls, sequences may claim more rows together than there are, and
    // their blocks more than 32 bits: nothing is computed.
    falls = __syncthreads_or(falls);
    uint32_t base = incl - mine, base_cost = incl_cost - mine_cost;
    for (int w = 0; w < crew * kWarps + warp; ++w) {
        base += s_w[w].x;
        base_cost += s_w[w].y;
    }
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b >= a.B)
            break;
        base += s_pre[b + 1];
        base_cost += s_cost[b + 1];
        s_pre[b + 1] = base;
        s_cost[b + 1] = base_cost;
    }
    if (threadIdx.x == 0)
        s_pre[0] = s_cost[0] = 0;
    __syncthreads();
    const uint32_t T = falls ? 0u : uint32_t(uniform(int(s_pre[a.B])));
    const uint32_t n_ranges = min(T, uint32_t(kv4_attention_ranges(R, D)));
    const Parts parts = parts_of<D, R>(a.workspace);
    uint32_t begin = T, end = T;
    if (id < n_ranges) {
        const uint64_t all = uint32_t(uniform(int(s_cost[a.B])));
        // both ends at once, by the odd and the even lanes
        uint32_t x = block_of(a, s_pre, s_cost, uint32_t(all * uint32_t(id + (lane & 1)) / n_ranges));
        if (a.whole_items)                 // the items that begin in the range
            x = item_from(a, s_pre, grp, R, x, T);
        begin = __shfl_sync(0xffffffffu, x, 0);
        end = __shfl_sync(0xffffffffu, x, 1);
    }
    Desc desc{begin, 0, 0, 0, 0, 0, {}};
    if (begin >= end) {
        if (tid == 0 && !a.whole_items)
            parts.desc[id] = desc;
        return;
    }

    // ---- copies ------------------------------------------------------------------
    // Each warp copies its own pairs.  32 lanes find the sources of 16 pairs at
    // once, so that the search and the page table's latency are paid once for
    // them, and issue them when their turn comes.
    // The first item's queries are requested before.
    Item it = uniform(item_at(a, s_pre, grp, R, begin));
    uint4 first_q[NJ];
    if (warp < NT)
        fetch_queries<D, NT, E>(a, it, grp, warp, first_q);
    const uint32_t n_blocks = end - begin;
    Copy copy{nullptr, 0};
    auto fill = [&](uint32_t k) {
        if (k >= n_blocks)
            return;
        if (k % 16 == 0) {
            const uint32_t x = begin + k + lane / 2;
            copy = x < end ? find_copy(a, s_pre, grp, R, kCell, x, warp * kPair, lane & 1)
                           : Copy{nullptr, 0};
        }
        if (lane / 2 == int(k % 16)) {
            uint8_t *to = ring + k % kStages * (2 * kCell) + (lane & 1) * kCell;
            uint64_t *bar = full + k % kStages;
            if (copy.bytes < 0) {
                // the tokens of a page outside the cache count as zeros
                for (int i = 0; i < -copy.bytes; i += 16)
                    *reinterpret_cast<uint4 *>(to + i) = make_uint4(0, 0, 0, 0);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            ptx::mbar_arrive_expect_tx(bar, uint32_t(max(copy.bytes, 0)));
            if (copy.bytes > 0)
                ptx::bulk_load(to, copy.src, uint32_t(copy.bytes), bar);
        }
    };
    // Failure-detection test: in the range that holds the line's middle the first warp's
    // first pair is to wait for 16 bytes that no copy brings.
    if (a.expire_wait_ns != 0u && tid == 0 && begin <= T / 2 && T / 2 < end) {
        s_limit = a.expire_wait_ns;
        ptx::mbar_expect_tx(full, 16);
    }
    for (uint32_t k = 0; k < kStages; ++k)
        fill(k);
    const uint32_t ring_at = ptx::smem_u32(ring);
    bool stuck = false;                    // a wait ran out, at block `done`
    uint32_t done = n_blocks;

    // this lane's places in a cell
    uint32_t at_K = ring_at + lane * (4 * NJ);
    uint32_t at_par = ring_at + kv4::k_par_off(D) + g * (4 * NG);
    uint32_t at_V[4];                      // of tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        at_V[x] = ring_at + kv4::v_off(D) +
                  kv4::v_swizzle((2 * c + (x & 1) + 8 * (x >> 1)) * (D / 2) + g * (D / 16));
        if (x < kVBases)
            keep(at_V[x]);
    }
    uint32_t at_Q = ptx::smem_u32(&s_q.frag[0][0][lane]);
    keep(at_K);
    keep(at_par);
    keep(at_Q);

    if (warp < NT)
        place_queries<D, G, NT, E>(a, it, grp, warp, first_q, s_q);
    sync_crew();
    for (uint32_t cur = begin; cur < end;) {
        const uint32_t stop = min(end, it.first + it.nb);
        const int rows = min(R, it.nq * grp - it.tile * R);         // rows of this tile
        float mul[NT][E], qbar[NT][NG][E];     // of columns 2 c, 2 c + 1 of n-tile nt
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int r = nt * 8 + 2 * c + e;
                mul[nt][e] = s_q.mul[r];
#pragma unroll
                for (int x = 0; x < NG; ++x)
                    qbar[nt][x][e] = s_q.bar[x][r];
            }

        // ---- the keys ----------------------------------------------------------
        float O[NT][D / 16][4], ref[NT][E], sum[NT][E], pm[NT][NG][E], up[NT][NG][E];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
                O[nt][x][0] = O[nt][x][1] = O[nt][x][2] = O[nt][x][3] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                ref[nt][e] = kNoRef;
                sum[nt][e] = 0.f;
#pragma unroll
                for (int x = 0; x < NG; ++x) {
                    pm[nt][x][e] = 0.f;
                    up[nt][x][e] = 1.f;
                }
            }
        }
        // The keys of kCells cells, from token `tok` on.  kMasked: some query row of
        // the tile does not see all of them, or the sequence ends among them.
        const int tok_end = key_end(a, it, (it.tile * R + rows - 1) / grp);
        auto step = [&](uint32_t slot, int tok, auto masked_tag) {
            constexpr bool kMasked = decltype(masked_tag)::value;
            constexpr int NC = kCells;
            constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;
            // S^T = K Q^T: lane (g, c) holds tokens g, g + 8 of each cell
            uint32_t kw[NC][2][NJ];
            load_tokens<NC, kCell, 0, 8 * (D / 2)>(kw, at_K + slot);
            float acc[NC][NT][NG][4];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                uint32_t a0[NC][4], a1[NC][4];
#pragma unroll
                for (int x = 0; x < NC; ++x) {
                    const uint32_t w0 = kw[x][0][j], w1 = kw[x][1][j];
                    const uint32_t y0 = w0 >> 8, y1 = w1 >> 8;
                    a0[x][0] = w0 & kLo, a0[x][1] = w1 & kLo, a0[x][2] = w0 & kHi,
                    a0[x][3] = w1 & kHi;
                    a1[x][0] = y0 & kLo, a1[x][1] = y1 & kLo, a1[x][2] = y0 & kHi,
                    a1[x][3] = y1 & kHi;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t q[4];
                    load_shared<0>(q, at_Q + (nt * NJ + j) * 512);
#pragma unroll
                    for (int x = 0; x < NC; ++x) {
                        float (&to)[4] = acc[x][nt][32 * j / G];
                        if (32 * j % G == 0)
                            mma_first(to, a0[x], q[0], q[1]);
                        else
                            mma(to, a0[x], q[0], q[1]);
                    }
#pragma unroll
                    for (int x = 0; x < NC; ++x)
                        mma(acc[x][nt][32 * j / G], a1[x], q[2], q[3]);
                }
            }
            // (scale, min) pairs of tokens g and g + 8
            uint32_t pk[NC][2][NG], pv[NC][2][NG];
            load_tokens<NC, kCell, 0, 32 * NG>(pk, at_par + slot);
            load_tokens<NC, kCell, 64 * NG, 32 * NG>(pv, at_par + slot);
            if constexpr (kMasked) {
                // behind the last key they may be anything, and count as 0
#pragma unroll
                for (int x = 0; x < NC; ++x)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (tok + 16 * x + g + 8 * t >= tok_end)
#pragma unroll
                            for (int y = 0; y < NG; ++y)
                                pk[x][t][y] = pv[x][t][y] = 0;
            }
            uint32_t pf[NC][NT][NG][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                bool seen[NC][2][E];
                // S - `from`, [token g, g + 8][column 2 c, 2 c + 1]
                auto score = [&](int x, int t, int e, float from) {
                    float s = bf16_lo(pk[x][t][0]) * acc[x][nt][0][2 * t + e], y = -from;
#pragma unroll
                    for (int gr = 1; gr < NG; ++gr)
                        s = fmaf(bf16_lo(pk[x][t][gr]), acc[x][nt][gr][2 * t + e], s);
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr)
                        y = fmaf(bf16_hi(pk[x][t][gr]), qbar[nt][gr][e], y);
                    return seen[x][t][e] ? fmaf(s, mul[nt][e], y) : -INFINITY;
                };
                float P[NC][2][E];
                // P s in fp16; whether one outgrew its power of two
                auto weigh = [&] {
                    float over = 0.f;
#pragma unroll
                    for (int x = 0; x < NC; ++x)
#pragma unroll
                        for (int y = 0; y < NG; ++y) {
                            float ps[2][2] = {{0.f, 0.f}, {0.f, 0.f}};     // [t][e]
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
#pragma unroll
                                for (int e = 0; e < E; ++e) {
                                    // (a product with s first might be infinite where P is 0)
                                    ps[t][e] = P[x][t][e] * up[nt][y][e] * bf16_lo(pv[x][t][y]);
                                    // a key that the row does not see adds nothing,
                                    // whatever its parameters are
                                    if (kMasked && !seen[x][t][e])
                                        ps[t][e] = 0.f;
                                }
                                if (E == 2)
                                    over = max3(over, ps[t][0], ps[t][1]);
                                pf[x][nt][y][t] = pack_f16(ps[t][0], ps[t][1]);
                            }
                            if (E == 1)
                                over = max3(over, ps[0][0], ps[1][0]);
                        }
                    return over > kMostPs;
                };
                float over = 0.f;
#pragma unroll
                for (int x = 0; x < NC; ++x)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            seen[x][t][e] = !kMasked || tok + 16 * x + g + 8 * t <
                                                            s_q.end[nt * 8 + 2 * c + e];
                            P[x][t][e] = ptx::ex2(score(x, t, e, ref[nt][e]));
                        }
                        if (E == 2)
                            over = max3(over, P[x][t][0], P[x][t][E - 1]);
                        else if (t == 1)
                            over = max3(over, P[x][0][0], P[x][1][0]);
                    }
                if (__any_sync(0xffffffffu, weigh() || over > kMostP)) {
                    // a row outgrew its reference, or a group its power of two: all go by
                    // the largest seen
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        float S[NC][2], m = ref[nt][e];
#pragma unroll
                        for (int x = 0; x < NC; ++x)
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                S[x][t] = score(x, t, e, 0.f);
                                m = fmaxf(m, S[x][t] + kRefAbove);
                            }
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        const float f = ptx::ex2(ref[nt][e] - m);
                        ref[nt][e] = m;
                        sum[nt][e] *= f;
#pragma unroll
                        for (int x = 0; x < NC; ++x)
#pragma unroll
                            for (int t = 0; t < 2; ++t)
                                P[x][t][e] = ptx::ex2(S[x][t] - m);
                        // the upper halves of two groups' largest P s a word
                        uint32_t big[(NG + 1) / 2] = {};
#pragma unroll
                        for (int y = 0; y < NG; ++y) {
                            float top = 0x1p7f * f * inverse(up[nt][y][e]);
#pragma unroll
                            for (int x = 0; x < NC; ++x)
                                top = max3(top, P[x][0][e] * bf16_lo(pv[x][0][y]),
                                           P[x][1][e] * bf16_lo(pv[x][1][y]));
                            big[y / 2] = __byte_perm(big[y / 2], __float_as_uint(top),
                                                     y % 2 ? 0x7610 : 0x3276);
                        }
#pragma unroll
                        for (int y = 0; y < (NG + 1) / 2; ++y)
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1)
                                big[y] = __vmaxu2(big[y], __shfl_xor_sync(0xffffffffu, big[y], o));
#pragma unroll
                        for (int y = 0; y < NG; ++y) {
                            const int log = 134 - int(y % 2 ? big[y / 2] >> 23 : big[y / 2] >> 7 & 255);
                            const float old = inverse(up[nt][y][e]);
                            up[nt][y][e] = pow2(max(-kMostUp, min(kMostUp, log)));
                            const float r = f * up[nt][y][e] * old;
                            pm[nt][y][e] *= f;
#pragma unroll
                            for (int q = 2 * y * (G / 32); q < 2 * (y + 1) * (G / 32); ++q) {
                                O[nt][q][e] *= r;
                                O[nt][q][2 + e] *= r;
                            }
                        }
                    }
                    weigh();
                }
#pragma unroll
                for (int x = 0; x < NC; ++x) {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        sum[nt][e] += P[x][0][e] + P[x][1][e];
#pragma unroll
                    for (int y = 0; y < NG; ++y)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
#pragma unroll
                            for (int e = 0; e < E; ++e) {
                                const float z =
                                    fmaf(P[x][t][e], bf16_hi(pv[x][t][y]), pm[nt][y][e]);
                                if (!kMasked || seen[x][t][e])
                                    pm[nt][y][e] = z;
                            }
                            pf[x][nt][y][t] = transpose8x8(pf[x][nt][y][t]);
                        }
                }
            }

            // O^T += V^T P^T: lane (g, c) holds its halves of tokens 2 c, 2 c + 1,
            // 2 c + 8, 2 c + 9; a half-word pair of two tokens is one A register
            uint32_t v[NC][4][D / 64];
            constexpr int kUp = kVBases == 2 ? 8 * (D / 2) : 0;
            load_values<NC, kCell, 0>(v, 0, at_V[0] + slot);
            load_values<NC, kCell, 0>(v, 1, at_V[1] + slot);
            load_values<NC, kCell, kUp>(v, 2, at_V[2 % kVBases] + slot);
            load_values<NC, kCell, kUp>(v, 3, at_V[3 % kVBases] + slot);
#pragma unroll
            for (int x = 0; x < NC; ++x)
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    const uint32_t sel = (q & 1) ? 0x7632 : 0x5410;
                    const uint32_t u = __byte_perm(v[x][0][q / 2], v[x][1][q / 2], sel);
                    const uint32_t y = __byte_perm(v[x][2][q / 2], v[x][3][q / 2], sel);
                    const uint32_t u8 = u >> 8, y8 = y >> 8;
                    const uint32_t a0[4] = {u & kLo, u & kHi, y & kLo, y & kHi};
                    const uint32_t a1[4] = {u8 & kLo, u8 & kHi, y8 & kLo, y8 & kHi};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t (&b)[2] = pf[x][nt][32 * q / G];
                        mma(O[nt][2 * q], a0, b[0], b[1]);
                        mma(O[nt][2 * q + 1], a1, b[0], b[1]);
                    }
                }
        };
        auto both = [&](uint32_t slot, int tok, auto masked_tag) {
#pragma unroll 1
            for (int x = 0; x < 2; x += kCells)
                step(slot + x * kCell, tok + x * kv4::kCellTokens, masked_tag);
        };
        const int all_end = key_end(a, it, it.tile * R / grp);   // all rows see the keys below
        int tok = int(cur - it.first) * kBlock + warp * kPair;
        uint32_t k = cur - begin;
        const uint32_t k_stop = stop - begin;
        const int n_full = max(0, (all_end - kPair - tok + kBlock) / kBlock);
        const uint32_t k_full = min(k_stop, k + uint32_t(n_full));
        auto landed = [&] {                // else the error is recorded and the crew writes
                                           // nothing of this item and the later ones
            stuck = stuck || !wait_pair(full + k % kStages, k / kStages & 1, &s_abort, a.err_word);
            done = stuck ? min(done, k) : done;
            return !stuck;
        };
        for (; k < k_full && landed(); ++k, tok += kBlock) {
            both(k % kStages * (2 * kCell), tok, std::false_type{});
            __syncwarp();                  // every lane has read the cells
            fill(k + kStages);
        }
        for (; k < k_stop && landed(); ++k, tok += kBlock) {
            if (tok < tok_end)
                both(k % kStages * (2 * kCell), tok, std::true_type{});
            __syncwarp();
            fill(k + kStages);
        }

        // ---- the warps' parts joined, and written ----------------------------
        // the next item's queries are on their way meanwhile
        const Item next = stop < end ? next_item(a, s_pre, grp, R, it) : it;
        uint4 qw[NJ];
        if (warp < NT && stop < end)
            fetch_queries<D, NT, E>(a, next, grp, warp, qw);
        else
            for (int j = 0; j < NJ; ++j)
                qw[j] = make_uint4(0, 0, 0, 0);
        const bool whole = cur == it.first && stop == it.first + it.nb;
        const int slot = 2 * id + (cur == it.first ? 1 : 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < E; ++e) {
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
                    s_ref[warp * kCols + nt * 8 + 2 * c + e] = ref[nt][e];
                    s_sum[warp * kCols + nt * 8 + 2 * c + e] = s;
                }
            }
        sync_crew();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // the upper warps' rows through shared memory into the lower warps'
            // registers, then the lower warps' rows for all to sum
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (warp / (kWarps / 2) == 1 - half) {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int col = nt * 8 + 2 * c + e;
                        float m = s_ref[col];
#pragma unroll
                        for (int w = 1; w < kWarps; ++w)
                            m = fmaxf(m, s_ref[w * kCols + col]);
                        const float f = ptx::ex2(ref[nt][e] - m);
                        float *row = s_O + (warp % (kWarps / 2) * 8 + 2 * c + e) * kRow + 4 * g;
#pragma unroll
                        for (int q = 0; q < D / 32; ++q) {
                            const float p = pm[nt][32 * q / G][e];
                            const float down = inverse(up[nt][32 * q / G][e]);
                            float4 y =
                                make_float4(fmaf(O[nt][2 * q][e] * 0x1p24f, down, p) * f,
                                            fmaf(O[nt][2 * q][2 + e] * 0x1p20f, down, p) * f,
                                            fmaf(O[nt][2 * q + 1][e] * 0x1p24f, down, p) * f,
                                            fmaf(O[nt][2 * q + 1][2 + e] * 0x1p20f, down, p) * f);
                            float4 *at = reinterpret_cast<float4 *>(row + 32 * q);
                            if (half == 1) {
                                const float4 z = *at;
                                y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
                            }
                            *at = y;
                        }
                    }
                } else if (half == 0 && nt == 0 && warp < NT && stop < end) {
                    place_queries<D, G, NT, E>(a, next, grp, warp, qw, s_q);
                }
                sync_crew();
            }
            // the rows' D values over the threads, four consecutive values each
            for (int x = tid; x < 4 * E * (D / 4); x += kThreads) {
                const int rr = x / (D / 4) * (2 / E), d4 = x % (D / 4) * 4;
                const int col = nt * 8 + rr, r = row_of<E>(col);
                float4 y = *reinterpret_cast<const float4 *>(s_O + rr * kRow + d4);
                float m = s_ref[col];
#pragma unroll
                for (int w = 1; w < kWarps / 2; ++w) {
                    const float4 z =
                        *reinterpret_cast<const float4 *>(s_O + (w * 8 + rr) * kRow + d4);
                    y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
                }
#pragma unroll
                for (int w = 1; w < kWarps; ++w)
                    m = fmaxf(m, s_ref[w * kCols + col]);
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    s = fmaf(s_sum[w * kCols + col], ptx::ex2(s_ref[w * kCols + col] - m), s);
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
            sync_crew();
        }
        if (cur == it.first && !whole) {
            desc.item_end = it.first + it.nb;
            desc.b = it.b;
            desc.kvh = it.kvh;
            desc.tile = it.tile;
        }
        cur = stop;
        it = next;
    }
    if (s_abort) {
        // a wait ran out: the join leaves out the items that have a part here, and the
        // copies under way must land before the crew ends
        desc.item_end = 0;
        desc.aborted = 1;
        if (a.expire_wait_ns != 0u && tid == 0 && begin <= T / 2 && T / 2 < end)
            ptx::mbar_complete_tx(full, 16);
        for (uint32_t k = done; k < min(done + kStages, n_blocks); ++k) {
            volatile int go_on = 0;
            ptx::mbar_wait_limited(full + k % kStages, k / kStages & 1, &go_on, a.err_word,
                                   kWaitTimeoutNs);
        }
    }
    if (tid == 0 && !a.whole_items)
        parts.desc[id] = desc;
}

// Joins the parts of the items that span ranges: blocks (x, *) the item that begins
// in range x and does not end there, kPart warps a row.  The warps of a row
// take every kPart-th part, eight loads of O under way at a time, and their sums
// are added in the order of the warps.  Few items have many parts each and take
// 8 warps a row (1 x 130001 keys in 76 parts: 28 us with one, 7 with eight); many
// items have a few and take one (64 x 8 items: 6 us, with eight 10).  An item with a
// part in a range where a wait ran out is not written: parts of it may be missing.
template <int D, int R, int kPart>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_kv4_join_kernel(const Kv4AttnArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kPer = D / 32;
    constexpr int kRows = kJoinWarps / kPart;      // of a block
    __shared__ float s_y[kJoinWarps][D], s_m[kJoinWarps], s_s[kJoinWarps];
    const Parts parts = parts_of<D, R>(a.workspace);
    const Desc desc = parts.desc[blockIdx.x];
    if (desc.item_end == 0)
        return;
    const int2 qb = queries_of(a, desc.b);
    const int grp = a.H / a.Hkv, all = qb.y * grp, row0 = desc.tile * R + blockIdx.y * kRows;
    if (row0 >= all)
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.y * kRows + warp / kPart;
    // the first part lies in its range's slot 1, the others in their ranges' slot 0
    auto place = [&](int p) { return (int64_t(2) * (blockIdx.x + p) + (p == 0)) * R + r; };
    // lane l: reference and sum of the warp's l-th part of 32
    float m = kNoRef, s = 0.f, y[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e)
        y[e] = 0.f;
    // the ranges from this one on that begin before the item's end
    int n_parts = 0;
    bool aborted = false;
    for (uint32_t in = ~0u; in == ~0u; n_parts += __popc(in)) {
        const uint32_t x = blockIdx.x + n_parts + lane;
        const bool part = x < gridDim.x && parts.desc[x].begin < desc.item_end;
        aborted = aborted || (part && parts.desc[x].aborted);
        in = __ballot_sync(0xffffffffu, part);
    }
    if (__any_sync(0xffffffffu, aborted))  // in every warp of the block alike
        return;
    if (desc.tile * R + r >= all)
        n_parts = 0;
    for (int p0 = warp % kPart; p0 < n_parts; p0 += 32 * kPart) {
        const int n = min(32, (n_parts - p0 + kPart - 1) / kPart);
        float2 ml = make_float2(kNoRef, 0.f);
        if (lane < n)
            ml = parts.ml[place(p0 + lane * kPart)];
        float top = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, m);
        const float old = ptx::ex2(m - top), f = lane < n ? ptx::ex2(ml.x - top) : 0.f;
        m = top;
        s = fmaf(ml.y, f, s * old);
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            y[e] *= old;
        for (int u0 = 0; u0 < n; u0 += 8) {
            float v[8][kPer];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float *src =
                    parts.O + place(p0 + min(u0 + u, n - 1) * kPart) * D + lane * kPer;
#pragma unroll
                for (int e = 0; e < kPer; e += 2) {
                    const float2 z = *reinterpret_cast<const float2 *>(src + e);
                    v[u][e] = z.x;
                    v[u][e + 1] = z.y;
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float w = __shfl_sync(0xffffffffu, f, (u0 + u) & 31);
                if (u0 + u < n)
#pragma unroll
                    for (int e = 0; e < kPer; ++e)
                        y[e] = fmaf(v[u][e], w, y[e]);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
    for (int e = 0; e < kPer; ++e)
        s_y[warp][lane * kPer + e] = y[e];
    if (lane == 0) {
        s_m[warp] = m;
        s_s[warp] = s;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kRows * D; e += kJoinWarps * 32) {
        const int w0 = e / D * kPart, x = e % D, at = row0 + e / D;
        if (at >= all)
            break;
        m = s_m[w0];
#pragma unroll
        for (int w = 1; w < kPart; ++w)
            m = fmaxf(m, s_m[w0 + w]);
        s = 0.f;
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < kPart; ++w) {
            const float f = ptx::ex2(s_m[w0 + w] - m);
            s = fmaf(s_s[w0 + w], f, s);
            o = fmaf(s_y[w0 + w][x], f, o);
        }
        const int i = at / grp, h = desc.kvh * grp + at % grp;
        const bool any = s > 0.f || s != s;
        static_cast<__nv_bfloat16 *>(a.O)[(int64_t(qb.x + i) * a.H + h) * D + x] =
            __float2bfloat16_rn(any ? o / s : 0.f);
        if (x == 0)
            a.lse[a.cu_seqlens_q ? int64_t(h) * a.total_q + qb.x + i
                                 : (int64_t(desc.b) * a.H + h) * a.Nq + i] =
                any ? (m + log2f(s)) * kLn2 : -INFINITY;
    }
}

template <int D, int G, int NT, int E>
int launch(const Kv4AttnArgs &a, cudaStream_t stream)
{
    constexpr int R = 4 * NT * E;
    constexpr int smem = Shared<D, G, NT>::all;
    static PerDeviceOnce once;
    if (!set_max_dynamic_smem(once, reinterpret_cast<const void *>(attn_kv4_kernel<D, G, NT, E>), smem))
        return FA_ERR_CUDA;
    constexpr int ranges = kv4_attention_ranges(R, D);
    if (launch_early(attn_kv4_kernel<D, G, NT, E>, dim3(kv4_attention_sms),
                     kThreads * kv4_attention_crews(R, D), smem, stream, a) != cudaSuccess)
        return FA_ERR_CUDA;
    if (a.whole_items)
        return FA_OK;                      // no parts
    const int64_t all_rows = int64_t(a.Nq) * (a.H / a.Hkv), items = int64_t(a.B) * a.Hkv *
                                                                  ((all_rows + R - 1) / R);
    const int rows = int(all_rows < R ? all_rows : R);
    const bool few = 16 * items <= ranges;
    const dim3 grid(ranges, few ? rows : (rows + kJoinWarps - 1) / kJoinWarps);
    const cudaError_t e =
        few ? launch_early(attn_kv4_join_kernel<D, R, kJoinWarps>, grid, kJoinWarps * 32, 0, stream, a)
            : launch_early(attn_kv4_join_kernel<D, R, 1>, grid, kJoinWarps * 32, 0, stream, a);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, int G>
int launch_rows(const Kv4AttnArgs &a, cudaStream_t stream)
{
    // Rows beyond 16 go on as further tiles, whose keys come from L2 the second
    // time.  Tiles of 32 rows, one cell at a time, take the same time where their rows
    // are filled (16 sequences x 4 queries x 8 heads a kv head: 66 us) and more where
    // not (5 queries: 109 us, so 88).
    switch (kv4_attention_rows(a.Nq, a.H, a.Hkv)) {
    case 4: return launch<D, G, 1, 1>(a, stream);
    case 8: return launch<D, G, 1, 2>(a, stream);
    default: return launch<D, G, 2, 2>(a, stream);
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
