// kv4_cache.cu -- writing K and V rows into the 4-bit paged cache, and reading
// them back as bf16.
//
// Writing: per group of `group` values m = min, s = bf16((max/2 - min/2) *
// f32(2/15)), code = rint((x/2 - m/2) * (1 / (s/2))).  m is one of the bf16
// inputs, so storing it in bf16 loses nothing; s loses half a step of bf16
// (2^-8), 0.06 of a code at the far end of the range.  Halving first keeps
// max - min finite for every pair of finite inputs.  Reading: m + s * code,
// rounded once to bf16.
//
// Both are bound by HBM: 4 d bytes of K and V and d + 8 d / group bytes of the
// cache per token and head.  A thread takes 16 values: the two words c of value
// blocks 2 jj and 2 jj + 1 of 32 (kv4.cuh), which stand side by side in a K row
// and whose halves pair up in a V row, so that no codes change lanes.  d / 16
// threads hold a row of a head, the group's extremes come from 2 or 3 shuffles of
// (min x, min -x), and a row's scale is found for 16 values at a time: with 8 a
// thread the quantising took more issue slots than the copy leaves.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/fa.h"
#include "fa_error.cuh"
#include "kv4.cuh"
#include "launch.h"

namespace fa {
namespace {

using kv4::bf16_hi;
using kv4::bf16_lo;

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 5;

// What a block needs to know of one of its rows.
struct RowAt {
    int64_t cell;   // byte offset in the cache of head 0's cell, or -1: skip the row
    int t;          // token within the cell
};

// Whether a sequence of n new rows from row c0 on, with L tokens in the end, is allowed.
__device__ __forceinline__ bool counts_fit(const Kv4CacheArgs &a, int64_t c0, int64_t n, int64_t L)
{
    return c0 >= 0 && n >= 0 && n <= a.N && c0 + n <= a.total && L >= n &&
           L <= int64_t(a.max_pages) * a.page_size;
}

// Records what no row shows: packed sequences without a row, or with rows that another
// one claims.  The first block looks, its last warps first: the first ones look for their
// rows meanwhile.
__device__ __forceinline__ void check_counts(const Kv4CacheArgs &a)
{
    if (a.cu_seqlens == nullptr || blockIdx.x != 0 || blockIdx.y != 0)
        return;
    for (int b = kThreads - 1 - int(threadIdx.x); b < a.B; b += kThreads) {
        const int64_t c0 = a.cu_seqlens[b];
        if (!counts_fit(a, c0, a.cu_seqlens[b + 1] - c0, a.seqlens[b]))
            record_device_error(a.err_word, FA_DEVERR_BAD_SEQLENS);
    }
}

// The place of packed row r: its sequence, its position (the rows of sequence
// b are its last n_b tokens), its page.
__device__ RowAt locate(const Kv4CacheArgs &a, int64_t r, int cell)
{
    RowAt at{-1, 0};
    int b;
    int64_t i, n;
    if (a.cu_seqlens == nullptr) {
        b = int(r / a.N);
        i = r - int64_t(b) * a.N;
        n = a.N;
    } else {
        int lo = 0, hi = a.B;   // last b with cu[b] <= r
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu_seqlens[mid] <= r)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
        const int64_t c0 = a.cu_seqlens[b], c1 = a.cu_seqlens[b + 1];
        if (r < c0 || r >= c1)
            return at;          // behind the last sequence
        i = r - c0;
        n = c1 - c0;
    }
    const int64_t L = a.seqlens[b];
    if (!counts_fit(a, r - i, n, L)) {
        record_device_error(a.err_word, FA_DEVERR_BAD_SEQLENS);
        return at;
    }
    const int pos = int(L - n + i);
    const int page = a.page_table[int64_t(b) * a.max_pages + pos / a.page_size];
    if (page < 0 || page >= a.num_pages) {
        record_device_error(a.err_word, FA_DEVERR_BAD_PAGE);
        return at;
    }
    const int cells = a.page_size / kv4::kCellTokens, in_page = pos % a.page_size;
    at.cell = (int64_t(page) * a.Hkv * cells + in_page / kv4::kCellTokens) * cell;
    at.t = in_page % kv4::kCellTokens;
    return at;
}

__device__ __forceinline__ uint32_t min_nan2(uint32_t x, uint32_t y)
{
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

__device__ __forceinline__ uint32_t max_nan2(uint32_t x, uint32_t y)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

// (min x, min -x) of 8 values, in the two halves of a word.
__device__ __forceinline__ uint32_t extremes(const uint4 &x)
{
    const uint32_t lo = min_nan2(min_nan2(x.x, x.y), min_nan2(x.z, x.w));
    const uint32_t hi = max_nan2(max_nan2(x.x, x.y), max_nan2(x.z, x.w)) ^ 0x80008000u;
    return min_nan2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
}

// A group's (scale, min) pair as stored, min / 2 and 1 / (scale / 2).
struct Scale {
    uint32_t pair;
    float half_min, inv;
    bool bad;
};

__device__ __forceinline__ Scale scale_of(uint32_t ext)
{
    Scale r;
    const float m = bf16_lo(ext), mx = -bf16_hi(ext);
    r.half_min = 0.5f * m;
    const float s32 = __fmul_rn(__fsub_rn(0.5f * mx, r.half_min), 2.0f / 15.0f);
    float s = __bfloat162float(__float2bfloat16_rn(s32));
    s = s < 1.17549435e-38f ? 0.f : s;           // below 2^-126: all codes 0
    r.inv = s > 0.f ? __frcp_rn(0.5f * s) : 0.f;
    r.bad = !(fabsf(m) < INFINITY && fabsf(mx) < INFINITY);
    r.pair = r.bad ? 0x7fc07fc0u : (__float_as_uint(s) >> 16) | (__float_as_uint(m) & 0xffff0000u);
    return r;
}

// The codes of 8 values, lowest nibble first.  (x - m) / s is in [0, 15.06], so
// rint needs no clamp; adding 1.5 * 2^23 rounds to nearest even and leaves the
// code in the low bits of a word 0x4b400000 + code, whose sum over the nibbles
// exceeds the codes by 0x3f400000 (mod 2^32).
__device__ __forceinline__ uint32_t codes_of(const uint4 &x, const Scale &s)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t sum = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        const float t1 = fmaf(bf16_hi(w[i]), 0.5f, -s.half_min);   // = rn(x / 2 - m / 2)
        const float t0 = fmaf(bf16_lo(w[i]), 0.5f, -s.half_min);
        sum = sum * 16 + __float_as_uint(__fadd_rn(__fmul_rn(t1, s.inv), 12582912.f));
        sum = sum * 16 + __float_as_uint(__fadd_rn(__fmul_rn(t0, s.inv), 12582912.f));
    }
    return s.bad ? 0u : sum - 0x3f400000u;
}

// What a thread does in every row: its head, its 16 values, their places.
template <int D, int G>
struct Part {
    static constexpr int kCell = kv4::cell_bytes(D, G), kLanes = D / 16, kN = D / 32;
    int h, jj, c;
    bool is_v;
    int64_t head;              // byte offset of the head's page from head 0's

    __device__ __forceinline__ Part(const Kv4CacheArgs &a, int p)
    {
        const int l = p % kLanes, h2 = p / kLanes;
        is_v = h2 >= a.Hkv;
        h = is_v ? h2 - a.Hkv : h2;
        jj = l / 4;
        c = l % 4;
        head = int64_t(h) * (a.page_size / kv4::kCellTokens) * kCell;
    }
    // element of the row at which word w = 4 (2 jj + x) + c begins
    __device__ __forceinline__ int element(int x) const { return h * D + (4 * (2 * jj + x) + c) * 8; }
    // byte of the cell at which the thread's K words, or its first V word, stand
    __device__ __forceinline__ int code_at(int t) const
    {
        return is_v ? kv4::v_off(D) + kv4::v_swizzle(t * (D / 2) + c * (kN * 4) + jj * 4)
                    : t * (D / 2) + (c * kN + 2 * jj) * 4;
    }
    // the second V word: halves of g = 2 c + 1
    static constexpr int kSecond = kN * 2;
    __device__ __forceinline__ int pair_at(int t) const
    {
        return (is_v ? kv4::v_par_off(D, G) : kv4::k_par_off(D)) +
               (t * (D / G) + (G == 32 ? 2 * jj : G == 64 ? jj : 0)) * 4;
    }
};

constexpr int kUnroll = 2;     // rows a thread has under way

// Grid: x over the rows, rows_per_block each; y over a row's threads (2 Hkv d / 16)
// beyond kThreads.
template <int D, int G>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    kv4_append_kernel(const Kv4CacheArgs a, int rows_per_block)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ RowAt at[];
    check_counts(a);
    const int64_t row0 = int64_t(blockIdx.x) * rows_per_block;
    const int rows = int(min(int64_t(rows_per_block), a.total - row0));
    for (int i = threadIdx.x; i < rows; i += kThreads)
        at[i] = locate(a, row0 + i, Part<D, G>::kCell);
    __syncthreads();
    const int all = 2 * a.Hkv * (D / 16), p0 = blockIdx.y * kThreads;
    const int width = min(all - p0, kThreads), side = kThreads / width;   // rows side by side
    const bool in = int(threadIdx.x) < width * side;
    const Part<D, G> part(a, p0 + threadIdx.x % width);
    const int64_t stride = part.is_v ? a.v_stride : a.k_stride;
    const auto *src = static_cast<const __nv_bfloat16 *>(part.is_v ? a.V : a.K) + row0 * stride;
    uint8_t *cache = static_cast<uint8_t *>(a.cache) + part.head;
    for (int r0 = 0; r0 < rows; r0 += side * kUnroll) {
        uint4 x[kUnroll][2];
        RowAt w[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int row = r0 + u * side + int(threadIdx.x) / width;
            w[u] = in && row < rows ? at[row] : RowAt{-1, 0};
            x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
            if (w[u].cell >= 0) {
                x[u][0] = *reinterpret_cast<const uint4 *>(src + row * stride + part.element(0));
                x[u][1] = *reinterpret_cast<const uint4 *>(src + row * stride + part.element(1));
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            // the lanes of a group: c = 0 .. 3, and jj with 128 values
            uint32_t e0 = extremes(x[u][0]), e1 = extremes(x[u][1]);
            if (G > 32)
                e0 = min_nan2(e0, e1);
#pragma unroll
            for (int o = 1; o < (G == 128 ? 8 : 4); o <<= 1) {
                e0 = min_nan2(e0, __shfl_xor_sync(0xffffffffu, e0, o));
                if (G == 32)
                    e1 = min_nan2(e1, __shfl_xor_sync(0xffffffffu, e1, o));
            }
            const Scale s0 = scale_of(e0), s1 = G == 32 ? scale_of(e1) : s0;
            const uint32_t c0 = codes_of(x[u][0], s0), c1 = codes_of(x[u][1], s1);
            if (w[u].cell < 0)
                continue;
            uint8_t *cell = cache + w[u].cell;
            uint8_t *to = cell + part.code_at(w[u].t);
            if (part.is_v) {
                *reinterpret_cast<uint32_t *>(to) = __byte_perm(c0, c1, 0x5410);
                *reinterpret_cast<uint32_t *>(to + part.kSecond) = __byte_perm(c0, c1, 0x7632);
            } else {
                *reinterpret_cast<uint2 *>(to) = make_uint2(c0, c1);
            }
            if (part.c == 0 && (G != 128 || part.jj == 0)) {
                uint8_t *p = cell + part.pair_at(w[u].t);
                if (G == 32)
                    *reinterpret_cast<uint2 *>(p) = make_uint2(s0.pair, s1.pair);
                else
                    *reinterpret_cast<uint32_t *>(p) = s0.pair;
            }
        }
    }
}

// min + scale * code of 8 codes: nibbles i and i + 4 as the bf16 pair 128 + code,
// exact, less 128; then one rounding.
__device__ __forceinline__ uint4 values_of(uint32_t code, uint32_t pair)
{
    const uint32_t s2 = __byte_perm(pair, pair, 0x1010), m2 = __byte_perm(pair, pair, 0x3232);
    const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162 *>(&s2);
    const __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162 *>(&m2);
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = ((code >> (4 * i)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 c = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&u),
                                         __float2bfloat162_rn(128.f));
        const __nv_bfloat162 y = __hfma2(s, c, m);
        v[i] = *reinterpret_cast<const uint32_t *>(&y);
    }
    return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                      __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

// The same lay-out, the other way.
template <int D, int G>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    kv4_read_kernel(const Kv4CacheArgs a, int rows_per_block)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ RowAt at[];
    check_counts(a);
    const int64_t row0 = int64_t(blockIdx.x) * rows_per_block;
    const int rows = int(min(int64_t(rows_per_block), a.total - row0));
    for (int i = threadIdx.x; i < rows; i += kThreads)
        at[i] = locate(a, row0 + i, Part<D, G>::kCell);
    __syncthreads();
    const int all = 2 * a.Hkv * (D / 16), p0 = blockIdx.y * kThreads;
    const int width = min(all - p0, kThreads), side = kThreads / width;
    if (int(threadIdx.x) >= width * side)
        return;
    const Part<D, G> part(a, p0 + threadIdx.x % width);
    const int64_t stride = part.is_v ? a.v_stride : a.k_stride;
    auto *dst = static_cast<__nv_bfloat16 *>(part.is_v ? a.V : a.K) + row0 * stride;
    const uint8_t *cache = static_cast<const uint8_t *>(a.cache) + part.head;
    for (int r0 = threadIdx.x / width; r0 < rows; r0 += side * kUnroll) {
        uint32_t c0[kUnroll], c1[kUnroll], p[kUnroll][2];
        bool put[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int row = r0 + u * side;
            const RowAt w = row < rows ? at[row] : RowAt{-1, 0};
            put[u] = w.cell >= 0;
            if (!put[u])
                continue;
            const uint8_t *cell = cache + w.cell, *from = cell + part.code_at(w.t);
            if (part.is_v) {
                c0[u] = *reinterpret_cast<const uint32_t *>(from);
                c1[u] = *reinterpret_cast<const uint32_t *>(from + part.kSecond);
            } else {
                const uint2 z = *reinterpret_cast<const uint2 *>(from);
                c0[u] = z.x;
                c1[u] = z.y;
            }
            p[u][0] = *reinterpret_cast<const uint32_t *>(cell + part.pair_at(w.t));
            p[u][1] = G == 32 ? *reinterpret_cast<const uint32_t *>(cell + part.pair_at(w.t) + 4)
                              : p[u][0];
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!put[u])
                continue;
            const uint32_t a0 = part.is_v ? __byte_perm(c0[u], c1[u], 0x5410) : c0[u];
            const uint32_t a1 = part.is_v ? __byte_perm(c0[u], c1[u], 0x7632) : c1[u];
            auto *row = dst + (r0 + u * side) * stride;
            *reinterpret_cast<uint4 *>(row + part.element(0)) = values_of(a0, p[u][0]);
            *reinterpret_cast<uint4 *>(row + part.element(1)) = values_of(a1, p[u][1]);
        }
    }
}

template <typename F>
int launch_rows(F kernel, const Kv4CacheArgs &a, cudaStream_t stream)
{
    // One row a block while that fills the SMs (a decode step's few rows).  Beyond,
    // whole waves of the blocks that are resident at once, of 8 rounds or fewer
    // each: finding its rows' pages costs a block a microsecond or two.
    const int all = 2 * a.Hkv * (a.d / 16);
    const int side = all < kThreads ? kThreads / all : 1, round = kUnroll * side;
    const int64_t resident = 152 * kBlocksPerSm;
    const int64_t waves = (a.total + 8 * round * resident - 1) / (8 * round * resident);
    int64_t rows = (a.total + waves * resident - 1) / (waves * resident);
    if (rows > side)
        rows = (rows + round - 1) / round * round;
    const int64_t blocks = (a.total + rows - 1) / rows;
    if (blocks > 0x7fffffffLL)
        return FA_ERR_TOO_LARGE;
    const dim3 grid(unsigned(blocks), unsigned((all + kThreads - 1) / kThreads));
    return launch_early(kernel, grid, kThreads, int(rows * sizeof(RowAt)), stream, a, int(rows)) ==
                   cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

int launch_kv4_append(const Kv4CacheArgs &a, cudaStream_t stream)
{
    if (a.d == 64)
        return a.group == 32 ? launch_rows(kv4_append_kernel<64, 32>, a, stream)
                             : launch_rows(kv4_append_kernel<64, 64>, a, stream);
    return a.group == 32   ? launch_rows(kv4_append_kernel<128, 32>, a, stream)
           : a.group == 64 ? launch_rows(kv4_append_kernel<128, 64>, a, stream)
                           : launch_rows(kv4_append_kernel<128, 128>, a, stream);
}

int launch_kv4_read(const Kv4CacheArgs &a, cudaStream_t stream)
{
    if (a.d == 64)
        return a.group == 32 ? launch_rows(kv4_read_kernel<64, 32>, a, stream)
                             : launch_rows(kv4_read_kernel<64, 64>, a, stream);
    return a.group == 32   ? launch_rows(kv4_read_kernel<128, 32>, a, stream)
           : a.group == 64 ? launch_rows(kv4_read_kernel<128, 64>, a, stream)
                           : launch_rows(kv4_read_kernel<128, 128>, a, stream);
}

}  // namespace fa
