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
// cache per token and head.  A lane takes 8 values (16 bytes of K or V, one
// 4-byte word of codes), so d / 8 lanes hold a row of a head and the group's
// extremes come from log2(group / 8) shuffles; a warp's loads and stores cover
// whole 128-byte lines of K and V and whole rows of codes.  V's 16-bit halves
// are exchanged by two shuffles so that codes leave (arrive) in whole words.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/fa.h"
#include "fa_error.cuh"
#include "kv4.cuh"
#include "launch.h"

namespace fa {
namespace {

constexpr int kThreads = 256;

// What a block needs to know of one of its rows.
struct RowAt {
    int64_t cell;   // byte offset in the cache of head 0's cell, or -1: skip the row
    int t;          // token within the cell
};

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
        if (n > a.N) {
            record_device_error(a.err_word, FA_DEVERR_BAD_SEQLENS);
            return at;
        }
    }
    const int64_t L = a.seqlens[b];
    if (L < n || L > int64_t(a.max_pages) * a.page_size) {
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

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Codes of 8 values (one word) and the group's (scale, min) pair; the group's
// lanes are the G / 8 consecutive ones around this lane.
template <int G>
__device__ __forceinline__ uint32_t quantise(const uint4 &x, uint32_t &pair)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    // (min x, min -x) in the two halves of one word: one shuffle a step
    uint32_t lo2 = min_nan2(min_nan2(w[0], w[1]), min_nan2(w[2], w[3]));
    uint32_t hi2 = min_nan2(min_nan2(w[0] ^ 0x80008000u, w[1] ^ 0x80008000u),
                            min_nan2(w[2] ^ 0x80008000u, w[3] ^ 0x80008000u));
    uint32_t ext = min_nan2(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1)
        ext = min_nan2(ext, __shfl_xor_sync(0xffffffffu, ext, o));
    const float m = bf16_lo(ext), mx = -bf16_hi(ext);
    const float half_m = 0.5f * m;
    const float s32 = __fmul_rn(__fsub_rn(0.5f * mx, half_m), 2.0f / 15.0f);
    const __nv_bfloat16 sb = __float2bfloat16_rn(s32);
    float s = __bfloat162float(sb);
    s = s < 1.17549435e-38f ? 0.f : s;           // below 2^-126: all codes 0
    const float r = s > 0.f ? __fdiv_rn(1.f, 0.5f * s) : 0.f;
    const bool bad = !(fabsf(m) < INFINITY && fabsf(mx) < INFINITY);
    pair = bad ? 0x7fc07fc0u
               : (__float_as_uint(s) >> 16) | (__float_as_uint(m) & 0xffff0000u);
    // (x - m) / s is in [0, 15.06], so rint needs no clamp; adding 1.5 * 2^23
    // rounds to nearest even and leaves the code in the low bits
    uint32_t code = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float t0 = fmaf(bf16_lo(w[i]), 0.5f, -half_m);   // = rn(x/2 - m/2)
        const float t1 = fmaf(bf16_hi(w[i]), 0.5f, -half_m);
        const uint32_t c0 = __float_as_uint(__fadd_rn(__fmul_rn(t0, r), 12582912.f));
        const uint32_t c1 = __float_as_uint(__fadd_rn(__fmul_rn(t1, r), 12582912.f));
        code |= (c0 & 15u) << (8 * i) | (c1 & 15u) << (8 * i + 4);
    }
    return bad ? 0u : code;
}

// grid: blocks of `rows_per_block` rows.  A block's threads are laid over
// (row, K or V, head, 8 values); `per_row` = 2 Hkv d / 8 items a row.
template <int D, int G>
__global__ void __launch_bounds__(kThreads)
    kv4_append_kernel(const Kv4CacheArgs a, int rows_per_block)
{
    constexpr int kCell = kv4::cell_bytes(D, G), kLanes = D / 8, kN = D / 32;
    extern __shared__ RowAt at[];
    const int64_t row0 = int64_t(blockIdx.x) * rows_per_block;
    const int rows = int(min(int64_t(rows_per_block), a.total - row0));
    for (int i = threadIdx.x; i < rows; i += kThreads)
        at[i] = locate(a, row0 + i, kCell);
    __syncthreads();
    const int per_row = 2 * a.Hkv * kLanes, items = rows * per_row;
    const int head_stride = a.page_size / kv4::kCellTokens * kCell;
    // every lane of a warp takes part in the shuffles, the last ones idle
    for (int it = threadIdx.x; (it & ~31) < items; it += kThreads) {
        const bool in = it < items;
        const int row = in ? it / per_row : 0, p = in ? it - row * per_row : 0;
        const int l = p % kLanes, h2 = p / kLanes;
        const bool is_v = h2 >= a.Hkv;
        const int h = is_v ? h2 - a.Hkv : h2;
        const RowAt w = at[row];
        const bool put = in && w.cell >= 0;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (put) {
            const auto *src = static_cast<const __nv_bfloat16 *>(is_v ? a.V : a.K) +
                              (row0 + row) * (is_v ? a.v_stride : a.k_stride) + h * D + l * 8;
            x = __ldg(reinterpret_cast<const uint4 *>(src));
        }
        uint32_t pair;
        uint32_t code = quantise<G>(x, pair);
        // V: this lane's stored word l holds halves q * 8 + g and (q + 1) * 8 + g
        const int g = 2 * l / kN, q = 2 * l % kN;
        const uint32_t c0 = __shfl_sync(0xffffffffu, code, q * 4 + g / 2, kLanes);
        const uint32_t c1 = __shfl_sync(0xffffffffu, code, (q + 1) * 4 + g / 2, kLanes);
        if (!put)
            continue;
        uint8_t *cell = static_cast<uint8_t *>(a.cache) + w.cell + int64_t(h) * head_stride;
        int off, par;
        if (is_v) {
            code = __byte_perm(c0, c1, (g & 1) ? 0x7632 : 0x5410);
            off = kv4::v_off(D) + kv4::v_swizzle(w.t * (D / 2) + l * 4);
            par = kv4::v_par_off(D, G);
        } else {
            off = w.t * (D / 2) + ((l % 4) * kN + l / 4) * 4;
            par = kv4::k_par_off(D);
        }
        *reinterpret_cast<uint32_t *>(cell + off) = code;
        if (l % (G / 8) == 0)
            *reinterpret_cast<uint32_t *>(cell + par + (w.t * (D / G) + l / (G / 8)) * 4) = pair;
    }
}

// The same lay-out, the other way.
template <int D, int G>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(const Kv4CacheArgs a, int rows_per_block)
{
    constexpr int kCell = kv4::cell_bytes(D, G), kLanes = D / 8, kN = D / 32;
    extern __shared__ RowAt at[];
    const int64_t row0 = int64_t(blockIdx.x) * rows_per_block;
    const int rows = int(min(int64_t(rows_per_block), a.total - row0));
    for (int i = threadIdx.x; i < rows; i += kThreads)
        at[i] = locate(a, row0 + i, kCell);
    __syncthreads();
    const int per_row = 2 * a.Hkv * kLanes, items = rows * per_row;
    const int head_stride = a.page_size / kv4::kCellTokens * kCell;
    for (int it = threadIdx.x; (it & ~31) < items; it += kThreads) {
        const bool in = it < items;
        const int row = in ? it / per_row : 0, p = in ? it - row * per_row : 0;
        const int l = p % kLanes, h2 = p / kLanes;
        const bool is_v = h2 >= a.Hkv;
        const int h = is_v ? h2 - a.Hkv : h2;
        const RowAt w = at[row];
        const bool put = in && w.cell >= 0;
        uint32_t code = 0, pair = 0;
        if (put) {
            const uint8_t *cell =
                static_cast<const uint8_t *>(a.cache) + w.cell + int64_t(h) * head_stride;
            const int off = is_v ? kv4::v_off(D) + kv4::v_swizzle(w.t * (D / 2) + l * 4)
                                 : w.t * (D / 2) + ((l % 4) * kN + l / 4) * 4;
            const int par = is_v ? kv4::v_par_off(D, G) : kv4::k_par_off(D);
            code = *reinterpret_cast<const uint32_t *>(cell + off);
            pair = *reinterpret_cast<const uint32_t *>(cell + par +
                                                       (w.t * (D / G) + l / (G / 8)) * 4);
        }
        // V: logical word l = halves 2 l and 2 l + 1, from two stored words
        const int w0 = (l % 4) * kN + ((l / 4) >> 1);
        const uint32_t c0 = __shfl_sync(0xffffffffu, code, w0, kLanes);
        const uint32_t c1 = __shfl_sync(0xffffffffu, code, w0 + kN / 2, kLanes);
        if (!put)
            continue;
        if (is_v)
            code = __byte_perm(c0, c1, ((l / 4) & 1) ? 0x7632 : 0x5410);
        const __nv_bfloat162 s = __bfloat162bfloat162(
            __ushort_as_bfloat16(static_cast<unsigned short>(pair & 0xffffu)));
        const __nv_bfloat162 m =
            __bfloat162bfloat162(__ushort_as_bfloat16(static_cast<unsigned short>(pair >> 16)));
        // nibbles i and i + 4 as the bf16 pair 128 + code, exact; then one
        // rounding in m + s * code
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = ((code >> (4 * i)) & 0x000f000fu) | 0x43004300u;
            const __nv_bfloat162 c = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&u),
                                             __float2bfloat162_rn(128.f));
            const __nv_bfloat162 y = __hfma2(s, c, m);
            v[i] = *reinterpret_cast<const uint32_t *>(&y);
        }
        const uint4 out = make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                                     __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
        auto *dst = static_cast<__nv_bfloat16 *>(is_v ? a.V : a.K) +
                    (row0 + row) * (is_v ? a.v_stride : a.k_stride) + h * D + l * 8;
        *reinterpret_cast<uint4 *>(dst) = out;
    }
}

template <typename F>
int launch_rows(F kernel, const Kv4CacheArgs &a, cudaStream_t stream)
{
    // one row a block while that fills the SMs (a decode step's few rows),
    // else enough rows for about 8 items a thread
    const int per_row = 2 * a.Hkv * (a.d / 8);
    int rows = (8 * kThreads + per_row - 1) / per_row;
    while (rows > 1 && (a.total + rows - 1) / rows < 2 * 152)
        rows /= 2;
    const int64_t blocks = (a.total + rows - 1) / rows;
    if (blocks > 0x7fffffffLL)
        return FA_ERR_TOO_LARGE;
    kernel<<<unsigned(blocks), kThreads, rows * sizeof(RowAt), stream>>>(a, rows);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
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
