// window.cuh -- what the kernels of the window attention share: a sequence's
// rows, and the keys that a block of its queries sees.
//
// Query i of the n of a sequence of L keys sits at position p = i + L - n and
// sees key j iff j <= p and (j > p - window or j < sinks).  The keys that the
// queries i0 .. i1 - 1 see are two ranges, [0, sinks) and [lo, hi); they are
// taken one behind the other, the sinks filled up to a multiple of `pad`, as
// places v = 0, 1, ...: place v < sp is key v, another one key lo + v - sp.
// Where the ranges meet (lo <= sp) they are one, [0, hi), and sp = 0.  A query
// at p sees the places
//     v <= vhi and (v >= vlo or v < sinks),
//     vhi = p - lo + sp,  vlo = max(sp, vhi - window + 1).
#pragma once

#include <cstdint>

#include "../../include/fa.h"
#include "fa_error.cuh"
#include "launch.h"

namespace fa {

struct WindowSeq {
    int64_t q0, k0;            // first rows of Q and K
    int n, L;                  // queries and keys
};

// False where the counts contradict the tensors.
__device__ __forceinline__ bool window_seq(const WindowArgs &a, int b, WindowSeq &s)
{
    if (a.cu_seqlens_q != nullptr) {
        const int64_t r0 = a.cu_seqlens_q[b], r1 = a.cu_seqlens_q[b + 1];
        if (r0 < 0 || r1 < r0 || r1 > a.total_q || r1 - r0 > a.Nq)
            return false;
        s.q0 = r0;
        s.n = int(r1 - r0);
    } else {
        s.q0 = int64_t(b) * a.Nq;
        s.n = a.Nq;
    }
    int64_t room = a.Nk;
    s.k0 = int64_t(b) * a.Nk;
    if (a.cu_seqlens_k != nullptr) {
        const int64_t r0 = a.cu_seqlens_k[b], r1 = a.cu_seqlens_k[b + 1];
        if (r0 < 0 || r1 < r0 || r1 > a.total_k)
            return false;
        s.k0 = r0;
        room = r1 - r0;
    }
    const int64_t L = a.seqlens_k != nullptr ? int64_t(a.seqlens_k[b]) : room;
    if (L < 0 || L > room || L > a.Nk)
        return false;
    s.L = int(L);
    return true;
}

struct WindowKeys {
    int lo, sp, places;        // places = sp + hi - lo (0: the queries see no key)
};

// Of queries i0 .. i1 - 1 (i1 > i0).
__device__ __forceinline__ WindowKeys window_keys(int window, int sinks, int i0, int i1, int off,
                                                  int pad)
{
    WindowKeys w;
    const int hi = i1 + off;   // <= L
    const int64_t first = int64_t(i0) + off - window + 1;
    w.lo = first > 0 ? int(first) : 0;
    const int s = sinks < w.lo ? sinks : w.lo;
    w.sp = (s + pad - 1) / pad * pad;
    if (w.sp >= w.lo)
        w.lo = w.sp = 0;
    w.places = hi > 0 ? w.sp + hi - w.lo : 0;
    return w;
}

// Tile `idx` of all tiles of `rows` queries of packed sequences, as (sequence, tile from the
// sequence's end); false behind the last.  A sequence whose counts do not fit has one (whose
// CTA flags it).  All lanes of a warp together.
__device__ __forceinline__ bool window_tile(const WindowArgs &a, int rows, int idx, int &b,
                                            int &tile)
{
    const int lane = threadIdx.x & 31;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        int n = 0;
        if (b0 + lane < a.B) {
            const int64_t len = int64_t(a.cu_seqlens_q[b0 + lane + 1]) - a.cu_seqlens_q[b0 + lane];
            n = len < 0 || len > a.Nq ? 1 : int((len + rows - 1) / rows);
        }
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            sum += lane >= o ? x : 0;
        }
        const int all = __shfl_sync(0xffffffffu, sum, 31);
        if (idx < all) {
            const unsigned behind = __ballot_sync(0xffffffffu, idx < sum);
            const int k = __ffs(int(behind)) - 1;
            b = b0 + k;
            tile = __shfl_sync(0xffffffffu, sum, k) - 1 - idx;
            return true;
        }
        idx -= all;
    }
    return false;
}

// How the grid's items (tiles of `rows` queries of a kv head) are laid out: B times the
// longest sequence's, or where packed sequences are unlike, as many as their rows have (an
// empty CTA of these kernels holds its SM for a microsecond or more).
struct WindowGrid {
    int per_head;              // items of a kv head, or (not packed) of a sequence's kv head
    int packed;
};
inline WindowGrid window_grid(const WindowArgs &a, int rows)
{
    const int64_t each = (int64_t(a.Nq) + rows - 1) / rows;
    const int64_t all = a.total_q / rows + a.B;
    if (a.cu_seqlens_q != nullptr && all < each * a.B && all < (int64_t(1) << 31))
        return {int(all), 1};
    return {int(each), 0};
}
inline int64_t window_items(const WindowArgs &a, const WindowGrid &g)
{
    return int64_t(g.per_head) * a.Hkv * (g.packed ? 1 : a.B);
}
// Item `idx` as (sequence, kv head, tile): the last tiles of a sequence first (early ones
// see less), tiles of a head one behind the other.
__device__ __forceinline__ bool window_item(const WindowArgs &a, const WindowGrid &g, int rows,
                                            unsigned idx, int &b, int &hk, int &tile)
{
    const unsigned bh = idx / unsigned(g.per_head);
    const int t = int(idx - bh * unsigned(g.per_head));
    if (g.packed) {
        hk = int(bh);
        return hk < a.Hkv && window_tile(a, rows, t, b, tile);
    }
    b = int(bh / unsigned(a.Hkv));
    hk = int(bh - unsigned(b) * unsigned(a.Hkv));
    tile = g.per_head - 1 - t;
    return b < a.B;
}

// CTAs that run at once, one an SM: the CTA this far behind in the grid is about the next
// on this one's SM, and its first tiles, which nobody reads before it, are brought into L2
// meanwhile (from DRAM its first product waited some 3 us for them).
constexpr int kWindowSms = 152;

// The lowest `n` bits, n clamped to 0 .. 32.
__device__ __forceinline__ uint32_t low_bits(int n)
{
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Which of the 32 places from v on a query sees.
__device__ __forceinline__ uint32_t window_bits(int v, int vlo, int vhi, int sinks)
{
    return low_bits(vhi - v + 1) & (~low_bits(vlo - v) | low_bits(sinks - v));
}

}  // namespace fa
