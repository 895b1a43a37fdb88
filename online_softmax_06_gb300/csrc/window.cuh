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

// How the rows of packed sequences are cut into numbered places without asking how many
// each sequence needs: sequence b has the places from F(cu[b], b) to F(cu[b + 1], b + 1),
// F(x, b) = floor(x mul / div) + add b.  With div = rows, mul = add = 1 that is enough for
// its tiles of `rows` rows; with add = 0 for what only long sequences have.
struct WindowCut {
    int mul, div, add;
    __host__ __device__ int64_t at(int64_t x, int64_t b) const
    {
        return (mul == 1 ? int64_t(uint32_t(x) / uint32_t(div)) : x * mul / div) + add * b;
    }
};
// The sequence whose places hold `idx` and idx's number among them; all lanes of a warp
// together (32 probes a round).  idx is below at(total, B).
__device__ __forceinline__ int window_find(const int32_t *cu, int B, const WindowCut &cut,
                                           int64_t idx, int64_t &number)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = B;                        // at(cu[lo], lo) <= idx < at(cu[hi], hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, probe = lo + lane * step;
        const bool below = probe < hi && cut.at(cu[probe], probe) <= idx;
        const unsigned ok = __ballot_sync(0xffffffffu, below);
        const int last = 31 - __clz(int(ok | 1u));
        lo += last * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    number = idx - cut.at(cu[lo], lo);
    return lo;
}

// How the grid's items (tiles of `rows` queries of a kv head) are laid out: B times the
// longest sequence's, or where packed sequences are unlike, as many as their rows have (an
// empty CTA of these kernels holds its SM for a microsecond or more).
struct WindowGrid {
    int per_head;              // items of a kv head, or (not packed) of a sequence's kv head
    int packed;
    WindowCut cut;
};
inline WindowGrid window_grid(const WindowArgs &a, int rows)
{
    const WindowCut cut{1, rows, 1};
    const int64_t each = (int64_t(a.Nq) + rows - 1) / rows, all = cut.at(a.total_q, a.B);
    const bool packed = a.cu_seqlens_q != nullptr && all < each * a.B && all < (int64_t(1) << 31);
    return {int(packed ? all : each), packed, cut};
}
inline int64_t window_items(const WindowArgs &a, const WindowGrid &g)
{
    return int64_t(g.per_head) * a.Hkv * (g.packed ? 1 : a.B);
}
// Item `idx` as (sequence, kv head, tile): tiles of a head one behind the other, the last
// of a sequence first where these are known (early ones see less).  The tile may lie behind
// the sequence's end.
__device__ __forceinline__ bool window_item(const WindowArgs &a, const WindowGrid &g, unsigned idx,
                                            int &b, int &hk, int &tile)
{
    const unsigned bh = idx / unsigned(g.per_head);
    const int t = int(idx - bh * unsigned(g.per_head));
    if (g.packed) {
        hk = int(bh);
        if (hk >= a.Hkv)
            return false;
        int64_t number;
        b = window_find(a.cu_seqlens_q, a.B, g.cut, t, number);
        // (rows behind the last sequence have places, too; nobody's where counts do not fit)
        if (number < 0 || number * g.cut.div >= a.Nq)
            return false;
        tile = int(number);
        return true;
    }
    b = int(bh / unsigned(a.Hkv));
    hk = int(bh - unsigned(b) * unsigned(a.Hkv));
    tile = g.per_head - 1 - t;
    return b < a.B;
}
// The grid's first CTA flags sequences whose counts do not fit: others might find no CTA.
__device__ __forceinline__ void window_check(const WindowArgs &a, const WindowGrid &g, unsigned idx)
{
    if (!g.packed || idx != 0)
        return;
    bool bad = false;
    WindowSeq s;
    for (int b = int(threadIdx.x); b < a.B; b += int(blockDim.x))
        bad |= !window_seq(a, b, s);
    if (bad)
        record_device_error(a.err_word, FA_DEVERR_BAD_SEQLENS);
}

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
