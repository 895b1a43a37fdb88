// attn_window_few.cu -- attention with a sliding window and sinks for few queries: a
// decode step, drafted tokens.
//
// What it computes is attn_window.cu's; what bounds it is reading K and V of the
// window once, so it is built to keep copies in flight, and the products (a hundredth
// of the time at the tensor cores' rate) are mma.sync's, whose 16 rows fit the few
// query rows (queries x heads of a kv head) where a tcgen05 tile would be empty but
// for them:
//   * a warp is on its own: blocks of 16 keys, K and V, in a ring of three, filled
//     by 16-byte cp.async.  No warp waits for another before the end; an SM's eight
//     warps (two CTAs) have 192 KB in flight or in use;
//   * its state is its own too: running maximum and sum of each row, O in fp32
//     registers.  P is rounded to bf16 (2^-9 relative; the largest of a row, 1 by the
//     exact running maximum, not at all);
//   * an item (sequence, kv head, 16 or 32 query rows) is taken by a cluster of 1 to
//     16 CTAs, a range of the places (window.cuh) each; the warps' parts meet in
//     shared memory, and each CTA sends its sums to the one that joins that share of
//     the values, through distributed shared memory: one launch, no workspace.
// Keys that no query of an item sees (behind the sequence, between sinks and window)
// are not read; their rows are zeros.
// 64 sequences of 300 to 16000 keys, window 4096, 32 heads on 8, d = 128 (941 MB of K and V):
// 139 us, 6.7 TB/s, the rate of a copy; 16 x 4 queries, 32 heads on 4, window 1024 (33 MB):
// 15.7 us; one query, 8 kv heads, window 8192 (34 MB): 12.1 us; window 256: 4.7 us, a launch,
// a cluster's start and two trips to memory.
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

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kKeys = 16;                     // keys of a block
constexpr int kStages = 3;
constexpr float kLn2 = 0.69314718055994531f;

template <int D, int MT>
struct Cfg {
    static constexpr int kRows = 16 * MT;
    static constexpr int kRowBytes = D * 2;
    static constexpr int kHalf = kKeys * kRowBytes;              // K or V of a block
    static constexpr int kRing = kWarps * kStages * 2 * kHalf;
    // behind the keys, the ring holds the warps' parts of O, then the CTAs' parts of
    // this CTA's share
    static constexpr int kPart = kRows * D * 4;
    static_assert((kWarps + 1) * kPart <= kRing, "shared memory");
    static constexpr int kOffQ = kRing;
    static constexpr int kOffMl = kOffQ + kRows * kRowBytes;     // the warps' rows' (m, l), weights
    static constexpr int kOffCl = kOffMl + kWarps * kRows * 8;   // the CTAs' (m, l)
    static constexpr int kSmem = kOffCl + 16 * kRows * 8;
};

struct Params {
    WindowArgs a;
    int G, row_blocks, split;
    float scale_log2;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// c += a b: a 16 x 16 and b 16 x 8 bf16 fragments
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int D, int MT>
__global__ void __launch_bounds__(kThreads) attn_window_few_kernel(const __grid_constant__ Params p)
{
    using C = Cfg<D, MT>;
    extern __shared__ __align__(128) uint8_t smem[];
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const WindowArgs &a = p.a;
    const int part = int(blockIdx.x % unsigned(p.split));
    const int item = int(blockIdx.x / unsigned(p.split));
    const int rb = item % p.row_blocks, bh = item / p.row_blocks;
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    // what follows is the same for all CTAs of a cluster
    WindowSeq sq;
    if (!window_seq(a, b, sq)) {
        if (threadIdx.x == 0 && rb == 0 && hk == 0 && part == 0)
            record_device_error(a.err_word, FA_DEVERR_BAD_SEQLENS);
        return;
    }
    const int rows = sq.n * p.G, r0 = rb * C::kRows;
    if (r0 >= rows)
        return;
    const int off = sq.L - sq.n;
    const int i0 = r0 / p.G, i1 = min(r0 + C::kRows - 1, rows - 1) / p.G + 1;
    const WindowKeys w = window_keys(a.window, a.sinks, i0, i1, off, kKeys);
    const int blocks = (w.places + kKeys - 1) / kKeys;
    const int first = int(int64_t(blocks) * part / p.split);
    const int last = int(int64_t(blocks) * (part + 1) / p.split);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = ptx::smem_u32(smem) + uint32_t(warp) * kStages * 2 * C::kHalf;

    // ---- copies: a lane takes one 16-byte unit of every kRowsPerCopy-th row -------------
    constexpr int kUnits = D / 8, kRowsPerCopy = 32 / kUnits, kCopies = kKeys / kRowsPerCopy;
    const int cu = lane % kUnits, cr = lane / kUnits;
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(a.K) + sq.k0 * a.k_stride +
                              int64_t(hk) * D + cu * 8;
    const __nv_bfloat16 *vp = static_cast<const __nv_bfloat16 *>(a.V) + sq.k0 * a.v_stride +
                              int64_t(hk) * D + cu * 8;
    const int64_t k_step = int64_t(kRowsPerCopy) * a.k_stride;
    const int64_t v_step = int64_t(kRowsPerCopy) * a.v_stride;
    auto copy = [&](int blk, int stage) {
        const uint32_t dst = ring + uint32_t(stage) * 2 * C::kHalf + cr * C::kRowBytes;
        const int v0 = blk * kKeys;
        if (v0 >= w.sp && v0 + kKeys <= w.places) {
            // a block of the window: consecutive rows, all there
            const int64_t key = w.lo + v0 - w.sp + cr;
            const __nv_bfloat16 *ks = kp + key * a.k_stride, *vs = vp + key * a.v_stride;
#pragma unroll
            for (int c = 0; c < kCopies; ++c) {
                const int row = cr + c * kRowsPerCopy;
                const uint32_t to = dst + c * kRowsPerCopy * C::kRowBytes + ((cu ^ (row & 7)) << 4);
                cp16(to, ks, true);
                cp16(to + C::kHalf, vs, true);
                ks += k_step;
                vs += v_step;
            }
            return;
        }
#pragma unroll 1
        for (int c = 0; c < kCopies; ++c) {
            const int row = cr + c * kRowsPerCopy, v = v0 + row;
            const bool ok = v < w.places && (v >= w.sp || v < a.sinks);
            const int64_t key = !ok ? 0 : v < w.sp ? v : w.lo + v - w.sp;
            const uint32_t to = dst + c * kRowsPerCopy * C::kRowBytes + ((cu ^ (row & 7)) << 4);
            cp16(to, kp + key * a.k_stride, ok);
            cp16(to + C::kHalf, vp + key * a.v_stride, ok);
        }
    };
    // the queries' rows, with the first block (rows behind the last: zeros)
    const uint32_t qs = ptx::smem_u32(smem) + C::kOffQ;
    for (int e = threadIdx.x; e < C::kRows * kUnits; e += kThreads) {
        const int r = e / kUnits, u = e % kUnits, i = (r0 + r) / p.G, g = (r0 + r) % p.G;
        const bool ok = r0 + r < rows;
        cp16(qs + r * C::kRowBytes + ((u ^ (r & 7)) << 4),
             static_cast<const __nv_bfloat16 *>(a.Q) + (ok ? (sq.q0 + i) * a.q_stride : 0) +
                 int64_t(hk * p.G + g) * D + u * 8,
             ok);
    }
    int next = first + warp;                       // this warp's blocks: every kWarps-th
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s, next += kWarps) {
        if (next < last)
            copy(next, s);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    // ---- queries as fragments (of 32 rows they are read again for each block) ----------------
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncthreads();
    uint32_t qa[D / 16][4];
    auto load_q = [&](int t, int k, uint32_t (&f)[4]) {
        const int r = 16 * t + (lane & 15), u = 2 * k + (lane >> 4);
        ldsm(f, qs + r * C::kRowBytes + ((u ^ (r & 7)) << 4));
    };
    if constexpr (MT == 1)
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            load_q(0, k, qa[k]);
    int vhi[MT][2], vlo[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = r0 + 16 * t + 8 * half + (lane >> 2);
            vhi[t][half] = r < rows ? r / p.G + off - w.lo + w.sp : -1;
            const int64_t vl = int64_t(vhi[t][half]) - a.window + 1;
            vlo[t][half] = vl > w.sp ? int(vl) : w.sp;
        }
    // places that all queries of the item see: [all0, all1]
    const int64_t al = int64_t(i1 - 1 + off - w.lo + w.sp) - a.window + 1;
    const int all0 = al > w.sp ? int(al) : w.sp, all1 = i0 + off - w.lo + w.sp;

    float m[MT][2], l[MT][2], o[MT][D / 8][4];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        m[t][0] = m[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.f;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[t][n][e] = 0.f;
    }
    const float sl = p.scale_log2;

    int stage = 0;
    for (int blk = first + warp; blk < last; blk += kWarps, next += kWarps) {
        {
            const int into = stage == 0 ? kStages - 1 : stage - 1;
            if (next < last)
                copy(next, into);
            asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();
        }
        const uint32_t ks = ring + uint32_t(stage) * 2 * C::kHalf, vs = ks + C::kHalf;
        // ---- S = Q K^T, 16 keys -----------------------------------------------------
        float s[MT][2][4] = {};
        const int mr = (lane & 7) + ((lane >> 4) << 3), mu = (lane >> 3) & 1;   // K's matrices
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t f[4];
            ldsm(f, ks + mr * C::kRowBytes + (((2 * k + mu) ^ (mr & 7)) << 4));
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if constexpr (MT > 1)
                    load_q(t, k, qa[k]);
                mma16(s[t][0], qa[k], f[0], f[1]);
                mma16(s[t][1], qa[k], f[2], f[3]);
            }
        }
        // ---- mask, running maximum, P -------------------------------------------------
        const int v0 = blk * kKeys;
        if (v0 < all0 || v0 + kKeys - 1 > all1) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int v = v0 + 8 * n + 2 * (lane & 3) + (e & 1);
                        if (v > vhi[t][e >> 1] || (v < vlo[t][e >> 1] && v >= a.sinks))
                            s[t][n][e] = -INFINITY;
                    }
        }
        uint32_t pa[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            float corr[2];
            bool grew = false;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float mx = fmaxf(fmaxf(s[t][0][2 * half], s[t][0][2 * half + 1]),
                                 fmaxf(s[t][1][2 * half], s[t][1][2 * half + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * sl;
                const float mn = fmaxf(m[t][half], mx);
                const float mu2 = mn == -INFINITY ? 0.f : mn;
                corr[half] = ptx::ex2(m[t][half] - mu2);
                grew |= mn > m[t][half];
                m[t][half] = mn;
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float pv = ptx::ex2(fmaf(s[t][n][2 * half + e], sl, -mu2));
                        s[t][n][2 * half + e] = pv;
                        sum += pv;
                    }
                l[t][half] = (mn == -INFINITY ? 0.f : l[t][half] * corr[half]) + sum;
            }
            pa[t][0] = ptx::pack_bf16x2(s[t][0][0], s[t][0][1]);
            pa[t][1] = ptx::pack_bf16x2(s[t][0][2], s[t][0][3]);
            pa[t][2] = ptx::pack_bf16x2(s[t][1][0], s[t][1][1]);
            pa[t][3] = ptx::pack_bf16x2(s[t][1][2], s[t][1][3]);
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[t][n][0] *= corr[0];
                    o[t][n][1] *= corr[0];
                    o[t][n][2] *= corr[1];
                    o[t][n][3] *= corr[1];
                }
            }
        }
        // ---- O += P V ---------------------------------------------------------------
        const int vr = lane & 15, vu = lane >> 4;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            uint32_t f[4];
            ldsm_t(f, vs + vr * C::kRowBytes + (((2 * n + vu) ^ (vr & 7)) << 4));
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                mma16(o[t][2 * n], pa[t], f[0], f[1]);
                mma16(o[t][2 * n + 1], pa[t], f[2], f[3]);
            }
        }
        __syncwarp();                              // the stage may be filled again
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- the warps' parts, through shared memory ----------------------------------------
    __syncthreads();                               // all are done with the ring
    float *parts = reinterpret_cast<float *>(smem);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::kOffMl);   // [warp][row]
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float sum = l[t][half];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const int r = 16 * t + 8 * half + (lane >> 2);
            if ((lane & 3) == 0)
                ml[warp * C::kRows + r] = make_float2(m[t][half], sum);
            float *dst = parts + (warp * C::kRows + r) * D + 2 * (lane & 3);
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2 *>(dst + 8 * n) =
                    make_float2(o[t][n][2 * half], o[t][n][2 * half + 1]);
        }
    // all CTAs of the cluster are done with their rings
    if (p.split > 1)
        ptx::cluster_sync();
    else
        __syncthreads();

    // (m, l) of several parts joined: the largest m, the sum of l at it; a part's factor
    auto weight = [](float mv, float M) { return mv == -INFINITY ? 0.f : ptx::ex2(mv - M); };
    const uint32_t share = ptx::smem_u32(smem) + kWarps * C::kPart;
    const uint32_t cl = ptx::smem_u32(smem) + C::kOffCl;
    constexpr int kQuads = C::kRows * D / 4;       // four values of a row each
    const int per = kQuads / p.split;              // of a CTA's share
    // a thread's quads are of the same columns of rows kThreads / (D / 4) apart
    for (int e = threadIdx.x; e < kQuads; e += kThreads) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        float2 s[kWarps];
        float4 x[kWarps];
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            s[k] = ml[k * C::kRows + r];
            x[k] = *reinterpret_cast<const float4 *>(parts + (k * C::kRows + r) * D + c);
        }
        const float M = fmaxf(fmaxf(s[0].x, s[1].x), fmaxf(s[2].x, s[3].x));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const float f = weight(s[k].x, M);
            v.x = fmaf(f, x[k].x, v.x);
            v.y = fmaf(f, x[k].y, v.y);
            v.z = fmaf(f, x[k].z, v.z);
            v.w = fmaf(f, x[k].w, v.w);
            sum = fmaf(f, s[k].y, sum);
        }
        const int owner = e / per;
        ptx::st_cluster4(ptx::cluster_addr(share + uint32_t(part * per + e % per) * 16, uint32_t(owner)), v);
        // the row's (m, l) to every CTA: one column's thread each
        const int to = c / 4;
        if (to < p.split)
            ptx::st_cluster2(ptx::cluster_addr(cl + uint32_t(part * C::kRows + r) * 8, uint32_t(to)),
                        make_float2(M, sum));
    }
    if (p.split > 1)
        ptx::cluster_sync();
    else
        __syncthreads();

    // ---- the CTAs' parts of this one's share ------------------------------------------------
    const float4 *mine = reinterpret_cast<const float4 *>(smem + kWarps * C::kPart);
    const float2 *cml = reinterpret_cast<const float2 *>(smem + C::kOffCl);
    for (int q = threadIdx.x; q < per; q += kThreads) {
        const int e = part * per + q, r = e / (D / 4), c = e % (D / 4) * 4;
        if (r0 + r >= rows)
            break;
        float M = -INFINITY;
#pragma unroll 4
        for (int k = 0; k < p.split; ++k)
            M = fmaxf(M, cml[k * C::kRows + r].x);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 4
        for (int k = 0; k < p.split; ++k) {
            const float2 s = cml[k * C::kRows + r];
            const float4 x = mine[k * per + q];
            const float f = weight(s.x, M);
            v.x = fmaf(f, x.x, v.x);
            v.y = fmaf(f, x.y, v.y);
            v.z = fmaf(f, x.z, v.z);
            v.w = fmaf(f, x.w, v.w);
            sum = fmaf(f, s.y, sum);
        }
        const int i = (r0 + r) / p.G, h = hk * p.G + (r0 + r) % p.G;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.O) +
                                   ((sq.q0 + i) * a.H + h) * D + c) =
            make_uint2(ptx::pack_bf16x2(v.x * inv, v.y * inv),
                       ptx::pack_bf16x2(v.z * inv, v.w * inv));
        if (c == 0)
            a.lse[a.cu_seqlens_q != nullptr ? int64_t(h) * a.total_q + sq.q0 + i
                                            : (int64_t(b) * a.H + h) * a.Nq + i] =
                sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
    }
}

template <int D, int MT>
int launch_d(const Params &p, int64_t blocks, cudaStream_t stream)
{
    auto kern = attn_window_few_kernel<D, MT>;
    static PerDeviceOnce once, once_c;
    constexpr int smem = Cfg<D, MT>::kSmem;
    if (!set_max_dynamic_smem(once, reinterpret_cast<const void *>(kern), smem))
        return FA_ERR_CUDA;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= PerDeviceOnce::kDevices)
        return FA_ERR_CUDA;
    std::call_once(once_c.flag[dev], [&] {
        once_c.err[dev] = cudaFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (once_c.err[dev] != cudaSuccess)
        return FA_ERR_CUDA;
    const cudaError_t e =
        p.split > 1
            ? launch_early_clusters(kern, dim3(unsigned(blocks)), kThreads, smem, p.split, stream, p)
            : launch_early(kern, dim3(unsigned(blocks)), kThreads, smem, stream, p);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

int launch_attention_window_few(const WindowArgs &a, cudaStream_t stream)
{
    Params p;
    p.a = a;
    p.G = a.H / a.Hkv;
    p.scale_log2 = float(double(a.scale) * 1.4426950408889634);
    const int64_t rows = int64_t(a.Nq) * p.G;
    const int mt = rows <= 16 ? 1 : 2;
    p.row_blocks = int((rows + 16 * mt - 1) / (16 * mt));
    const int64_t items = int64_t(a.B) * a.Hkv * p.row_blocks;
    // CTAs of an item: a power of two.  Up to one for each of the 304 places there are,
    // as long as each has 128 keys at least (4 x 16 sequences of 1043 keys: 15.7 us with
    // four CTAs, 16.8 with two, 24.7 with eight, which are more than the places); one step
    // more where each then has 1024 (8 items of 8196 keys: 12.1 us with 16, 14.1 with 8;
    // 512 items of 4100: 137 with one, 143 with two, 177 with eight).
    int64_t keys = int64_t(a.window) + a.Nq - 1 + a.sinks;
    keys = keys < a.Nk ? keys : a.Nk;
    p.split = 1;
    while (p.split < 16 && ((items * p.split * 2 <= 304 && keys >= int64_t(p.split) * 2 * 128) ||
                            (items * p.split < 304 && keys >= int64_t(p.split) * 2 * 1024)))
        p.split *= 2;
    const int64_t blocks = items * p.split;
    if (blocks > 0x7fffffffLL)
        return FA_ERR_TOO_LARGE;
    if (a.d == 64)
        return mt == 1 ? launch_d<64, 1>(p, blocks, stream) : launch_d<64, 2>(p, blocks, stream);
    return mt == 1 ? launch_d<128, 1>(p, blocks, stream) : launch_d<128, 2>(p, blocks, stream);
}

}  // namespace fa
