// norm_rope.cu -- the norm of each head of Q and K and the rotation by position
// before the attention, in one pass, and its gradient.
//
// For a head's row x of d values, a weight w and the token's position p:
//     x^ = x r,  r = 1 / sqrt(mean(x^2) + eps),   n = x^ o w,   y = R_p n,
// where R_p turns pair j of the first `rot` values by p f_j ("half" pairs: j and
// j + rot / 2; interleaved: 2 j and 2 j + 1).  With g = R_-p dy, h = g o w:
//     dw = sum over rows of g o x^,   dx = r (h - x^ mean(h o x^)).
// r is formed again from x in the gradient: x has to be read there anyway.
//
// Bound by memory: 4 bytes a value forward, 6 backward, a handful of operations.
// A row is served by d / 8 lanes, eight values each, four of them the partners
// of the other four (half pairs: two 8-byte accesses rot / 2 apart), so that the
// rotation needs no exchange; a lane's four angles hold for all heads of a token,
// so a warp takes a token's heads one after the other, kRows at a time.  Angles:
// f_j / (2 pi) as a 64-bit fraction of a turn, times p modulo 2^64 -- exact where
// an fp32 product would be off by p f_j 2^-24 (0.06 at a position of 10^6) --
// and its upper 32 bits to sincospif.
// Sums are fp32; each output is rounded once.
// 32768 tokens, 32 + 8 heads of 128: forward 109 us, 6.2 TB/s (0.91 of a copy's rate), gradient
// 173 us, 5.8 TB/s (issue slots two thirds used: the arithmetic of a value is what is left beside
// memory); the weights' sums joined in 5 us.  64 tokens: 3.2 us, a launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/fa.h"
#include "launch.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;                  // a CTA's
constexpr int kFwdRows = 4, kBwdRows = 2;  // rows a lane has in flight

struct Params {
    const __nv_bfloat16 *x[2], *g[2];      // of Q and of K: inputs, gradients of the outputs
    __nv_bfloat16 *y[2];                   // outputs, or gradients of the inputs
    int64_t xs[2], gs[2], ys[2];           // elements between tokens
    const float *w[2];
    const double *freq;
    const int32_t *pos;
    float *partial;                        // backward: [CTAs][2][d] sums of dw
    int64_t tokens;
    int heads[2], steps[2];                // steps: passes of a warp over a token's heads
    int unit_steps, token_units;           // passes a unit of work has, units a token has
    int rot;
    float eps;
};

// f / (2 pi) modulo 1 as a 64-bit fraction, in whole numbers: f = m 2^e, times 2^66 /
// (2 pi), shifted.  (Products in fp64, of which an SM has two lanes, took half of the
// kernel's time where a warp has one token.)
__device__ __forceinline__ uint64_t turns(double f)
{
    const uint64_t bits = uint64_t(__double_as_longlong(f));
    const int ex = int(bits >> 52) & 0x7ff;
    const uint64_t m = (bits & 0xfffffffffffffull) | (ex != 0 ? 1ull << 52 : 0);
    constexpr uint64_t c = 0xa2f9836e4e44152aull;    // round(2^66 / (2 pi))
    const uint64_t lo = m * c, hi = __umul64hi(m, c);
    const int s = 2 + 1075 - (ex != 0 ? ex : 1);     // result = (hi : lo) >> s, modulo 2^64
    uint64_t r = 0;
    if (s <= 0)
        r = s > -64 ? lo << -s : 0;
    else if (s < 64)
        r = (hi << (64 - s)) | (lo >> s);
    else if (s < 128)
        r = hi >> (s - 64);
    return (bits >> 63) != 0 ? 0 - r : r;
}

// What a lane does in its row, the same for all rows of a token.
template <int D, bool PAIRS>
struct Lane {
    static constexpr int kLanes = D / 8, kPerWarp = 32 / kLanes;
    int sub, oa, ob;                       // row of the warp; first element of each four
    bool turned;
    uint64_t turn[4];                      // a position's share of a turn, 64-bit fraction
    float c[4], s[4];

    __device__ __forceinline__ explicit Lane(const Params &p)
    {
        const int lane = threadIdx.x & 31, l = lane % kLanes;
        sub = lane / kLanes;
        turned = l < p.rot / 8;
        oa = PAIRS || !turned ? 8 * l : 4 * l;
        ob = PAIRS || !turned ? oa + 4 : p.rot / 2 + oa;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            turn[i] = turned ? turns(p.freq[4 * l + i]) : 0;
    }
    __device__ __forceinline__ void at(int32_t pos)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // the upper half of the product as a signed fraction of half a turn
            const int32_t t = int32_t((uint64_t(int64_t(pos)) * turn[i]) >> 32);
            sincospif(float(t) * 4.656612873077393e-10f, &s[i], &c[i]);  // 2^-31
        }
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *row, uint2 (&v)[2]) const
    {
        if constexpr (PAIRS) {
            const uint4 q = *reinterpret_cast<const uint4 *>(row + oa);
            v[0] = make_uint2(q.x, q.y);
            v[1] = make_uint2(q.z, q.w);
        } else {
            v[0] = *reinterpret_cast<const uint2 *>(row + oa);
            v[1] = *reinterpret_cast<const uint2 *>(row + ob);
        }
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *row, const float (&f)[8]) const
    {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = ptx::pack_bf16x2(f[2 * i], f[2 * i + 1]);
        if constexpr (PAIRS) {
            *reinterpret_cast<uint4 *>(row + oa) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
            *reinterpret_cast<uint2 *>(row + oa) = make_uint2(u[0], u[1]);
            *reinterpret_cast<uint2 *>(row + ob) = make_uint2(u[2], u[3]);
        }
    }
    __device__ __forceinline__ void weights(const float *w, float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = w != nullptr ? w[oa + i] : 1.f;
            f[4 + i] = w != nullptr ? w[ob + i] : 1.f;
        }
    }
    // turns the pairs by the angles, or (back) by their negatives
    template <bool BACK>
    __device__ __forceinline__ void rotate(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float &a = f[PAIRS ? 2 * i : i], &b = f[PAIRS ? 2 * i + 1 : 4 + i];
            const float sn = BACK ? -s[i] : s[i];
            const float t = a * c[i] - b * sn;
            b = a * sn + b * c[i];
            a = t;
        }
    }
    static __device__ __forceinline__ float sum(float v)
    {
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
};

__device__ __forceinline__ void unpack(const uint2 (&v)[2], float (&f)[8])
{
    const uint32_t u[4] = {v[0].x, v[0].y, v[1].x, v[1].y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

template <int D, bool PAIRS>
__global__ void __launch_bounds__(32 * kWarps, 4)
    norm_rope_fwd_kernel(const __grid_constant__ Params p)
{
    using L = Lane<D, PAIRS>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    L lane(p);
    const int64_t unit = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (unit >= p.tokens * p.token_units)
        return;
    const int64_t t = unit / p.token_units;
    const int first = int(unit - t * p.token_units) * p.unit_steps;
    const int last = min(first + p.unit_steps, p.steps[0] + p.steps[1]);
    if (p.rot > 0)
        lane.at(p.pos[t]);
    else
        lane.at(0);
    int kind = -1;
    float w[8];
    for (int step = first; step < last; ++step) {
        const int of = step >= p.steps[0];                     // 0: Q, 1: K
        if (of != kind)
            lane.weights(p.w[of], w);
        kind = of;
        const int h0 = (step - (of ? p.steps[0] : 0)) * kFwdRows * L::kPerWarp + lane.sub;
        const __nv_bfloat16 *x = p.x[of] + t * p.xs[of];
        __nv_bfloat16 *y = p.y[of] + t * p.ys[of];
        uint2 v[kFwdRows][2];
#pragma unroll
        for (int u = 0; u < kFwdRows; ++u) {
            const int h = h0 + u * L::kPerWarp;
            v[u][0] = v[u][1] = make_uint2(0, 0);
            if (h < p.heads[of])
                lane.load(x + h * D, v[u]);
        }
#pragma unroll
        for (int u = 0; u < kFwdRows; ++u) {
            const int h = h0 + u * L::kPerWarp;
            float f[8], ss = 0.f;
            unpack(v[u], f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss = fmaf(f[i], f[i], ss);
            const float r = rsqrtf(L::sum(ss) * (1.f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = f[i] * r * w[i];
            if (lane.turned)
                lane.template rotate<false>(f);
            if (h < p.heads[of])
                lane.store(y + h * D, f);
        }
    }
}

// Rows, positions and weights of the gradient come through shared memory: a thread's own
// copies (nobody else reads them), kStages - 1 passes ahead, so that an SM's loads in
// flight do not depend on its registers.
constexpr int kStages = 4;
template <int D>
struct BwdSmem {
    static constexpr int kSlot = 16 * 32 * kWarps;              // 16 bytes a thread
    static constexpr int kSlots = 2 * kBwdRows;                 // x and g of each row
    static constexpr int kOffPos = kStages * kSlots * kSlot;
    static constexpr int kOffW = kOffPos + kStages * 4 * 32 * kWarps;
    static constexpr int kBytes = kOffW + 2 * D * 4;
    static_assert(kWarps * 2 * D * 4 <= kOffPos, "the warps' sums use the rows' place");
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
                 : "memory");
}

// Where a warp is in its units: pass `step` of token `t`.
struct Place {
    int64_t unit, t;
    int step, last;
    __device__ __forceinline__ void enter(const Params &p, int64_t u)
    {
        unit = u;
        t = p.token_units == 1 ? u : u / p.token_units;
        step = p.token_units == 1 ? 0 : int(u - t * p.token_units) * p.unit_steps;
        last = min(step + p.unit_steps, p.steps[0] + p.steps[1]);
    }
    __device__ __forceinline__ void next(const Params &p, int64_t stride)
    {
        if (++step == last)
            enter(p, unit + stride);
    }
};

template <int D, bool PAIRS>
__global__ void __launch_bounds__(32 * kWarps, 2)
    norm_rope_bwd_kernel(const __grid_constant__ Params p)
{
    using L = Lane<D, PAIRS>;
    using S = BwdSmem<D>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    L lane(p);
    const uint32_t base = ptx::smem_u32(smem);
    const int64_t units = p.tokens * p.token_units, stride = int64_t(gridDim.x) * kWarps;
    float *ws = reinterpret_cast<float *>(smem + S::kOffW);
    for (int i = threadIdx.x; i < 2 * D; i += 32 * kWarps)
        ws[i] = p.w[i / D] != nullptr ? p.w[i / D][i % D] : 1.f;

    auto slot = [&](int stage, int n) { return uint32_t((stage * S::kSlots + n) * S::kSlot); };
    auto fetch = [&](const Place &at, int stage) {
        const int of = at.step >= p.steps[0];                  // 0: Q, 1: K
        const int h0 = (at.step - (of ? p.steps[0] : 0)) * kBwdRows * L::kPerWarp + lane.sub;
        const __nv_bfloat16 *x = p.x[of] + at.t * p.xs[of], *g = p.g[of] + at.t * p.gs[of];
#pragma unroll
        for (int n = 0; n < S::kSlots; ++n) {
            const int h = h0 + (n >> 1) * L::kPerWarp;
            if (h < p.heads[of]) {
                const __nv_bfloat16 *row = (n & 1 ? g : x) + h * D;
                const uint32_t to = base + slot(stage, n);
                if constexpr (PAIRS) {
                    copy_async<16>(to + threadIdx.x * 16, row + lane.oa);
                } else {
                    copy_async<8>(to + threadIdx.x * 8, row + lane.oa);
                    copy_async<8>(to + S::kSlot / 2 + threadIdx.x * 8, row + lane.ob);
                }
            }
        }
        if (p.rot > 0)
            copy_async<4>(base + S::kOffPos + uint32_t(stage * 32 * kWarps + threadIdx.x) * 4,
                          p.pos + at.t);
    };
    auto row = [&](int stage, int n, float (&f)[8]) {
        const uint8_t *from = smem + slot(stage, n);
        uint2 v[2];
        if constexpr (PAIRS) {
            const uint4 q = *reinterpret_cast<const uint4 *>(from + threadIdx.x * 16);
            v[0] = make_uint2(q.x, q.y);
            v[1] = make_uint2(q.z, q.w);
        } else {
            v[0] = *reinterpret_cast<const uint2 *>(from + threadIdx.x * 8);
            v[1] = *reinterpret_cast<const uint2 *>(from + S::kSlot / 2 + threadIdx.x * 8);
        }
        unpack(v, f);
    };

    Place ahead, at;
    ahead.enter(p, int64_t(blockIdx.x) * kWarps + warp);
    at = ahead;
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        if (ahead.unit < units) {
            fetch(ahead, s);
            ahead.next(p, stride);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __syncthreads();                                           // the weights
    float dw[2][8] = {};
    int stage = 0;
    int64_t angles = -1;                                       // the token whose angles these are
    while (at.unit < units) {
        if (ahead.unit < units) {
            fetch(ahead, stage == 0 ? kStages - 1 : stage - 1);
            ahead.next(p, stride);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        if (at.t != angles) {
            angles = at.t;
            lane.at(p.rot > 0 ? *reinterpret_cast<const int32_t *>(
                                    smem + S::kOffPos + (stage * 32 * kWarps + threadIdx.x) * 4)
                              : 0);
        }
        const int of = at.step >= p.steps[0];
        const int h0 = (at.step - (of ? p.steps[0] : 0)) * kBwdRows * L::kPerWarp + lane.sub;
        __nv_bfloat16 *y = p.y[of] + at.t * p.ys[of];
        const float4 wa = *reinterpret_cast<const float4 *>(ws + of * D + lane.oa);
        const float4 wb = *reinterpret_cast<const float4 *>(ws + of * D + lane.ob);
        const float w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int u = 0; u < kBwdRows; ++u) {
            const int h = h0 + u * L::kPerWarp;
            float f[8], q[8], ss = 0.f, hx = 0.f;
            row(stage, 2 * u, f);
            row(stage, 2 * u + 1, q);
            if (lane.turned)
                lane.template rotate<true>(q);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = fmaf(f[i], f[i], ss);
                hx = fmaf(q[i] * w[i], f[i], hx);
            }
            const float r = rsqrtf(L::sum(ss) * (1.f / D) + p.eps);
            const float m = L::sum(hx) * r * (1.f / D);        // mean(h o x^)
            if (h < p.heads[of]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float hat = f[i] * r;
                    if (of == 0)
                        dw[0][i] = fmaf(q[i], hat, dw[0][i]);
                    else
                        dw[1][i] = fmaf(q[i], hat, dw[1][i]);
                    f[i] = r * fmaf(-hat, m, q[i] * w[i]);
                }
                lane.store(y + h * D, f);
            }
        }
        at.next(p, stride);
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    // the CTA's sums: rows of a warp, then warps, in a fixed order
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float *part = reinterpret_cast<float *>(smem);             // [warp][2][D]
#pragma unroll
    for (int of = 0; of < 2; ++of)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v = dw[of][i];
#pragma unroll
            for (int o = 16; o >= L::kLanes; o >>= 1)
                v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane.sub == 0)
                part[(warp * 2 + of) * D + (i < 4 ? lane.oa + i : lane.ob + i - 4)] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += 32 * kWarps) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k)
            v += part[k * 2 * D + i];
        p.partial[int64_t(blockIdx.x) * 2 * D + i] = v;
    }
}

// dw = the sum of the CTAs' partial sums, 32 values a CTA, in a fixed order.
__global__ void __launch_bounds__(1024)
    norm_rope_dw_kernel(const float *partial, int n, int d, float *dwq, float *dwk)
{
    __shared__ float part[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
    float v = 0.f;
#pragma unroll 4
    for (int i = row; i < n; i += 32)
        v += partial[int64_t(i) * 2 * d + col];
    part[row][threadIdx.x & 31] = v;
    __syncthreads();
    if (row == 0) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v += part[i][threadIdx.x];
        float *out = col < d ? dwq : dwk;
        if (out != nullptr)
            out[col < d ? col : col - d] = v;
    }
}

// Units of work: a token's passes together where there are tokens enough to fill
// the GPU with warps (their angles are formed once), fewer where not.
Params make_params(const NormRopeArgs &a, int rows, int64_t *units)
{
    Params p{};
    const int per_step = rows * 32 / (a.d / 8);
    for (int i = 0; i < 2; ++i) {
        p.x[i] = static_cast<const __nv_bfloat16 *>(a.x[i]);
        p.g[i] = static_cast<const __nv_bfloat16 *>(a.g[i]);
        p.y[i] = static_cast<__nv_bfloat16 *>(a.y[i]);
        p.xs[i] = a.xs[i];
        p.gs[i] = a.gs[i];
        p.ys[i] = a.ys[i];
        p.w[i] = a.heads[i] > 0 ? a.w[i] : nullptr;   // (not read without heads)
        p.heads[i] = a.heads[i];
        p.steps[i] = (a.heads[i] + per_step - 1) / per_step;
    }
    p.freq = a.freq;
    p.pos = a.pos;
    p.partial = a.partial;
    p.tokens = a.tokens;
    p.rot = a.rot;
    p.eps = a.eps;
    constexpr int64_t kUnits = 152 * 32;
    const int64_t steps = p.steps[0] + p.steps[1];
    const int64_t want = (a.tokens * steps + kUnits - 1) / kUnits;
    p.unit_steps = int(want < 1 ? 1 : want > steps ? steps : want);
    p.token_units = int((steps + p.unit_steps - 1) / p.unit_steps);
    *units = a.tokens * p.token_units;
    return p;
}

template <int D, bool PAIRS>
int launch_bwd(const Params &p, int64_t blocks, cudaStream_t stream)
{
    auto kern = norm_rope_bwd_kernel<D, PAIRS>;
    static PerDeviceOnce once;
    constexpr int smem = BwdSmem<D>::kBytes;
    if (!set_max_dynamic_smem(once, reinterpret_cast<const void *>(kern), smem))
        return FA_ERR_CUDA;
    return launch_early(kern, dim3(unsigned(blocks)), 32 * kWarps, smem, stream, p) == cudaSuccess
               ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

int launch_norm_rope_fwd(const NormRopeArgs &a, cudaStream_t stream)
{
    int64_t units;
    const Params p = make_params(a, kFwdRows, &units);
    const int64_t blocks = (units + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL)
        return FA_ERR_TOO_LARGE;
    const dim3 grid{unsigned(blocks)};
    cudaError_t e;
    if (a.d == 64)
        e = a.interleaved ? launch_early(norm_rope_fwd_kernel<64, true>, grid, 32 * kWarps, 0, stream, p)
                          : launch_early(norm_rope_fwd_kernel<64, false>, grid, 32 * kWarps, 0, stream, p);
    else
        e = a.interleaved ? launch_early(norm_rope_fwd_kernel<128, true>, grid, 32 * kWarps, 0, stream, p)
                          : launch_early(norm_rope_fwd_kernel<128, false>, grid, 32 * kWarps, 0, stream, p);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int launch_norm_rope_bwd(const NormRopeArgs &a, cudaStream_t stream)
{
    int64_t units;
    const Params p = make_params(a, kBwdRows, &units);
    int64_t blocks = (units + kWarps - 1) / kWarps;
    blocks = blocks > kNormRopeCtas ? kNormRopeCtas : blocks;
    cudaError_t e = cudaSuccess;
    if (blocks > 0) {
        const int rc = a.d == 64 ? a.interleaved ? launch_bwd<64, true>(p, blocks, stream)
                                                 : launch_bwd<64, false>(p, blocks, stream)
                       : a.interleaved ? launch_bwd<128, true>(p, blocks, stream)
                                       : launch_bwd<128, false>(p, blocks, stream);
        if (rc != FA_OK)
            return rc;
    }
    if (a.dw[0] != nullptr || a.dw[1] != nullptr)
        e = launch_early(norm_rope_dw_kernel, dim3(unsigned(2 * a.d / 32)), 1024, 0, stream,
                         static_cast<const float *>(a.partial), int(blocks), a.d, a.dw[0], a.dw[1]);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa
