// launch.h -- host-side entry points of the kernels, called by fa_api.cu after
// argument validation.  Each returns an FA_* code.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <mutex>

namespace fa {

// A kernel's dynamic shared-memory limit is raised once per device (the
// attribute belongs to the current device's context): one PerDeviceOnce per
// kernel and call site.
struct PerDeviceOnce {
    static constexpr int kDevices = 64;
    std::once_flag flag[kDevices];
    cudaError_t err[kDevices] = {};
};

inline bool set_max_dynamic_smem(PerDeviceOnce &o, const void *kernel, int bytes)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= PerDeviceOnce::kDevices)
        return false;
    std::call_once(o.flag[dev], [&] {
        o.err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          bytes);
    });
    return o.err[dev] == cudaSuccess;
}

// Row softmax of x [rows, N] into y (y may equal x).
int launch_softmax_rows(const float *x, float *y, int64_t rows, int64_t N, cudaStream_t stream);

// Arguments shared by both attention paths.  Layout rules are those of fa.h.
struct AttnArgs {
    const void *Q, *K, *V;
    void *O;
    float *lse;
    int B, H, N, d;
    int H_row = 0;            // heads per token row in memory (0: H); > H for a
                              // view of heads [h0, h0 + H): Q/K/V/O point at head
                              // h0 of row 0, lse at head h0's first entry
    int64_t total;            // packed token count (B * N when dense)
    float scale;
    int causal;
    const int32_t *cu_seqlens;  // device pointer or nullptr (dense)
    int *err_word;            // device error word
    // split-KV (dense bf16 only): keys per sequence, causal offset (query i
    // sees keys j <= i + kv_off), key ranges per Q-tile pair, fp32 scratch
    int Nk = 0;               // 0: same as N
    int kv_off = 0;
    int splits = 1;
    float *O_accum = nullptr; // [splits, B, N, H, d] (packed: [splits, total, H, d])
    float *lse_accum = nullptr;  // [splits, B, H, N] (packed: [splits, H, total])
    // split-KV on packed batches: key rows per sequence; cu_seqlens holds the
    // query rows, total the query row count
    const int32_t *cu_seqlens_k = nullptr;
    int64_t total_k = 0;
    // failure-detection test (fa_debug_expire_next_wait): nonzero makes the
    // bf16 kernel's MMA warp first wait this many ns on a barrier that nothing
    // arrives at, so the wait runs out and every CTA takes its abort path
    uint32_t expire_wait_ns = 0;
};

int launch_attention_bf16(const AttnArgs &a, cudaStream_t stream);
int launch_attention_f32(const AttnArgs &a, cudaStream_t stream);

// Merges `splits` partial results (O_accum, lse_accum as above) into O (bf16,
// [B, N, H, d]) and lse ([B, H, N]).
int launch_attention_combine(const AttnArgs &a, cudaStream_t stream);

// Number of key splits the library picks for a dense problem (>= 1).
int choose_num_splits(int B, int H, int N, int Nk);

// 3-D TMA map over a [total, H, d] bf16 tensor: box = 64 head-dim elements
// (128 bytes, the 128-byte swizzle span) x 1 head x box_rows rows (128 unless
// given); rows past `total` read as zero.  With H_row > 0 the map covers H
// heads of rows that hold H_row heads (a head-range view; base points at its
// first head).  False if the driver refuses the map.
bool make_tmap_bf16(CUtensorMap *tm, const void *base, int64_t total, int H, int d,
                    int box_rows = 128, int H_row = 0);

// 5-D TMA map (64 values, group, rows, 64-value chunks, heads) over rows of heads * group
// * d bf16 values, `stride` elements apart: box = 64 values (the 128-byte swizzle span) x
// the `group` heads of one of `heads` groups x box_rows rows x all chunks where these fill
// 128 rows each (one copy a tile then, its chunks 16 KB apart), else one chunk.  Rows past
// `rows` read as zero and are not stored.
inline int tmap_heads_chunks(int group, int d, int box_rows)
{
    return group * box_rows == 128 ? d / 64 : 1;
}
bool make_tmap_heads(CUtensorMap *tm, const void *base, int64_t rows, int heads, int group, int d,
                     int64_t stride, int box_rows);

// TMA maps over the FP8 forward's e4m3 tensors: rows of Q' / K' ([total, H, d]
// bytes, box d x 1 x 128, d = 128 so a row is one 128-byte swizzle span) and
// the transposed V' ([rows = B*H*d, n_pad] bytes, box 128 keys x d rows).
bool make_tmap_e4m3_rows(CUtensorMap *tm, const void *base, int64_t total, int H, int d);
bool make_tmap_e4m3_vt(CUtensorMap *tm, const void *base, int64_t rows, int64_t n_pad, int d);
// 4-D TMA map over a dense [B, N, H, d] tensor (bf16, or e4m3 bytes): box = one
// 128-byte row segment (64 bf16 or 128 e4m3) x 1 head x 128 rows x 1 sequence,
// 128-byte swizzle.  Rows past N of a sequence read as zero and are not stored.
bool make_tmap_seq_4d(CUtensorMap *tm, const void *base, bool e4m3, int B, int N, int H, int d);

// FP8 attention forward on the quantised tensors (dense; d = 128).
struct AttnFp8Args {
    const uint8_t *Qf, *Kf, *Vt;
    const float *sq, *sk, *sv;
    void *O;
    float *lse;
    int B, H, N, d, n_pad;
    float scale;
    int causal;
    int *err_word;
    const int32_t *cu_seqlens = nullptr;  // packed: [B + 1] prefix sums; N = longest
    int64_t total = 0;                    // packed: rows of Q, K, V, O
};
int launch_attention_fp8(const AttnFp8Args &a, cudaStream_t stream);

// Backward of the bf16 attention (dense [B, N, H, d] or packed [total, H, d]);
// layouts as in fa.h.
struct AttnBwdArgs {
    const void *Q, *K, *V, *O, *dO;
    const float *lse;          // [B, H, N] (packed: [H, total]), natural log, from the forward
    void *dQ, *dK, *dV;
    float *D;                  // the same layout as lse, scratch: D_i = dO_i . O_i
    int B, H, N, d;            // packed: N = longest sequence (an upper bound)
    float scale;
    int causal;
    int *err_word;
    const int32_t *cu_seqlens = nullptr;  // packed: device [B + 1] prefix sums
    int64_t total = 0;                    // packed: rows of the tensors
    float *dq_acc = nullptr;              // one-pass form: the workspace (see below)
    // failure-detection test (fa_debug_expire_next_wait), one-pass form only:
    // nonzero makes the tensor-core warp wait that long on a barrier that
    // nothing arrives at, so that the timeout path runs
    uint32_t expire_wait_ns = 0;
};
int launch_attention_bwd(const AttnBwdArgs &a, cudaStream_t stream);
// One-pass backward (d = 64 or 128, dense or packed): dQ summed over the key tiles
// by fp32 atomic adds into the workspace a.dq_acc, then converted.
int launch_attention_bwd_atomic(const AttnBwdArgs &a, cudaStream_t stream);
inline int64_t bwd_atomic_n_pad(int N) { return (int64_t(N) + 63) / 64 * 64; }
// Workspace of the one-pass form (d = 64, 128): the fp32 dQ accumulator [B H,
// n_pad, d], then (lse log2 e, D) pairs [B H, n_pad]; packed batches: the
// accumulator [H, total + 64, d], then the pairs [H, B, n_pad].
inline int64_t bwd_atomic_workspace_bytes(int B, int H, int N, int d)
{
    return int64_t(B) * H * bwd_atomic_n_pad(N) * (d + 2) * 4;
}
inline int64_t bwd_atomic_varlen_workspace_bytes(int B, int H, int N, int64_t total, int d)
{
    return int64_t(H) * (total + 64) * d * 4 + int64_t(H) * B * bwd_atomic_n_pad(N) * 8;
}

// Quantisation pass of the FP8 forward (dense [B, N, H, d] bf16 inputs).
struct Fp8QuantArgs {
    const void *Q, *K, *V;
    const float *signs;        // [d], +-1
    uint8_t *Qf, *Kf;          // [B*N, H, d] e4m3 (Q M, K M over scales)
    uint8_t *Vt;               // [B, H, d, n_pad] e4m3, n_pad = 128 * n_tiles
    float *sq, *sk, *vamax;    // [B, H, n_tiles]
    float *sv;                 // [B, H]
    int B, H, N, d;
    int *err_word;             // device error word (bounded waits)
    const int32_t *cu_seqlens = nullptr;  // packed: [B + 1]; Q, K, V, Qf, Kf [total, H, d]
    int64_t total = 0;
};
int launch_fp8_quantize(const Fp8QuantArgs &a, cudaStream_t stream);

// Launches a kernel that waits for those before it (griddepcontrol.wait) ahead of its
// first access to memory: its start overlaps their end (1 x 200 keys, call after call:
// 6.2 us, with plain launches 8.2).  What it reads may be written after it has started,
// so not through the read-only path (__ldg).
template <typename K, typename... Args>
cudaError_t launch_early(K kernel, dim3 grid, int threads, int smem, cudaStream_t stream,
                         const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...), last = cudaGetLastError();
    return e == cudaSuccess ? last : e;
}

// The same in clusters of `size` CTAs.
template <typename K, typename... Args>
cudaError_t launch_early_clusters(K kernel, dim3 grid, int threads, int smem, int size,
                                  cudaStream_t stream, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(size);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...), last = cudaGetLastError();
    return e == cudaSuccess ? last : e;
}

// Writing to and reading from the 4-bit paged cache (layouts as in fa.h).
struct Kv4CacheArgs {
    void *K, *V;               // read by the appending kernel, written by the reading one
    int64_t k_stride, v_stride;
    void *cache;               // the other way round
    int num_pages, page_size;
    const int32_t *page_table;
    int max_pages;
    const int32_t *seqlens;
    const int32_t *cu_seqlens; // or nullptr: N rows each
    int B, N;
    int64_t total;
    int Hkv, d, group;
    int *err_word;
};
int launch_kv4_append(const Kv4CacheArgs &a, cudaStream_t stream);
int launch_kv4_read(const Kv4CacheArgs &a, cudaStream_t stream);

// Attention over the 4-bit paged cache.
struct Kv4AttnArgs {
    const void *Q;
    int64_t q_stride;          // elements between query rows
    const void *cache;
    int num_pages, page_size;
    const int32_t *page_table;
    int max_pages;
    const int32_t *seqlens;
    const int32_t *cu_seqlens_q;  // or nullptr: Nq queries each
    void *O;
    float *lse;
    int B, Nq, Nk;             // Nq, Nk: the most queries and keys of a sequence
    int64_t total_q;
    int H, Hkv, d, group;
    float scale;
    int causal;
    void *workspace;           // not used with whole_items
    int whole_items;           // Nk <= kKv4Short
    int *err_word;
    uint32_t expire_wait_ns;   // failure-detection test (fa_debug_expire_next_wait), or 0
};
constexpr int kKv4Short = 1024;    // keys up to which a crew takes a sequence's head whole
constexpr int kKv4MaxSeqs = 1024;  // each CTA lays the sequences' work out in shared memory
// Query rows (queries x heads of a kv head) that a crew takes at once.  4 fill every second of
// 8 columns, and the others' share of the softmax is left out (64 x 8k keys, 4 rows, 103
// us, as 8 rows 109; 256 x 1k 80 and 88).
inline int kv4_attention_rows(int Nq, int H, int Hkv)
{
    const int64_t rows = int64_t(Nq) * (H / Hkv);
    return rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
}
// A CTA an SM, of as many crews of four warps as the registers allow; each crew takes a
// range of the keys.  More crews of fewer registers take one cell at a time or spill:
// with d = 128 four crews of 8 rows took 111 us on 64 x 8k keys, three 109, and on 256 x
// 1k with groups of 32 96, so 88; three of 16 rows 67.5 on 16 x 4 queries, two 65.7.  With
// d = 64 (accumulators half as large) four instead of three took 49.6 us, not 51.5,
// on 32 x 4k, and three of 16 rows instead of two 43.7, not 47.2, on 16 x 4 queries.
constexpr int kv4_attention_sms = 152;
__host__ __device__ constexpr int kv4_attention_crews(int rows, int d)
{
    return (rows <= 8 ? 3 : 2) + (d == 64);
}
__host__ __device__ constexpr int kv4_attention_ranges(int rows, int d)
{
    return kv4_attention_sms * kv4_attention_crews(rows, d);
}

// The form for many query rows (attn_kv4_many.cu): fp16 copies of Q ([Hkv, total_q,
// H / Hkv, d]) and of the cache ([B, Hkv, 128 n_tiles, d] each), and their factors.
struct Kv4ManyBuffers {
    __half *Q, *K, *V;
    float *q_mul;                  // a row of Q's factor
    // a tile's: K's, and the exponent of V's, floats whose lower halves are 0 and hold each
    // group's first token with a V that is not finite, a byte each
    uint2 *tile;
    float *O_part;                 // with splits > 1: [splits, rows of Q, d], unnormalised
    float2 *ml;                    // and [splits, rows of Q]: (reference, sum)
    int n_tiles;                   // tiles of 128 keys of the longest sequence
    int splits, chunk;             // ranges of `chunk` tiles that its keys are cut into
};
struct Kv4ManyLayout {
    int64_t q, k, v, q_mul, tile, O_part, ml, bytes;
    int n_tiles, splits, chunk;
};
// CTAs of 256 rows of a kv head, as far as the host can tell.
inline int64_t kv4_many_items(int B, int64_t total_q, int H, int Hkv)
{
    const int64_t pairs = (total_q * (H / Hkv) + 255) / 256;
    return (pairs > B ? pairs : B) * Hkv;
}
inline Kv4ManyLayout kv4_many_layout(int B, int64_t total_q, int Nk, int H, int Hkv, int d)
{
    auto up = [](int64_t x) { return (x + 255) & ~int64_t(255); };
    Kv4ManyLayout L;
    L.n_tiles = (Nk + 127) / 128;
    // The CTAs (256 rows of a kv head each) should come to two and a half waves of
    // 152, so that long sequences and the last wave do not leave SMs idle; a range
    // has 16 tiles at least, which pays for its part.
    const int64_t items = kv4_many_items(B, total_q, H, Hkv);
    int64_t splits = items > 0 ? (380 + items - 1) / items : 1;
    splits = splits < L.n_tiles / 16 ? splits : L.n_tiles / 16;
    splits = splits < 1 ? 1 : splits > 8 ? 8 : splits;
    L.chunk = L.n_tiles > 0 ? int((L.n_tiles + splits - 1) / splits) : 1;
    L.splits = L.n_tiles > 0 ? (L.n_tiles + L.chunk - 1) / L.chunk : 1;
    const int64_t tiles = int64_t(B) * Hkv * L.n_tiles;
    L.q = 0;
    L.k = up(total_q * H * d * 2);
    L.v = L.k + up(tiles * 128 * d * 2);
    L.q_mul = L.v + up(tiles * 128 * d * 2);
    L.tile = L.q_mul + up(total_q * H * 4);
    L.O_part = L.tile + up(tiles * 8);
    L.ml = L.O_part + (L.splits > 1 ? up(L.splits * total_q * H * d * 4) : 0);
    L.bytes = L.ml + (L.splits > 1 ? up(L.splits * total_q * H * 8) : 0);
    return L;
}
// Whether a call takes that form.  It writes the whole cache out once, which pays
// where a sequence has 128 rows a kv head or more on average (8 kv heads: 4 x 16k keys
// 128 us against 164, 1 x 16k and 4 x 2k the same), and from 96 on where many heads of
// 128 fill the GPU (64 x 4k keys with 96 rows 421 us against 492, 16 x 1k 37 against
// 51, but 1 x 16k 49 against 43 and 16 x 4k with d = 64 88 against 84; 64 x 4k with 64
// rows 416 against 333); its kernels pay where there is some work (4 x 256 queries on
// 256 keys, 16 heads, 2 GFLOP: 19 us against 34), and some tens of its CTAs where each
// has few tiles.
inline bool kv4_many(int B, int64_t total_q, int Nk, int H, int Hkv, int d)
{
    const int64_t limit = (int64_t(1) << 31) - 512;
    const int64_t rows = total_q > limit ? 0 : total_q * (H / Hkv);   // of a kv head, all sequences
    const int least = d == 128 && int64_t(B) * Hkv >= 128 ? 96 : 128;
    if (rows < int64_t(least) * B || Nk < 128 || B > kKv4MaxSeqs || double(rows) * Hkv > limit ||
        double(B) * Hkv * (Nk + 127.0) > limit ||
        4.0 * rows * Hkv * Nk * d < 1e9)
        return false;
    const Kv4ManyLayout L = kv4_many_layout(B, total_q, Nk, H, Hkv, d);
    return kv4_many_items(B, total_q, H, Hkv) * L.splits >= 24 && L.bytes <= int64_t(8) << 30;
}

// Workspace: that form's copies; otherwise descriptors (32 bytes a range), then for
// two parts a range the (reference, sum) and the fp32 O of each row.
inline int64_t kv4_attention_workspace_bytes(int B, int Nq, int64_t total_q, int Nk, int H, int Hkv,
                                             int d)
{
    if (kv4_many(B, total_q, Nk, H, Hkv, d))
        return kv4_many_layout(B, total_q, Nk, H, Hkv, d).bytes;
    if (Nk <= kKv4Short)
        return 0;
    const int rows = kv4_attention_rows(Nq, H, Hkv);
    return int64_t(kv4_attention_ranges(rows, d)) * (32 + 2 * rows * (8 + 4 * d));
}
int launch_attention_kv4_many(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_attention_kv4(const Kv4AttnArgs &a, cudaStream_t stream);

// Attention with a sliding window and sinks (layouts as in fa.h).
struct WindowArgs {
    const void *Q, *K, *V;
    int64_t q_stride, k_stride, v_stride;  // elements between rows
    void *O;
    float *lse;
    int B, Nq, Nk;             // Nq, Nk: the most queries and keys of a sequence
    int64_t total_q, total_k;
    int H, Hkv, d;
    float scale;
    int window, sinks;
    const int32_t *cu_seqlens_q;  // or nullptr: Nq queries each
    const int32_t *cu_seqlens_k;  // or nullptr: rows b * Nk on
    const int32_t *seqlens_k;     // or nullptr: all of a sequence's rows
    int *err_word;
    uint32_t expire_wait_ns;   // failure-detection test (fa_debug_expire_next_wait), or 0
};
int launch_attention_window(const WindowArgs &a, cudaStream_t stream);
// The form for few query rows (attn_window_few.cu).
int launch_attention_window_few(const WindowArgs &a, cudaStream_t stream);
inline bool window_few(int Nq, int H, int Hkv) { return int64_t(Nq) * (H / Hkv) <= 64; }

// Its gradient: a's queries and keys are the same tokens, O and lse read.
struct WindowBwdArgs {
    WindowArgs a;
    const void *dO;
    void *dQ, *dK, *dV;
    int64_t dq_stride, dk_stride, dv_stride;
    void *workspace;
};
// Its workspace: D, laid out as lse, and the fp32 parts of the tiles with sinks in
// them: their window's, and one for each `piece` tiles of 128 queries behind it.  A piece is
// as long as a window's steps (its CTA takes as long as another one's), and has 8 tiles
// at least, which pays for its part.
// A sequence has 1 + ceil((tiles - near) / piece) parts where its tiles are more than the
// window's `near`, so that it is y > 1 times 128 near long, and at most 2 + floor(y) parts.
// Packed sequences have floor(3 x / (128 near)) places up to row x, so such a one has 3
// floor(y) at least; or each the longest one's parts, whichever is less (with sequences of
// one length the latter).
struct WindowBwdLayout {
    int64_t D, parts, places, bytes;
    int sink_tiles, slots, piece, cut_div;     // cut_div: 128 near, or 0
};
inline WindowBwdLayout window_bwd_layout(int B, int N, int64_t total, int H, int Hkv, int d,
                                         int window, int sinks)
{
    auto up = [](int64_t x) { return (x + 255) & ~int64_t(255); };
    WindowBwdLayout L;
    if (sinks >= N)            // every earlier key is seen
        window = N;
    const int64_t n_qt = (int64_t(N) + 127) / 128, near = (int64_t(window) + 127 + 127) / 128;
    L.piece = int(near < 8 ? 8 : near > n_qt ? n_qt : near);
    // tile 0 has the most queries behind its window
    const int64_t far = n_qt > near ? (n_qt - near + L.piece - 1) / L.piece : 0;
    L.slots = sinks > 0 && far > 0 ? int(far) + 1 : 1;
    L.sink_tiles = L.slots > 1 ? int(((sinks < N ? sinks : N) + 127) / 128) : 0;
    L.cut_div = 0;
    L.places = L.slots > 1 ? int64_t(B) * L.slots : 0;
    if (L.slots > 1 && 3 * total / (128 * near) < L.places) {
        L.cut_div = int(128 * near);
        L.places = 3 * total / (128 * near);
    }
    L.D = 0;
    L.parts = up(total * H * 4);
    L.bytes = L.parts + L.places * Hkv * L.sink_tiles * 2 * 128 * d * 4;
    return L;
}
int launch_attention_window_bwd(const WindowBwdArgs &a, cudaStream_t stream);

// Norm and rotation of the heads of Q (index 0) and K (1), and its gradient.
struct NormRopeArgs {
    const void *x[2], *g[2];   // inputs; backward: gradients of the outputs
    void *y[2];                // outputs; backward: gradients of the inputs
    int64_t xs[2], gs[2], ys[2];  // elements between tokens
    const float *w[2];         // or nullptr: ones
    float *dw[2];              // backward, or nullptr
    const double *freq;        // [rot / 2]
    const int32_t *pos;        // [tokens]
    float *partial;            // backward: workspace
    int64_t tokens;
    int heads[2];
    int d, rot, interleaved;
    float eps;
};
constexpr int kNormRopeCtas = 152 * 2;     // the gradient's CTAs, each with sums of its own
int launch_norm_rope_fwd(const NormRopeArgs &a, cudaStream_t stream);
int launch_norm_rope_bwd(const NormRopeArgs &a, cudaStream_t stream);

}  // namespace fa
