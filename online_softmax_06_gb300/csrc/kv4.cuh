// kv4.cuh -- the 4-bit paged key/value cache: where things stand in a cell.
//
// A cache is uint8 [pages, Hkv, page_size / 16 * cell]; a cell holds 16 tokens
// of one head (include/fa.h states the format of a value):
//   K codes [16][d/2] bytes, V codes [16][d/2], K parameters [16][d/group] of
//   (scale, min) bf16 pairs, V parameters likewise.
// The orders inside a row are those in which the attention kernel's lanes feed
// their matrix instructions (attn_kv4.cu), so that a lane reads its share of a
// row as one piece:
//   K row: 32-bit word w = 4 j + c (values 8 w .. 8 w + 7, lowest nibble first)
//          stands at word c * (d / 32) + j: lane c of a quad owns d / 32
//          consecutive words, and its j-th word lies in values 32 j .. 32 j + 31.
//   V row: 16-bit half h = 8 q + g (values 4 h .. 4 h + 3) stands at half
//          g * (d / 32) + q, and the 32-byte sector s of the cell's V codes
//          stands at sector (s & ~3) | ((s + (s >> 2)) & 3): lanes that read
//          tokens 0, 2, 4, 6 (or 1, 3, 5, 7) at once hit different banks.
#pragma once

#include <cstdint>

namespace fa {
namespace kv4 {

constexpr int kCellTokens = 16;

__host__ __device__ constexpr int cell_bytes(int d, int group)
{
    return kCellTokens * (d + 8 * (d / group));
}
__host__ __device__ constexpr int v_off(int d) { return kCellTokens * (d / 2); }
__host__ __device__ constexpr int k_par_off(int d) { return kCellTokens * d; }
__host__ __device__ constexpr int v_par_off(int d, int group)
{
    return kCellTokens * (d + 4 * (d / group));
}

// Byte of the V codes at which byte `a` (token * d / 2 + byte of the row) stands.
__device__ __forceinline__ int v_swizzle(int a)
{
    const int s = a >> 5;
    return (((s & ~3) | ((s + (s >> 2)) & 3)) << 5) | (a & 31);
}

// The two bf16 numbers of a word.
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

}  // namespace kv4
}  // namespace fa
