// pmqa_latent.cuh -- the latent row and its layout as an operand in shared memory,
// shared by the sparse MLA decode and the attention to all latent tokens: 512 value
// columns in groups of 8 rows with the 128-byte swizzle, 64 rotary columns with
// the 64-byte swizzle.
#pragma once

#include <cstdint>

namespace pmqa {
namespace mla {

constexpr int kDim = 576;    // latent row: 512 value columns + 64 rotary columns
constexpr int kVDim = 512;   // value columns
constexpr int kChunks = kDim / 16;
constexpr uint32_t kVGroup = 4u * 1024u;          // 8 rows x 4 value blocks of 128 bytes
constexpr uint32_t kVStage = 16u * kVGroup;       // 128 rows of value columns (64 KB)
constexpr uint32_t kRGroup = 512u;                // 8 rows x 64 rotary bytes
constexpr uint32_t kRStage = 16u * kRGroup;       // 128 rows of rotary columns (8 KB)

// Byte offset of value chunk c (0..31) of row t: groups of 8 rows 4096 bytes
// apart, four 1024-byte blocks of 8 rows x 128 bytes, 128-byte swizzle.
__host__ __device__ constexpr uint32_t v_offset(int t, int c)
{
    return (uint32_t)(t >> 3) * kVGroup + (uint32_t)(c >> 3) * 1024u + (uint32_t)(t & 7) * 128u +
           ((uint32_t)((c & 7) ^ (t & 7)) << 4);
}

// Byte offset of rotary chunk c (0..3) of row t: groups of 8 rows x 64 bytes,
// 64-byte swizzle (chunk c of row r at c ^ (r >> 1)).
__host__ __device__ constexpr uint32_t r_offset(int t, int c)
{
    return (uint32_t)(t >> 3) * kRGroup + (uint32_t)(t & 7) * 64u +
           ((uint32_t)((c ^ ((t & 7) >> 1)) & 3) << 4);
}

}  // namespace mla
}  // namespace pmqa
