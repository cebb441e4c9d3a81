// smla_tile.cuh -- the 128-token MMA tile shared by the kernels that multiply it with the 64
// heads of a query: its descriptors, the score MMAs and the cross-lane reductions.
//
// Shared-memory layout (128-byte swizzle): the tile is 8 K-blocks of [128 tokens x 64 dims]
// bf16, 16 KB each; Q is 8 K-blocks of [64 heads x 64 dims], 8 KB each.
#pragma once

#include <cstdint>

#include "sm100_ptx.cuh"

namespace smla {

constexpr int kTile = 128;                     // topk slots per MMA tile (the M of S^T)
constexpr uint32_t kIdescQK = idesc_bf16(128, 64, false, false);
constexpr uint32_t kIdescPV = idesc_bf16(128, 64, true, true);

// Reduces N (16 or 32) per-thread values across the 32 lanes of a warp, value i with
// value i of every other lane.  Each round halves the live entries: a lane keeps the
// half selected by its lane bit and sends the other half to its partner.  With N = 32
// lane j ends with entry j; with N = 16 lanes 2j and 2j+1 end with entry j.
template <bool kMax, int N>
__device__ __forceinline__ float warp_transpose_reduce(float (&v)[N], int lane) {
    static_assert(N == 16 || N == 32, "16 or 32 entries");
#pragma unroll
    for (int w = N / 2, off = 16; w >= 1; w >>= 1, off >>= 1) {
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float send = upper ? v[i] : v[i + w];
            const float keep = upper ? v[i + w] : v[i];
            const float got = __shfl_xor_sync(0xffffffffu, send, off);
            v[i] = kMax ? fmaxf(keep, got) : keep + got;
        }
    }
    if constexpr (N == 16) {
        const float got = __shfl_xor_sync(0xffffffffu, v[0], 1);
        return kMax ? fmaxf(v[0], got) : v[0] + got;
    }
    return v[0];
}

// 16 consecutive floats of shared memory (16-byte aligned) into registers.
__device__ __forceinline__ void load16(const float *src, float (&v)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 t = reinterpret_cast<const float4 *>(src)[j];
        v[4 * j] = t.x;
        v[4 * j + 1] = t.y;
        v[4 * j + 2] = t.z;
        v[4 * j + 3] = t.w;
    }
}

// Descriptor words (128-byte swizzle, see sw128_desc): the high word holds SBO = 1024
// (8 rows of 128 bytes), the version and the swizzle mode; the low word holds the
// address (16-byte units) and LBO.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
    return ((saddr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}

// S^T += K.Q^T over dims chunk cp: 2 K-blocks x 4 steps of K = 16 (the K rows are
// 128 bytes per K-block, K-blocks 16 KB apart; Q K-blocks 8 KB apart).
__device__ __forceinline__ void issue_qk_chunk(uint32_t d, uint32_t a_lo, uint32_t b_lo, bool first) {
    if (first)
        mma_bf16_ss(d, desc_from(a_lo, kDescHi), desc_from(b_lo, kDescHi), kIdescQK, 0u);
    else
        mma_bf16_ss_acc(d, desc_from(a_lo, kDescHi), desc_from(b_lo, kDescHi), kIdescQK);
#pragma unroll
    for (int k = 1; k < 8; ++k) {
        const uint32_t ao = (k >> 2) * ((kTile * 128) >> 4) + (k & 3) * 2;
        const uint32_t bo = (k >> 2) * (8192 >> 4) + (k & 3) * 2;
        mma_bf16_ss_acc(d, desc_from(a_lo + ao, kDescHi), desc_from(b_lo + bo, kDescHi), kIdescQK);
    }
}

}  // namespace smla
