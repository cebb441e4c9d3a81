// smla_reader.cu -- cached tokens read back: the rows of n (request, position) pairs as dense
// 512-d latents, bf16 or fp32.  The inverse of the cache writer: nope value = e4m3 * 2^(s-127)
// of its 64-dim group, rope value as stored.
//
// The product is exact in fp32 (4 significant bits, exponents -136..135, above the range an
// infinity), and so is the fp32 output.  The bf16 output is that product rounded once to
// nearest even: it is exact too unless s < 10 (subnormal bf16) or the value leaves the range.
//
// HBM-bound: 584 bytes read and 1024 (bf16) or 2048 (fp32) written per token; 120,000 tokens as fp32
// (317 MB) take 54 us, 89 % of the measured copy bandwidth.  A warp takes
// kReadTokens tokens at a time, so that the three dependent loads (request and position, block
// table, row) of several tokens are in flight together.  A lane holds 8 (bf16) or 4 (fp32)
// consecutive dims of each pass, so that every store of a warp is 512 contiguous bytes.
#include <cuda_runtime.h>

#include <cstdint>

#include "smla_device.cuh"
#include "smla_host.cuh"

namespace smla {
namespace reader {

constexpr int kReadWarps = 8;
constexpr int kReadTokens = 4;

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// A token's raw bytes in this lane: dims 256k + 8 lane.. (bf16 output, k = 0, 1; the last 8
// lanes of k = 1 hold 8 rope values) or 128k + 4 lane.. (fp32 output, k = 0..3; the last 16
// lanes of k = 3 hold 4 rope values).
template <bool kBf16>
struct Raw;
template <>
struct Raw<true> {
    uint2 nope0, scales;
    uint4 part1;
    __device__ __forceinline__ void load(const uint8_t *cache, int code, int lane) {
        const uint8_t *row = token_row(cache, code);
        nope0 = ld_stream_v2(row + 8 * lane);
        if (lane < 24) {
            const uint2 v = ld_stream_v2(row + 256 + 8 * lane);
            part1 = make_uint4(v.x, v.y, 0u, 0u);
        } else {
            part1 = ld_stream_v4(row + kNope + 16 * (lane - 24));
        }
        scales = ld_stream_v2(token_scales(cache, code));
    }
    __device__ __forceinline__ void store(void *out, size_t token, int lane, bool valid) const {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + token * kDim) + lane;
        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
        if (valid) {
            float x[8];
            const float s0 = ue8m0_value(scale_byte(scales, lane >> 3));
            e4m3x4_values(nope0.x, s0, x);
            e4m3x4_values(nope0.y, s0, x + 4);
            a = pack8(x);
            if (lane < 24) {
                const float s1 = ue8m0_value(scale_byte(scales, 4 + (lane >> 3)));
                e4m3x4_values(part1.x, s1, x);
                e4m3x4_values(part1.y, s1, x + 4);
                b = pack8(x);
            } else {
                b = part1;
            }
        }
        __stcs(dst, a);
        __stcs(dst + 32, b);
    }
};
template <>
struct Raw<false> {
    uint32_t nope[3];
    uint2 part3, scales;
    __device__ __forceinline__ void load(const uint8_t *cache, int code, int lane) {
        const uint8_t *row = token_row(cache, code);
#pragma unroll
        for (int k = 0; k < 3; ++k) nope[k] = ld_stream_u32(row + 128 * k + 4 * lane);
        if (lane < 16)
            part3 = make_uint2(ld_stream_u32(row + 384 + 4 * lane), 0u);
        else
            part3 = ld_stream_v2(row + kNope + 8 * (lane - 16));
        scales = ld_stream_v2(token_scales(cache, code));
    }
    __device__ __forceinline__ void store(void *out, size_t token, int lane, bool valid) const {
        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) + token * kDim) + lane;
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (valid) e4m3x4_values(nope[k], ue8m0_value(scale_byte(scales, 2 * k + (lane >> 4))), x);
            __stcs(dst + 32 * k, make_float4(x[0], x[1], x[2], x[3]));
        }
        if (valid) {
            if (lane < 16) {
                e4m3x4_values(part3.x, ue8m0_value(scale_byte(scales, 6)), x);
            } else {
                x[0] = __uint_as_float(part3.x << 16);
                x[1] = __uint_as_float(part3.x & 0xFFFF0000u);
                x[2] = __uint_as_float(part3.y << 16);
                x[3] = __uint_as_float(part3.y & 0xFFFF0000u);
            }
        }
        __stcs(dst + 96, make_float4(x[0], x[1], x[2], x[3]));
    }
};

template <bool kBf16>
__global__ void __launch_bounds__(32 * kReadWarps) read_kv_kernel(
    const uint8_t *__restrict__ cache, const int32_t *__restrict__ req, const int32_t *__restrict__ pos, int n,
    const int32_t *__restrict__ block_table, int B, int max_blocks, long long num_pages, void *__restrict__ out,
    uint32_t *err) {
    const int lane = threadIdx.x & 31;
    const long long first = (static_cast<long long>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5)) * kReadTokens;
    if (first >= n) return;  // warp-uniform
    const int count = static_cast<int>(min(static_cast<long long>(kReadTokens), n - first));
    int code = -1;
    if (lane < count) {
        const int b = __ldg(req + first + lane), p = __ldg(pos + first + lane);
        int page = -1;
        if (b >= 0 && b < B && p >= 0 && (p >> 8) < max_blocks)
            page = __ldg(block_table + static_cast<size_t>(b) * max_blocks + (p >> 8));
        if (page >= 0 && page < num_pages)
            code = page * kPageTokens + (p & (kPageTokens - 1));
        else if (err)
            atomicOr(err, SMLA_FLAG_BAD_PAGE);
    }
    Raw<kBf16> raw[kReadTokens];
    int codes[kReadTokens];
#pragma unroll
    for (int u = 0; u < kReadTokens; ++u) {
        codes[u] = __shfl_sync(0xffffffffu, code, u);
        if (codes[u] >= 0) raw[u].load(cache, codes[u], lane);
    }
#pragma unroll
    for (int u = 0; u < kReadTokens; ++u)
        if (u < count) raw[u].store(out, static_cast<size_t>(first) + u, lane, codes[u] >= 0);
}

}  // namespace reader
}  // namespace smla

extern "C" int smla_read_kv(const uint8_t *kv_cache, const int32_t *req, const int32_t *pos, int n,
                            const int32_t *block_table, int B, int max_blocks, int num_pages, void *out,
                            int out_bf16, uint32_t *err, void *stream) {
    using namespace smla::reader;
    using smla::host::aligned;
    if (n < 0 || B < 1 || max_blocks < 1 || num_pages < 1 || num_pages >= (1 << 23)) return SMLA_ERR_INVALID;
    if (n == 0) return SMLA_OK;
    if (!kv_cache || !req || !pos || !block_table || !out) return SMLA_ERR_INVALID;
    if (!aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(req, 4) || !aligned(pos, 4) ||
        !aligned(block_table, 4) || !aligned(err, 4))
        return SMLA_ERR_INVALID;
    int dev = 0, sms = 0;
    const int rc = smla::host::current_device(dev, sms);
    if (rc != SMLA_OK) return rc;
    (void)cudaGetLastError();
    const long long per_block = kReadWarps * kReadTokens;
    const unsigned blocks = static_cast<unsigned>((n + per_block - 1) / per_block);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (out_bf16)
        read_kv_kernel<true><<<blocks, 32 * kReadWarps, 0, st>>>(kv_cache, req, pos, n, block_table, B, max_blocks,
                                                                 num_pages, out, err);
    else
        read_kv_kernel<false><<<blocks, 32 * kReadWarps, 0, st>>>(kv_cache, req, pos, n, block_table, B, max_blocks,
                                                                  num_pages, out, err);
    return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}
