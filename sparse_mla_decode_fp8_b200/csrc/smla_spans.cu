// smla_spans.cu -- spans of 64 consecutive tokens (a quarter of a page) as the unit of a cheap
// selection: their keys, and the best of them by given scores.
//
// span_keys: key of span j = the mean of its tokens' dequantised latents (those below the
// sequence length), summed in fp32 in a fixed order and rounded once to bf16 (2^-8 of the
// value at most: the scores made from the keys only rank spans).
// select_spans: the nsel best spans of a request, by score, ties to the lower index.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "smla_device.cuh"
#include "smla_host.cuh"

namespace smla {
namespace spans {

constexpr int kSpan = SMLA_SPAN_TOKENS;
constexpr int kPageSpans = kPageTokens / kSpan;
static_assert(kSpan == 64 && kPageTokens % kSpan == 0, "a span is a quarter of a page");

// ------------------------------------------------------------------ span keys
// One block of 256 threads per span, whose 64 rows are 36,864 contiguous bytes.  Thread
// (g, c) = (t / 36, t % 36), g < 7, sums 16-byte chunk c of the rows g, g + 7, ...: the
// block's loads are contiguous.  The 7 partial sums of a dim are added in shared memory.
// HBM-bound: 584 bytes read per token, 1024 written per span.
constexpr int kKeyThreads = 256;
constexpr int kKeyGroups = 7;
static_assert(kKeyGroups * kRowChunks <= kKeyThreads, "one thread per chunk of 7 rows");

__global__ void __launch_bounds__(kKeyThreads) span_keys_kernel(
    const uint8_t *__restrict__ cache, const int32_t *__restrict__ block_table, const int32_t *__restrict__ seq_lens,
    const int32_t *__restrict__ req, const int32_t *__restrict__ span, int B, int max_blocks, long long num_pages,
    uint16_t *__restrict__ keys, uint32_t *err) {
    __shared__ float part[kKeyGroups][kDim];
    const int t = threadIdx.x;
    const int b = __ldg(req + blockIdx.x), j = __ldg(span + blockIdx.x);
    int page = -1, n = 0;
    if (b >= 0 && b < B && j >= 0 && j / kPageSpans < max_blocks) {
        const long long left = static_cast<long long>(__ldg(seq_lens + b)) - static_cast<long long>(j) * kSpan;
        n = static_cast<int>(max(0ll, min(static_cast<long long>(kSpan), left)));
        if (n > 0) page = __ldg(block_table + static_cast<size_t>(b) * max_blocks + j / kPageSpans);
    }
    if (page < 0 || page >= num_pages) {  // block-uniform
        if (t == 0 && err) atomicOr(err, SMLA_FLAG_BAD_PAGE);
        return;
    }
    const int code = page * kPageTokens + (j % kPageSpans) * kSpan;
    if (t < kKeyGroups * kRowChunks) {
        const int g = t / kRowChunks, c = t - g * kRowChunks;
        const uint8_t *row = token_row(cache, code) + 16 * c;
        float acc[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[k] = 0.0f;
        if (c < kNopeChunks) {
            const uint8_t *sc = token_scales(cache, code) + (c >> 2);
#pragma unroll 5
            for (int r = g; r < n; r += kKeyGroups) {
                const uint4 v = ld_stream_v4(row + r * kRowBytes);
                const float s = ue8m0_value(ld_stream_u8(sc + r * kScaleRowBytes));
                float x[16];
                e4m3x4_values(v.x, s, x);
                e4m3x4_values(v.y, s, x + 4);
                e4m3x4_values(v.z, s, x + 8);
                e4m3x4_values(v.w, s, x + 12);
#pragma unroll
                for (int k = 0; k < 16; ++k) acc[k] += x[k];
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) part[g][16 * c + k] = acc[k];
        } else {
#pragma unroll 5
            for (int r = g; r < n; r += kKeyGroups) {
                const uint4 v = ld_stream_v4(row + r * kRowBytes);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[2 * k] += __uint_as_float(w[k] << 16);
                    acc[2 * k + 1] += __uint_as_float(w[k] & 0xFFFF0000u);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) part[g][kNope + 8 * (c - kNopeChunks) + k] = acc[k];
        }
    }
    __syncthreads();
    float m[2] = {0.0f, 0.0f};  // dims 2t, 2t + 1
#pragma unroll
    for (int g = 0; g < kKeyGroups; ++g) {
        m[0] += part[g][2 * t];
        m[1] += part[g][2 * t + 1];
    }
    const float count = static_cast<float>(n);
    reinterpret_cast<uint32_t *>(keys + (static_cast<size_t>(page) * kPageSpans + j % kPageSpans) * kDim)[t] =
        pack_bf16x2(m[0] / count, m[1] / count);
}

// ------------------------------------------------------------------ selection
// One block per request.  Scores become 32-bit keys in the order of the selection (kept spans
// above all, NaN as -inf, -0 as +0; 0 = no span here).  The nsel-th largest key is built bit by
// bit from the top, counting the keys above each candidate, and the search stops early once a
// candidate separates exactly nsel keys.  Then one pass in index order writes the spans above
// the key and the first of those equal to it.  Latency-bound: a few microseconds of
// barriers, over 4 bytes read per span.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (isnan(x)) x = -INFINITY;
    if (x == 0.0f) x = 0.0f;
    const uint32_t u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

struct SelectParams {
    const float *scores;
    const int32_t *seq_lens;
    int32_t *spans;
    int32_t *topk_idx;
    int width;  // scores per request
    int nsel, keep_first, keep_last;
};

__device__ __forceinline__ uint32_t span_key(const SelectParams &p, const float *row, int j, int count) {
    if (j >= count) return 0u;
    if (j < p.keep_first || j >= count - p.keep_last) return 0xFFFFFFFFu;
    return order_key(__ldg(row + j));
}

// Sum over the block (every thread gets it); `slot` alternates between calls.
template <int kThreads>
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t *slots, int &slot) {
    v = __reduce_add_sync(0xffffffffu, v);
    uint32_t *s = slots + (slot % 3) * 32;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    ++slot;  // three rows: a row is written again only after another barrier
    const uint32_t w = (threadIdx.x & 31) < kThreads / 32 ? s[threadIdx.x & 31] : 0u;
    return __reduce_add_sync(0xffffffffu, w);
}

// kHeld keys per thread in registers when width <= kThreads * kHeld; kHeld = 0 reads the scores
// again on every pass (from L2).
template <int kThreads, int kHeld>
__global__ void __launch_bounds__(kThreads) select_spans_kernel(const SelectParams p) {
    __shared__ uint32_t slots[3 * 32];
    __shared__ uint32_t warp_base[2][kThreads / 32];
    int slot = 0;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const size_t b = blockIdx.x;
    const int len = __ldg(p.seq_lens + b);
    const int count = len <= 0 ? 0 : min(p.width, static_cast<int>((static_cast<long long>(len) + kSpan - 1) / kSpan));
    const float *row = p.scores + b * p.width;
    const uint32_t need = static_cast<uint32_t>(min(p.nsel, count));
    // thread t holds the spans kHeld t ..: index order over the threads
    uint32_t held[kHeld ? kHeld : 1];
    if (kHeld) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) held[k] = span_key(p, row, kHeld * t + k, count);
    }
    auto count_ge = [&](uint32_t bound) {
        uint32_t c = 0;
        if (kHeld) {
#pragma unroll
            for (int k = 0; k < kHeld; ++k) c += held[k] >= bound ? 1u : 0u;
        } else {
            for (int j = t; j < count; j += kThreads) c += span_key(p, row, j, count) >= bound ? 1u : 0u;
        }
        return block_sum<kThreads>(c, slots, slot);
    };
    // the largest key with at least `need` keys at or above it
    uint32_t key = 0, above = static_cast<uint32_t>(count);  // keys >= key
    if (need < static_cast<uint32_t>(count)) {
        for (int bit = 31; bit >= 0 && above != need; --bit) {
            const uint32_t c = count_ge(key | (1u << bit));
            if (c >= need) {
                key |= 1u << bit;
                above = c;
            }
        }
    }
    if (key == 0) key = 1;  // everything that is a span
    // `above` keys are >= key; if that is more than needed, those equal to key are taken from the
    // lowest index on (key + 1 cannot wrap: at most nsel spans are kept, so no tie is among them)
    const bool ties = above != need;
    const uint32_t quota = ties ? need - count_ge(key + 1u) : 0u;  // of the equal ones
    int32_t *out = p.spans + b * p.nsel;
    uint32_t done_gt = 0, done_eq = 0;
    const int chunk = kThreads * (kHeld ? kHeld : 1);
    for (int base = 0; base < count; base += chunk) {
        const int j0 = base + (kHeld ? kHeld : 1) * t;
        uint32_t k0[kHeld ? kHeld : 1];
        uint32_t gt = 0, eq = 0;
#pragma unroll
        for (int k = 0; k < (kHeld ? kHeld : 1); ++k) {
            k0[k] = kHeld ? held[k] : span_key(p, row, j0 + k, count);
            const bool taken = ties ? k0[k] > key : k0[k] >= key;
            gt += taken ? 1u : 0u;
            eq += (ties && k0[k] == key) ? 1u : 0u;
        }
        // exclusive prefix of (gt, eq) over the block
        uint32_t pg = gt, pe = eq;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = __shfl_up_sync(0xffffffffu, pg, o), e = __shfl_up_sync(0xffffffffu, pe, o);
            if (lane >= o) pg += a, pe += e;
        }
        __syncthreads();  // warp_base is free again
        if (lane == 31) warp_base[0][warp] = pg, warp_base[1][warp] = pe;
        __syncthreads();
        uint32_t bg = done_gt, be = done_eq, tg = 0, te = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            const uint32_t a = warp_base[0][w], e = warp_base[1][w];
            if (w < warp) bg += a, be += e;
            tg += a, te += e;
        }
        uint32_t g = bg + pg - gt, e = be + pe - eq;  // taken and equal before this thread's spans
#pragma unroll
        for (int k = 0; k < (kHeld ? kHeld : 1); ++k) {
            const bool equal = ties && k0[k] == key;
            const bool taken = ties ? k0[k] > key : k0[k] >= key;
            if (taken || (equal && e < quota)) out[g + min(e, quota)] = j0 + k;
            g += taken ? 1u : 0u;
            e += equal ? 1u : 0u;
        }
        done_gt += tg, done_eq += te;
    }
    for (int k = static_cast<int>(need) + t; k < p.nsel; k += kThreads) out[k] = -1;
    if (p.topk_idx == nullptr) return;
    __syncthreads();  // the spans are written (global writes of this block, read back below)
    int32_t *idx = p.topk_idx + b * p.nsel * kSpan;
    for (int i = t; i < p.nsel * kSpan; i += kThreads) {
        const int j = i / kSpan < static_cast<int>(need) ? out[i / kSpan] : -1;
        const int token = j * kSpan + (i % kSpan);
        idx[i] = (j >= 0 && token < len) ? token : -1;
    }
}

}  // namespace spans
}  // namespace smla

extern "C" {

int smla_span_keys(const uint8_t *kv_cache, const int32_t *block_table, const int32_t *seq_lens, const int32_t *req,
                   const int32_t *span, int n, int B, int max_blocks, int num_pages, void *keys, uint32_t *err,
                   void *stream) {
    using namespace smla::spans;
    using smla::host::aligned;
    if (n < 0 || B < 1 || max_blocks < 1 || num_pages < 1 || num_pages >= (1 << 23)) return SMLA_ERR_INVALID;
    if (n == 0) return SMLA_OK;
    if (!kv_cache || !block_table || !seq_lens || !req || !span || !keys) return SMLA_ERR_INVALID;
    if (!aligned(kv_cache, 16) || !aligned(keys, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(req, 4) || !aligned(span, 4) || !aligned(err, 4))
        return SMLA_ERR_INVALID;
    int dev = 0, sms = 0;
    const int rc = smla::host::current_device(dev, sms);
    if (rc != SMLA_OK) return rc;
    (void)cudaGetLastError();
    span_keys_kernel<<<static_cast<unsigned>(n), kKeyThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        kv_cache, block_table, seq_lens, req, span, B, max_blocks, num_pages, static_cast<uint16_t *>(keys), err);
    return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

int smla_select_spans(const float *scores, int width, const int32_t *seq_lens, int nsel, int keep_first,
                      int keep_last, int32_t *spans, int32_t *topk_idx, int B, void *stream) {
    using namespace smla::spans;
    using smla::host::aligned;
    if (B < 1 || width < 1 || width > SMLA_MAX_SPANS || nsel < 1 || nsel > SMLA_MAX_NSEL || keep_first < 0 ||
        keep_last < 0 || keep_first > nsel || keep_last > nsel - keep_first)
        return SMLA_ERR_INVALID;
    if (!scores || !seq_lens || !spans) return SMLA_ERR_INVALID;
    if (!aligned(scores, 4) || !aligned(seq_lens, 4) || !aligned(spans, 4) || !aligned(topk_idx, 4))
        return SMLA_ERR_INVALID;
    int dev = 0, sms = 0;
    const int rc = smla::host::current_device(dev, sms);
    if (rc != SMLA_OK) return rc;
    (void)cudaGetLastError();
    const SelectParams p{scores, seq_lens, spans, topk_idx, width, nsel, keep_first, keep_last};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned blocks = static_cast<unsigned>(B);
    if (width <= 256 * 8)
        select_spans_kernel<256, 8><<<blocks, 256, 0, st>>>(p);
    else if (width <= 1024 * 8)
        select_spans_kernel<1024, 8><<<blocks, 1024, 0, st>>>(p);
    else
        select_spans_kernel<1024, 0><<<blocks, 1024, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

}  // extern "C"
