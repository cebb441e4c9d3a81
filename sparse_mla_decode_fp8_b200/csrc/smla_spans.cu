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
#include <mutex>

#include "smla_device.cuh"
#include "smla_host.cuh"

namespace smla {
namespace spans {

constexpr int kSpan = SMLA_SPAN_TOKENS;
constexpr int kPageSpans = kPageTokens / kSpan;
static_assert(kSpan == 64 && kPageTokens % kSpan == 0, "a span is a quarter of a page");

// ------------------------------------------------------------------ span keys
// A block takes a span at a time, whose 64 rows are 36,864 contiguous bytes: one bulk copy into shared
// memory, and one for the scale rows; four blocks on an SM copy and sum in turn.  Seven warps sum the
// nope chunks, thread (g, c) of 8 x 28 chunk c of the rows g, g + 8, ..; two warps the rope chunks, thread
// (g, c) of 8 x 8.  The 8 partial sums of a dim are added in shared memory.  The lookups of a span
// (request and span, length and page) are made ahead.
// 584 bytes are read per token and 1,024 written per span: 438.5 MB for 11,426 spans take 93 to 95 us, 71 % of
// the measured copy bandwidth.  Instructions to issue bound it next to HBM (ncu: issue slots 70 % busy, DRAM 57 % of its
// peak, the load-store pipe 44 %): 144 us when warps mixed nope and rope chunks, 133 us with rows by loads (whose pipe
// takes a cycle for 32 bytes).  A block has one stage, so nothing of it is in flight while it sums; the other three
// blocks of the SM cover that in part.
constexpr int kKeyGroups = 8;
constexpr int kKeyNopeThreads = kKeyGroups * kNopeChunks;  // 224
constexpr int kKeyRopeChunks = kRowChunks - kNopeChunks;
constexpr int kKeyThreads = kKeyGroups * kRowChunks;       // 288
constexpr int kKeyStage = kSpan * (kRowBytes + kScaleRowBytes);  // rows, then scale rows
constexpr int kKeySmem = kKeyStage + kKeyGroups * kDim * 4;
constexpr int kKeyBlocks = 4;       // per SM
constexpr unsigned long long kKeyTimeoutNs = 1000000000ull;
static_assert(kKeyNopeThreads % 32 == 0 && kKeyThreads % 32 == 0, "whole warps");
static_assert(kKeyStage % 16 == 0 && kKeyBlocks * (kKeySmem + 1024) <= 228 * 1024, "the blocks of an SM");

struct KeyParams {
    const uint8_t *cache;
    const int32_t *block_table, *seq_lens, *req, *span;
    uint16_t *keys;
    uint32_t *err;
    long long num_pages;
    int n, B, max_blocks;
};

// acc += e4m3 * scale (each product is exact, so an fma rounds once as the sum does).
__device__ __forceinline__ void add_e4m3x4(uint32_t four, float scale, float *acc) {
    float x[4];
    e4m3x4_values(four, x);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = fmaf(x[k], scale, acc[k]);
}

// A listed span: its first token's code, or -1, and how many tokens count.
struct KeyItem {
    int code, count;
};
__device__ __forceinline__ KeyItem key_item(const KeyParams &p, int b, int j) {
    KeyItem k{-1, 0};
    if (b < 0 || b >= p.B || j < 0 || j / kPageSpans >= p.max_blocks) return k;
    const long long left = static_cast<long long>(__ldg(p.seq_lens + b)) - static_cast<long long>(j) * kSpan;
    const int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks + j / kPageSpans);
    if (left <= 0 || page < 0 || page >= p.num_pages) return k;
    k.count = static_cast<int>(min(static_cast<long long>(kSpan), left));
    k.code = page * kPageTokens + (j % kPageSpans) * kSpan;
    return k;
}

__global__ void __launch_bounds__(kKeyThreads, kKeyBlocks) span_keys_kernel(const __grid_constant__ KeyParams p) {
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ uint64_t bar;
    float(*part)[kDim] = reinterpret_cast<float(*)[kDim]>(stage + kKeyStage);
    const int t = threadIdx.x;
    const bool nope = t < kKeyNopeThreads;
    const int g = nope ? t / kNopeChunks : (t - kKeyNopeThreads) / kKeyRopeChunks;
    const int c = nope ? t % kNopeChunks : kNopeChunks + (t - kKeyNopeThreads) % kKeyRopeChunks;
    // unsigned: an index two steps past the last of up to 2^31 - 1 spans is still a number
    const uint32_t step = gridDim.x, n = static_cast<uint32_t>(p.n);
    if (t == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
    }
    __syncthreads();
    // the copies of an item: one arrival on the barrier, also for an item without a span
    const auto copy = [&](const KeyItem &k) {
        const uint32_t rows = k.count * kRowBytes, scales = (k.count * kScaleRowBytes + 15) & ~15;
        mbar_arrive_expect_tx(&bar, rows + scales);
        if (k.count > 0) {
            bulk_load(smem_addr(stage), token_row(p.cache, k.code), rows, &bar);
            bulk_load(smem_addr(stage) + kSpan * kRowBytes, token_scales(p.cache, k.code), scales, &bar);
        }
    };
    const auto listed = [&](uint32_t i, int &b, int &j) {
        b = i < n ? __ldg(p.req + i) : -1;
        j = i < n ? __ldg(p.span + i) : 0;
    };
    int b, j;
    listed(blockIdx.x, b, j);
    KeyItem now = key_item(p, b, j);
    listed(blockIdx.x + step, b, j);
    uint32_t parity = 0;
    for (uint32_t i = blockIdx.x; i < n; i += step, parity ^= 1) {
        if (t == 0) copy(now);  // every thread is done with the span before (the barriers below)
        const KeyItem next = key_item(p, b, j);
        listed(i + 2 * step, b, j);
        const bool landed = mbar_wait(&bar, parity, kKeyTimeoutNs);
        const int count = landed ? now.count : 0;
        float acc[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[k] = 0.0f;
        if (nope) {
#pragma unroll
            for (int k = 0; k < kSpan / kKeyGroups; ++k) {
                const int r = g + kKeyGroups * k;
                if (r < count) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(stage + r * kRowBytes + 16 * c);
                    const float f = ue8m0_value(stage[kSpan * kRowBytes + r * kScaleRowBytes + (c >> 2)]);
                    add_e4m3x4(v.x, f, acc);
                    add_e4m3x4(v.y, f, acc + 4);
                    add_e4m3x4(v.z, f, acc + 8);
                    add_e4m3x4(v.w, f, acc + 12);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                reinterpret_cast<float4 *>(&part[g][16 * c])[k] =
                    make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
        } else {
#pragma unroll
            for (int k = 0; k < kSpan / kKeyGroups; ++k) {
                const int r = g + kKeyGroups * k;
                if (r < count) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(stage + r * kRowBytes + 16 * c);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[2 * e] += __uint_as_float(w[e] << 16);
                        acc[2 * e + 1] += __uint_as_float(w[e] & 0xFFFF0000u);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
                reinterpret_cast<float4 *>(&part[g][kNope + 8 * (c - kNopeChunks)])[k] =
                    make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
        }
        if (__syncthreads_or(!landed)) {  // the block gives up: NaN keys for the rest of its list
            if (t == 0 && p.err) atomicOr(p.err, SMLA_FLAG_TIMEOUT);
            for (; i < n; i += step) {
                const KeyItem k = key_item(p, __ldg(p.req + i), __ldg(p.span + i));
                for (int d = t; k.count > 0 && d < kDim; d += kKeyThreads)
                    p.keys[static_cast<size_t>(k.code / kSpan) * kDim + d] = 0x7FC0u;
            }
            (void)mbar_wait(&bar, parity, kKeyTimeoutNs);  // the copy in flight
            return;
        }
        if (now.count > 0) {
            uint16_t *key = p.keys + static_cast<size_t>(now.code / kSpan) * kDim;
            if (t < kDim / 2) {  // dims 2t, 2t + 1
                float2 m = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < kKeyGroups; ++k) {
                    const float2 v = reinterpret_cast<const float2 *>(part[k])[t];
                    m.x += v.x;
                    m.y += v.y;
                }
                const float tokens = static_cast<float>(now.count);
                reinterpret_cast<uint32_t *>(key)[t] = pack_bf16x2(m.x / tokens, m.y / tokens);
            }
        } else if (t == 0 && p.err) {
            atomicOr(p.err, SMLA_FLAG_BAD_PAGE);
        }
        __syncthreads();
        now = next;
    }
}

// ------------------------------------------------------------------ selection
// One block per request.  Scores become 32-bit keys in the order of the selection (kept spans
// above all, NaN as -inf, -0 as +0; 0 = no span here).  The nsel-th largest key is built bit by
// bit from the top, counting the keys above each candidate, and the search stops early once a
// candidate separates exactly nsel keys.  Then one pass in index order writes the spans above
// the key and the first of those equal to it.  Bound by its chain of barriers, over 4 bytes read per
// span: in a graph 5.6 us for one row of 128 spans, 8.5 us for 256 rows of up to 2,048.
// The block is the smallest that holds a row in registers, 8 or 16 keys a thread: fewer warps at a
// barrier.  256 rows (in a graph) of 2,048 spans: 256 x 8 8.7 us, 256 x 16 11.8, 512 x 16 18.0, 1,024 x 16 35;
// of 4,096: 256 x 16 12.7, 256 x 32 19.8, 512 x 16 19.0; of 8,192: 512 x 16 21.3, 256 x 32 24.2, 1,024 x 8 26.1,
// held nowhere 81.  64 rows of 16,384: 1,024 x 16 22.7, held nowhere 79.  Longer rows are read again from
// L2 on every pass: 154 us for 64 rows of 32,768 (1,024 x 32 spills registers).
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
    {
        static std::mutex mutex;
        static bool ready[smla::host::kMaxDevices] = {};
        std::lock_guard<std::mutex> lock(mutex);
        if (!ready[dev] && cudaFuncSetAttribute(span_keys_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeySmem) != cudaSuccess)
            return SMLA_ERR_CUDA;
        ready[dev] = true;
    }
    const KeyParams p{kv_cache, block_table, seq_lens, req, span, static_cast<uint16_t *>(keys), err, num_pages, n, B, max_blocks};
    const int blocks = n < kKeyBlocks * sms ? n : kKeyBlocks * sms;
    span_keys_kernel<<<static_cast<unsigned>(blocks), kKeyThreads, kKeySmem, static_cast<cudaStream_t>(stream)>>>(p);
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
    else if (width <= 256 * 16)
        select_spans_kernel<256, 16><<<blocks, 256, 0, st>>>(p);
    else if (width <= 512 * 16)
        select_spans_kernel<512, 16><<<blocks, 512, 0, st>>>(p);
    else if (width <= 1024 * 16)
        select_spans_kernel<1024, 16><<<blocks, 1024, 0, st>>>(p);
    else
        select_spans_kernel<1024, 0><<<blocks, 1024, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

}  // extern "C"
