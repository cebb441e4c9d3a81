// smla_span_scores.cu -- how much of a request's attention each of its spans should get, estimated
// from the span keys: score_j = sum over the 64 heads of softmax_j(sm_scale q_h . key_j).
//
// Mathematics.  x_hj = sm_scale log2(e) q_h . key_j (exact bf16 products, fp32 sums).  The first kernel
// leaves x and, per 128 spans and head, their maximum m and sum l = sum_j 2^(x - m); the second
// joins these to lambda_h = M + log2 sum l 2^(m - M) and sums 2^(x_hj - lambda_h) over the heads in a
// fixed order.  All of it is fp32.  The second is launched while the first still runs and waits for it, before it
// reads anything (2 us a call less); it reads what the first wrote through L2.
//
// Work: 1,024 bytes and 65,536 flops per span, 64 flop/byte: bound by the keys' way through HBM.  One CTA
// per SM walks an equal contiguous part of all requests' 128-span tiles (lengths are read on the
// device) and keeps up to 7 of the 8 key chunks [128 spans x 64 dims] in flight; Q stays in
// shared memory for the CTA's tiles of a request.  x (256 bytes a span) goes through L2.
// 64 requests of 65,536 tokens take 26.5 us in a graph for a floor of 11 (67 MB of keys, which are partly in L2
// from one call to the next; 39 us with L2 flushed, launch included): besides HBM the load-store pipe counts, a
// cycle for 32 bytes of keys and of x (x by 16-byte stores, half a sector each: 2 us more), and the chain start -
// load - MMA - statistics - second kernel, which is nearly all of the 10 to 12 us that few spans take.  The ranges are
// whole tiles: those 512 tiles are 4 for each of 128 CTAs, and 20 SMs get none.
// Every block of the second kernel reads the statistics of all tiles of its request, n^2 / 16 bytes for n spans in
// all: as much as the keys at 16,384 spans (a million tokens; one such request takes 22 us, eight 62 us), and
// more than all else beyond.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "smla_device.cuh"
#include "smla_host.cuh"
#include "smla_range.cuh"
#include "smla_tile.cuh"

namespace smla {
namespace span_scores {

constexpr int kSpan = SMLA_SPAN_TOKENS;
constexpr int kPageSpans = kPageTokens / kSpan;
constexpr int kLoadThreads = 128;   // warps 0..3: key rows
constexpr int kStatThreads = 128;   // warps 4..7: x, maxima, sums
constexpr int kMmaWarp = 8;
constexpr int kThreads = kLoadThreads + kStatThreads + 32;
constexpr int kInFlight = 7;        // chunks
constexpr uint32_t kBarIdLoad = 1, kBarIdStat = 2;
constexpr int kScoreThreads = 256;
constexpr int kScoreSpans = 64;     // spans per block of the second kernel

constexpr int kSmemQ = 0;                      // 64 KB: 8 K-blocks x [64 heads x 128 B], TMA-written
constexpr int kSmemKeys = kSmemQ + 65536;      // 128 KB: 8 K-blocks x [128 spans x 128 B]
constexpr int kSmemCodes = kSmemKeys + 131072; // [128] key rows of the tile being loaded
constexpr int kSmemRed = kSmemCodes + 512;     // [4][64] per-warp maxima or sums
constexpr int kSmemMax = kSmemRed + 1024;      // [64] maxima of the tile, 0 where it has none
constexpr int kSmemScan = kSmemMax + 256;
constexpr int kSmemBars = kSmemScan + 8 * (kThreads / 32 + 2) + 8;
enum Bar : int {
    kBarFull = 0,           // + chunk: landed (128 threads)
    kBarFree = 8,           // + chunk: its MMAs are done
    kBarS = 16,             // + buffer: S^T complete
    kBarSFree = 18,         // + buffer: read (4 warps)
    kBarQ = 20,
    kBarQFree = 21,         // the MMAs that read Q are done
    kBarDrain = 22,
    kNumBars = 23,
};
constexpr int kSmemTmemSlot = kSmemBars + 8 * kNumBars;
constexpr int kSmemAbort = kSmemTmemSlot + 4;
constexpr int kSmemBytes = kSmemAbort + 4;
static_assert(kSmemBars % 8 == 0 && kSmemScan % 8 == 0, "8-byte alignment");
static_assert(kSmemBytes <= 232448, "exceeds the 227 KB per-block shared memory limit");
constexpr uint32_t kTmemCols = 128;            // two S^T buffers of 64 columns

extern __shared__ __align__(1024) uint8_t g_smem[];

struct Params {
    const uint8_t *keys;   // bf16 rows of 1,024 bytes
    const int32_t *block_table;
    const int32_t *seq_lens;
    float *scores;
    float *x;              // [B][width][64], log2 units
    float2 *stats;         // [B][tiles][64]: (maximum, sum) of a tile
    uint32_t *err;
    long long num_pages;
    unsigned long long timeout_ns;
    int B, max_blocks, width, tiles;  // width = 4 max_blocks, tiles = ceil(width / 128)
    float scale_log2;
    uint32_t debug_flags;
};

__device__ __forceinline__ uint64_t *sm_bar(int i) { return reinterpret_cast<uint64_t *>(g_smem + kSmemBars) + i; }
__device__ __forceinline__ volatile int *sm_abort() { return reinterpret_cast<volatile int *>(g_smem + kSmemAbort); }

// Bounded wait of a whole warp on an mbarrier phase, a uniform verdict: false when the CTA has been
// aborted or the time is out (which aborts it and sets the error word).
__device__ __noinline__ bool wait_slow(int bar, uint32_t parity, const Params &p) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait_for(sm_bar(bar), parity, 1000000u)) {
        if (*sm_abort()) return false;
        if (global_timer_ns() - t0 > p.timeout_ns) {
            *sm_abort() = 1;
            atomicOr(p.err, SMLA_FLAG_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool all_wait(int bar, uint32_t parity, const Params &p) {
    const bool ok = mbar_test_wait(sm_bar(bar), parity) || wait_slow(bar, parity, p);
    return __all_sync(0xffffffffu, ok) != 0;
}

__device__ __forceinline__ int spans_of(const Params &p, int b) {
    const int len = p.seq_lens[b];
    return len <= 0 ? 0 : static_cast<int>(min(static_cast<long long>(p.width), (static_cast<long long>(len) + kSpan - 1) / kSpan));
}

// The tiles of a CTA, one after the other.
struct Cursor {
    long long left;
    int b, tile, tiles, spans;
    __device__ __forceinline__ Cursor(const Params &p, const Range &r) : left(r.end - r.begin), b(r.b), tile(static_cast<int>(r.at)) {
        spans = left > 0 ? spans_of(p, b) : 0;
        tiles = (spans + kTile - 1) / kTile;
    }
    __device__ __forceinline__ void next(const Params &p) {
        --left;
        ++tile;
        while (left > 0 && tile >= tiles) {
            ++b;
            tile = 0;
            spans = spans_of(p, b);
            tiles = (spans + kTile - 1) / kTile;
        }
    }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

// ------------------------------------------------------------------ key rows
// Thread t copies the 16-byte unit t & 7 of the rows (t >> 3) + 16 j of every chunk.  Rows without a
// key are zeros.  A chunk is handed over once it has landed, kInFlight - 1 chunks after it was asked for.
__device__ __forceinline__ void load_role(const Params &p, const Range &r, int t) {
    int *codes = reinterpret_cast<int *>(g_smem + kSmemCodes);
    const uint32_t dst = smem_addr(g_smem + kSmemKeys) + (t >> 3) * 128 + (((t & 7) ^ ((t >> 3) & 7)) << 4);
    uint32_t n = 0;  // chunks asked for
    bool ok = true;
    const auto hand_over = [&](uint32_t i) {
        fence_proxy_async_smem();
        if (ok) mbar_arrive(sm_bar(kBarFull + (i & 7)));  // never a chunk that was not copied
    };
    for (Cursor c(p, r); c.left > 0; c.next(p)) {
        const int j = c.tile * kTile + t;
        int code = -1;
        if (j < c.spans) {
            const int page = p.block_table[static_cast<size_t>(c.b) * p.max_blocks + j / kPageSpans];
            if (page >= 0 && page < p.num_pages)
                code = page * kPageSpans + j % kPageSpans;
            else
                atomicOr(p.err, SMLA_FLAG_BAD_PAGE);
        }
        named_barrier_sync(kBarIdLoad, kLoadThreads);  // the codes of the tile before have been read
        codes[t] = code;
        named_barrier_sync(kBarIdLoad, kLoadThreads);
        int mine[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mine[i] = codes[(t >> 3) + 16 * i];
#pragma unroll 1
        for (int kb = 0; kb < 8; ++kb, ++n) {
            // a warp whose wait failed keeps step with the others (the named barriers above) but copies nothing
            ok = ok && (n < 8 || all_wait(kBarFree + kb, ((n >> 3) & 1) ^ 1, p));
            if (ok) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    copy16(dst + kb * (kTile * 128) + 16 * 128 * i,
                           p.keys + static_cast<size_t>(max(mine[i], 0)) * (kDim * 2) + kb * 128 + (t & 7) * 16, mine[i] >= 0);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (n >= kInFlight - 1) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kInFlight - 1) : "memory");
                hand_over(n - (kInFlight - 1));
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (uint32_t i = n > kInFlight - 1 ? n - (kInFlight - 1) : 0; i < n; ++i) hand_over(i);
}

// ------------------------------------------------------------------ MMA issue (one warp)
__device__ __forceinline__ void mma_role(const Params &p, const Range &r, const CUtensorMap *tmap_q, uint32_t tmem) {
    const uint32_t qk_a = desc_lo(smem_addr(g_smem + kSmemKeys), 16), qk_b = desc_lo(smem_addr(g_smem + kSmemQ), 16);
    const bool leader = elect_one();
    int loaded = -1;
    uint32_t n = 0, loads = 0;
    bool ok = true;
    for (Cursor c(p, r); ok && c.left > 0; c.next(p), ++n) {
        if (c.b != loaded) {
            // the MMAs of the request before have read its Q
            if (loads > 0) {
                if (leader) mma_commit(sm_bar(kBarQFree));
                __syncwarp();
                ok = all_wait(kBarQFree, (loads - 1) & 1, p);
                if (!ok) break;
            }
            if (leader) {
                mbar_arrive_expect_tx(sm_bar(kBarQ), kHeads * kDim * 2);
#pragma unroll
                for (int kb = 0; kb < 8; ++kb)
                    tma_load_2d(g_smem + kSmemQ + kb * 8192, tmap_q, 64 * kb, kHeads * c.b, sm_bar(kBarQ));
            }
            __syncwarp();
            loaded = c.b;
            ++loads;
            ok = all_wait(kBarQ, (loads - 1) & 1, p);
            if (!ok) break;
        }
        const uint32_t buf = n & 1;
        ok = n < 2 || all_wait(kBarSFree + buf, ((n >> 1) & 1) ^ 1, p);
#pragma unroll 1
        for (int kb = 0; ok && kb < 8; ++kb) {
            ok = all_wait(kBarFull + kb, n & 1, p);
            if (!ok) break;
            tc_fence_after_sync();
            if (leader) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16_ss(tmem + 64 * buf, desc_from(qk_a + kb * ((kTile * 128) >> 4) + 2 * k, kDescHi),
                                desc_from(qk_b + kb * (8192 >> 4) + 2 * k, kDescHi), kIdescQK, (kb > 0 || k > 0) ? 1u : 0u);
                mma_commit(sm_bar(kBarFree + kb));
            }
            __syncwarp();
        }
        const bool hook = n == 0 && (p.debug_flags & SMLA_DEBUG_SKIP_FIRST_COMMIT);
        if (ok && leader && !hook) mma_commit(sm_bar(kBarS + buf));
        __syncwarp();
    }
    // every MMA and copy issued must be complete before tensor and shared memory are released
    if (leader) {
        if (loads) (void)mbar_wait(sm_bar(kBarQ), (loads - 1) & 1, kDrainNs);
        mma_commit(sm_bar(kBarDrain));
        (void)mbar_wait(sm_bar(kBarDrain), 0, kDrainNs);
    }
    __syncwarp();
}

// ------------------------------------------------------------------ x, maxima, sums
// Warp q (0..3) owns tensor-memory lanes 32q..: a span a thread, 64 heads.
__device__ __forceinline__ void stat_role(const Params &p, const Range &r, uint32_t tmem, int q, int lane) {
    float *red = reinterpret_cast<float *>(g_smem + kSmemRed), *base = reinterpret_cast<float *>(g_smem + kSmemMax);
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const int t = 32 * q + lane;
    uint32_t n = 0;
    bool ok = true;
    for (Cursor c(p, r); c.left > 0; c.next(p), ++n) {
        const uint32_t buf = n & 1;
        const int j = c.tile * kTile + t;
        bool valid = false;
        if (j < c.spans) {
            const int page = p.block_table[static_cast<size_t>(c.b) * p.max_blocks + j / kPageSpans];
            valid = page >= 0 && page < p.num_pages;
        }
        ok = ok && all_wait(kBarS + buf, (n >> 1) & 1, p);
        ok = !barrier_or(kBarIdStat, kStatThreads, !ok);
        float2 *stats = p.stats + (static_cast<size_t>(c.b) * p.tiles + c.tile) * kHeads;
        if (!ok) {  // the tile's request becomes NaN; the tiles after it too
            if (t < kHeads) stats[t] = make_float2(NAN, NAN);
            continue;
        }
        tc_fence_after_sync();
        float *out = p.x + (static_cast<size_t>(c.b) * p.width + j) * kHeads;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            float x[32], y[32];
            tmem_ld32(lane_addr + 64 * buf + 32 * half, x);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 32; ++h) y[h] = x[h] = valid ? x[h] * p.scale_log2 : -INFINITY;
            if (j < c.spans)
#pragma unroll
                for (int g = 0; g < 4; ++g) st_global_v8(out + 32 * half + 8 * g, x + 8 * g);
            red[q * 64 + 32 * half + lane] = warp_transpose_reduce<true, 32>(y, lane);
        }
        named_barrier_sync(kBarIdStat, kStatThreads);
        float top = 0.0f;  // of head t
        if (t < kHeads) {
            top = fmaxf(fmaxf(red[t], red[64 + t]), fmaxf(red[128 + t], red[192 + t]));
            // the maximum passes NaN over: where it is -inf, weights 2^(x - 0) are 0 for -inf and NaN for NaN
            base[t] = top == -INFINITY ? 0.0f : top;
        }
        named_barrier_sync(kBarIdStat, kStatThreads);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            float x[32];
            tmem_ld32(lane_addr + 64 * buf + 32 * half, x);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 32; ++h) {
                x[h] = valid ? fast_exp2(x[h] * p.scale_log2 - base[32 * half + h]) : 0.0f;
            }
            red[q * 64 + 32 * half + lane] = warp_transpose_reduce<false, 32>(x, lane);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm_bar(kBarSFree + buf));
        named_barrier_sync(kBarIdStat, kStatThreads);
        if (t < kHeads) stats[t] = make_float2(top, (red[t] + red[64 + t]) + (red[128 + t] + red[192 + t]));
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    span_logits_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tmap_q) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Launched while the kernel before it drains (1.5 us a call).  No load in here is of the read-only kind, which
    // holds only for data older than the kernel's launch.
    wait_for_prior_kernel();
    let_next_kernel_start();
    const Range range = find_range<kThreads>(
        [&](int b) { return static_cast<long long>((spans_of(p, b) + kTile - 1) / kTile); }, p.B,
        reinterpret_cast<long long *>(g_smem + kSmemScan), nullptr);
    if (range.begin >= range.end) return;
    if (smem_addr(g_smem) & 1023u) {  // the same for every CTA: the swizzled tiles need this alignment
        if (tid == 0) atomicOr(p.err, SMLA_FLAG_SMEM);
        for (Cursor c(p, range); c.left > 0; c.next(p))
            if (tid < kHeads) p.stats[(static_cast<size_t>(c.b) * p.tiles + c.tile) * kHeads + tid] = make_float2(NAN, NAN);
        return;
    }
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(g_smem + kSmemTmemSlot);
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    } else if (tid == 0) {
        for (int i = 0; i < 8; ++i) {
            mbar_init(sm_bar(kBarFull + i), kLoadThreads);
            mbar_init(sm_bar(kBarFree + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sm_bar(kBarS + i), 1);
            mbar_init(sm_bar(kBarSFree + i), kStatThreads / 32);
        }
        mbar_init(sm_bar(kBarQ), 1);
        mbar_init(sm_bar(kBarQFree), 1);
        mbar_init(sm_bar(kBarDrain), 1);
        *sm_abort() = 0;
        fence_barrier_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    if (warp < kLoadThreads / 32)
        load_role(p, range, tid);
    else if (warp < kMmaWarp)
        stat_role(p, range, tmem, warp - kLoadThreads / 32, lane);
    else
        mma_role(p, range, &tmap_q, tmem);
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Block (x, b): kScoreSpans spans of request b.  lambda per head from the tiles' statistics, then the
// sum over the heads, 16 lanes of 4 heads per span.
__global__ void __launch_bounds__(kScoreThreads) span_scores_kernel(const __grid_constant__ Params p) {
    __shared__ float part_m[4][kHeads], part_l[4][kHeads], lambda[kHeads];
    const int t = threadIdx.x, b = blockIdx.y, first = blockIdx.x * kScoreSpans;
    // Every block waits, also one that needs nothing (this kernel must not end before the first one), and before it reads
    // the lengths, which a kernel ahead of both may have written.
    wait_for_prior_kernel();
    const int spans = spans_of(p, b), tiles = (spans + kTile - 1) / kTile;
    float *scores = p.scores + static_cast<size_t>(b) * p.width;
    if (first >= spans) {  // block-uniform: behind the sequence
        if (t < kScoreSpans && first + t < p.width) scores[first + t] = 0.0f;
        return;
    }
    const int h = t & 63, part = t >> 6;
    float m = -INFINITY, l = 0.0f;
    bool bad = false;  // a tile whose CTA gave up
    for (int i = part; i < tiles; i += 4) {
        const float2 s = __ldcg(p.stats + (static_cast<size_t>(b) * p.tiles + i) * kHeads + h);
        bad |= isnan(s.y);
        const float up = fmaxf(m, s.x);
        if (up != -INFINITY) l = l * exp2f(m - up) + s.y * exp2f(s.x - up);
        m = up;
    }
    part_m[part][h] = m;
    part_l[part][h] = bad ? NAN : l;
    __syncthreads();
    if (t < kHeads) {
        const float up = fmaxf(fmaxf(part_m[0][t], part_m[1][t]), fmaxf(part_m[2][t], part_m[3][t]));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sum += up == -INFINITY ? part_l[i][t] : part_l[i][t] * exp2f(part_m[i][t] - up);
        // no span has a key: every x is -inf, and 0 lets 2^(x - lambda) be 0
        lambda[t] = up == -INFINITY && sum == 0.0f ? 0.0f : up + log2f(sum);
    }
    __syncthreads();
    const int lane = t & 31, g = lane & 15;
    const float4 lam = reinterpret_cast<const float4 *>(lambda)[g];
    for (int i = 2 * (t >> 5) + (lane >> 4); i < kScoreSpans; i += 2 * (kScoreThreads / 32)) {
        const int j = first + i;
        float s = 0.0f;
        if (j < spans) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(p.x + (static_cast<size_t>(b) * p.width + j) * kHeads) + g);
            s = (exp2f(x.x - lam.x) + exp2f(x.y - lam.y)) + (exp2f(x.z - lam.z) + exp2f(x.w - lam.w));
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (g == 0 && j < p.width) {
            // a request with a NaN: its spans in bad pages still score 0 (x = -inf, less a lambda of NaN)
            if (isnan(s)) {
                const int page = p.block_table[static_cast<size_t>(b) * p.max_blocks + j / kPageSpans];
                if (page < 0 || page >= p.num_pages) s = 0.0f;
            }
            scores[j] = s;
        }
    }
}

}  // namespace span_scores
}  // namespace smla

namespace {

using namespace smla::span_scores;

// Workspace after the header: statistics, x.
struct Layout {
    size_t stats, x, bytes;
};
Layout layout_for(int B, int max_blocks) {
    const size_t width = static_cast<size_t>(max_blocks) * kPageSpans, tiles = (width + smla::kTile - 1) / smla::kTile;
    Layout l;
    l.stats = SMLA_WORKSPACE_HEADER;
    l.x = l.stats + smla::host::round256(B * tiles * SMLA_HEADS * sizeof(float2));
    l.bytes = l.x + B * width * SMLA_HEADS * sizeof(float);
    return l;
}

int prepare_kernel(int dev) {
    static std::mutex mutex;
    static bool ready[smla::host::kMaxDevices] = {};
    std::lock_guard<std::mutex> lock(mutex);
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(span_logits_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess)
            return SMLA_ERR_CUDA;
        ready[dev] = true;
    }
    return SMLA_OK;
}

bool sizes_ok(int B, int max_blocks) {
    return B >= 1 && B <= 65535 && max_blocks >= 1 && max_blocks <= SMLA_MAX_SPANS / kPageSpans;
}

}  // namespace

extern "C" {

size_t smla_span_scores_workspace_bytes(int B, int max_blocks) {
    return sizes_ok(B, max_blocks) ? layout_for(B, max_blocks).bytes : 0;
}

int smla_span_scores(const void *q, const void *keys, const int32_t *block_table, const int32_t *seq_lens,
                     float sm_scale, float *scores, int B, int H, int max_blocks, int num_pages, void *workspace,
                     size_t workspace_bytes, const smla_options *opts, void *stream) {
    using smla::host::aligned;
    if (!q || !keys || !block_table || !seq_lens || !scores || !workspace) return SMLA_ERR_INVALID;
    if (!sizes_ok(B, max_blocks) || H != SMLA_HEADS || num_pages < 1 || num_pages >= (1 << 23)) return SMLA_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(keys, 16) || !aligned(workspace, 256) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(scores, 4))
        return SMLA_ERR_INVALID;
    if (!std::isfinite(sm_scale) || (opts && (opts->nsplit != 0 || opts->out_bf16 != 0))) return SMLA_ERR_INVALID;
    const Layout l = layout_for(B, max_blocks);
    if (workspace_bytes < l.bytes) return SMLA_ERR_INVALID;
    int dev = 0, sms = 0;
    int rc = smla::host::current_device(dev, sms);
    if (rc != SMLA_OK) return rc;
    rc = prepare_kernel(dev);
    if (rc != SMLA_OK) return rc;
    alignas(64) CUtensorMap tmap_q;
    rc = smla::host::encode_q_map(&tmap_q, q, B);
    if (rc != SMLA_OK) return rc;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    Params p{};
    p.keys = static_cast<const uint8_t *>(keys);
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.scores = scores;
    p.x = reinterpret_cast<float *>(ws + l.x);
    p.stats = reinterpret_cast<float2 *>(ws + l.stats);
    p.err = reinterpret_cast<uint32_t *>(ws);
    p.num_pages = num_pages;
    p.timeout_ns = (opts && opts->wait_timeout_ns) ? opts->wait_timeout_ns : 1000000000ull;
    p.B = B;
    p.max_blocks = max_blocks;
    p.width = max_blocks * kPageSpans;
    p.tiles = (p.width + smla::kTile - 1) / smla::kTile;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    p.debug_flags = opts ? opts->debug_flags : 0u;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    (void)cudaGetLastError();
    const long long most = static_cast<long long>(B) * p.tiles;
    const dim3 ctas(static_cast<unsigned>(most < sms ? most : sms));
    if (smla::host::launch_after(span_logits_kernel, ctas, kThreads, kSmemBytes, st, p, tmap_q) != cudaSuccess) return SMLA_ERR_LAUNCH;
    const dim3 grid(static_cast<unsigned>((p.width + kScoreSpans - 1) / kScoreSpans), static_cast<unsigned>(B));
    if (smla::host::launch_after(span_scores_kernel, grid, kScoreThreads, 0, st, p) != cudaSuccess) return SMLA_ERR_LAUNCH;
    return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

}  // extern "C"
