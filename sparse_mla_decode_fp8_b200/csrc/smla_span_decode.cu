// smla_span_decode.cu -- attention of one new token per request over its whole cached sequence,
// or over a list of its 64-token spans: softmax(sm_scale q K^T) K with K the dequantised latents
// (K is key and value), 64 heads per request, split over the sequence and joined.
//
// Mathematics.  For the tokens t a CTA has seen, it keeps per head a reference m >= the scores
// less kRescaleThreshold (log2 units, s = sm_scale log2(e) q.k), L = sum_t 2^(s_t - m) and
// O^T = sum_t 2^(s_t - m) k_t.  A part of a request is O / L with lambda = m + log2 L; parts join
// by weights 2^(lambda_i - max lambda).  Sums and statistics are fp32.  The weights 2^(s - m)
// enter the second product as bf16 (half a step: 2^-8 of each weight, in proportion to the
// weight, so at most 2^-8 of sum p |k| / L before the bf16 output's own rounding; L and the
// log-sum-exp sum the unrounded weights).
//
// Work: 584 bytes and 131,072 flops per token, 224 flop/byte, near the balance of the machine
// (252): the token rows have to stream while the tensor core is nearly always busy.
//
// Split: the tokens of all requests form one sequence of 128-token tiles (two spans), cut into
// equal contiguous ranges, one per CTA (one CTA per SM).  Lengths are read on the device, so
// a captured graph serves any lengths.  A request inside one CTA's range is finished by it;
// the others leave parts (at most two per CTA) that the join kernel adds in a fixed order.
//
// Roles (16 warps): 8 warps dequantise, 4 run the softmax and the epilogue, one thread
// issues the MMAs, one warp walks the CTA's range and publishes a tile's pages in a ring.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "smla_device.cuh"
#include "smla_host.cuh"
#include "smla_tile.cuh"

namespace smla {
namespace span_decode {

constexpr int kSpan = SMLA_SPAN_TOKENS;
constexpr int kDequantWarps = 8;
constexpr int kSoftmaxWarps = 4;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kMmaWarp = kDequantWarps + kSoftmaxWarps;  // 12
constexpr int kWalkWarp = kMmaWarp + 1;                  // 13
constexpr int kThreads = 512;                            // 16 warps: 128 registers a thread
constexpr int kRing = 4;                                 // tiles published ahead
constexpr uint32_t kBarIdSoftmax = 1;                    // named barrier of the softmax warps
constexpr float kRescaleThreshold = 64.0f;               // log2 units
constexpr int kCombineThreads = 256;

// Dynamic shared memory map (bytes from a 1024-aligned base).
constexpr int kSmemQ = 0;                          // 64 KB: 8 K-blocks x [64 heads x 128 B], TMA-written
constexpr int kSmemKV = kSmemQ + 65536;            // 128 KB: 8 K-blocks x [128 tokens x 128 B]
constexpr int kSmemP = kSmemKV + 131072;           // 16 KB: P^T [128 tokens x 64 heads] bf16
constexpr int kSmemRing = kSmemP + 16384;          // [kRing] Tile
constexpr int kSmemRed = kSmemRing + kRing * 32;   // [4][64] f32: per-quadrant maxima or sums
constexpr int kSmemHeadM = kSmemRed + 1024;        // [64] m per head
constexpr int kSmemAlpha = kSmemHeadM + 256;       // [64] rescale factors; 1/L in the epilogue
constexpr int kSmemScan = kSmemAlpha + 256;        // block scan of the tile counts: [16] + 4 int64
constexpr int kSmemBars = kSmemScan + 160;
enum Bar : int {
    kBarRingFull = 0,               // + slot
    kBarRingEmpty = kRing,          // + slot: dequant warps, softmax warps and the MMA thread are done with it
    kBarQ = 2 * kRing,              // Q of the current request landed
    kBarKvFull = kBarQ + 1,         // + dims chunk c: chunk written (8 warps)
    kBarKvFree = kBarKvFull + 4,    // + c: the PV of chunk c is done
    kBarS = kBarKvFree + 4,         // S^T of the tile complete
    kBarP = kBarS + 1,              // P^T written (4 warps)
    kBarDrain = kBarP + 1,
    kBarSpare = kBarDrain + 1,      // test hook target
    kNumBars = kBarSpare + 1,
};
constexpr int kSmemTmemSlot = kSmemBars + 8 * kNumBars;
constexpr int kSmemAbort = kSmemTmemSlot + 4;
constexpr int kSmemBytes = kSmemAbort + 4;
static_assert(kSmemBars % 8 == 0 && kSmemScan % 8 == 0, "8-byte alignment");
static_assert(kSmemBytes <= 232448, "exceeds the 227 KB per-block shared memory limit");

// Tensor memory: O^T chunk c (dims 128c..) in columns [64c, 64c + 64), then S^T, then L per lane.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 256;
constexpr uint32_t kTmemL = 320;

extern __shared__ __align__(1024) uint8_t g_smem[];

// A published tile: the two spans' codes (page * 4 + quarter, or -1) and how many tokens of each
// count; the request; what the tile is in its segment (a request's part in this CTA's range).
struct alignas(16) Tile {
    int code[2];
    int count[2];
    int b;     // -1: no more tiles
    int flags;
    int part;  // of the segment's last tile: index of the part to write, -1: the request is whole
    int pad;
};
constexpr int kFirst = 1, kLast = 2;

struct Params {
    const uint8_t *cache;
    const int32_t *block_table;
    const int32_t *spans;  // null: all
    const int32_t *seq_lens;
    uint16_t *out;
    float *lse;
    float *part_o;         // [2 grid][64][512]
    float *part_lambda;    // [2 grid][64], log2 units
    long long *prefix;     // [B + 1] tiles before each request
    int32_t *failed;       // [grid]
    uint32_t *err;
    long long num_pages;
    unsigned long long timeout_ns;
    int B, max_blocks, nsel;
    float scale_log2;
    uint32_t debug_flags;
};

__device__ __forceinline__ uint64_t *sm_bar(int i) { return reinterpret_cast<uint64_t *>(g_smem + kSmemBars) + i; }
__device__ __forceinline__ Tile *sm_ring() { return reinterpret_cast<Tile *>(g_smem + kSmemRing); }
__device__ __forceinline__ float *sm_red() { return reinterpret_cast<float *>(g_smem + kSmemRed); }
__device__ __forceinline__ float *sm_head_m() { return reinterpret_cast<float *>(g_smem + kSmemHeadM); }
__device__ __forceinline__ float *sm_alpha() { return reinterpret_cast<float *>(g_smem + kSmemAlpha); }
__device__ __forceinline__ long long *sm_scan() { return reinterpret_cast<long long *>(g_smem + kSmemScan); }
__device__ __forceinline__ volatile int *sm_abort() { return reinterpret_cast<volatile int *>(g_smem + kSmemAbort); }

// Bounded wait on an mbarrier phase: false when the CTA has been aborted or the time is out
// (which aborts it and sets the error word).
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, const Params &p) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t k = 1;; ++k) {
        if (mbar_test_wait(bar, parity)) return true;
        if ((k & 31u) != 0) continue;
        if (*sm_abort()) return false;
        if (global_timer_ns() - t0 > p.timeout_ns) {
            *sm_abort() = 1;
            atomicOr(p.err, SMLA_FLAG_TIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_bar(int bar, uint32_t parity, const Params &p) {
    return mbar_test_wait(sm_bar(bar), parity) || wait_slow(sm_bar(bar), parity, p);
}
// Lane 0 waits, the warp follows.
__device__ __forceinline__ bool warp_wait(int bar, uint32_t parity, const Params &p, int lane) {
    int ok = 1;
    if (lane == 0) ok = wait_bar(bar, parity, p) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();  // orders the other lanes after lane 0's observation
    return ok != 0;
}

// Number of tiles of request b.
__device__ __forceinline__ long long tiles_of(const Params &p, int b) {
    const int len = __ldg(p.seq_lens + b);
    if (len <= 0) return 0;
    if (p.spans) return (p.nsel + 1) / 2;
    const long long n = min(static_cast<long long>(len), static_cast<long long>(p.max_blocks) * kPageTokens);
    return (n + kTile - 1) / kTile;
}

// The CTA's range of tiles [begin, end) and where it begins.
struct Range {
    long long begin, end, per;
    int b;               // request of tile `begin`
    long long at;        // its first tile's index inside that request
};

// Every thread of the CTA.  The tile counts are scanned over the block; CTA 0 leaves the
// prefix sums for the join kernel.
__device__ __forceinline__ Range find_range(const Params &p, int tid) {
    const int lane = tid & 31, warp = tid >> 5;
    const int each = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * each), b1 = min(p.B, b0 + each);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += tiles_of(p, b);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    long long *scan = sm_scan();
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const long long v = scan[w];
        if (w < warp) before += v;
        total += v;
    }
    before += incl - mine;
    Range r;
    r.per = max(1ll, (total + gridDim.x - 1) / gridDim.x);
    r.begin = min(total, r.per * blockIdx.x);
    r.end = min(total, r.begin + r.per);
    if (before <= r.begin && r.begin < before + mine) {
        long long at = before;
        int b = b0;
        for (;; ++b) {
            const long long n = tiles_of(p, b);
            if (r.begin < at + n) break;
            at += n;
        }
        scan[16] = b;
        scan[17] = r.begin - at;
    }
    if (blockIdx.x == 0) {
        long long at = before;
        for (int b = b0; b < b1; ++b) {
            p.prefix[b] = at;
            at += tiles_of(p, b);
        }
        if (tid == 0) p.prefix[p.B] = total;
    }
    __syncthreads();
    r.b = r.begin < r.end ? static_cast<int>(scan[16]) : p.B;
    r.at = r.begin < r.end ? scan[17] : 0;
    return r;
}

// ------------------------------------------------------------------ the walk
// One warp publishes the CTA's tiles.  32 tiles at a time, a lane each: the page lookups of 32
// tiles are in flight together.
__device__ __forceinline__ void span_code(const Params &p, int b, int len, long long slot, int &code, int &count) {
    code = -1;
    count = 0;
    long long j = slot;
    if (p.spans) {
        if (slot >= p.nsel) return;
        j = __ldg(p.spans + static_cast<size_t>(b) * p.nsel + slot);
    }
    if (j < 0 || j * kSpan >= len || j / (kPageTokens / kSpan) >= p.max_blocks) return;
    const int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks + j / (kPageTokens / kSpan));
    if (page < 0 || page >= p.num_pages) {
        atomicOr(p.err, SMLA_FLAG_BAD_PAGE);
        return;
    }
    code = page * (kPageTokens / kSpan) + static_cast<int>(j % (kPageTokens / kSpan));
    count = static_cast<int>(min(static_cast<long long>(kSpan), len - j * kSpan));
}

__device__ __forceinline__ void walk(const Params &p, const Range &r, int lane) {
    long long left = r.end - r.begin;
    long long at = r.at;
    int k = 0;  // tiles published
    for (int b = r.b; left > 0; ++b, at = 0) {
        const long long total = tiles_of(p, b);
        const int len = __ldg(p.seq_lens + b);
        const long long n = min(left, total - at);  // tiles of this segment
        if (n <= 0) continue;
        left -= n;
        // a part: the first segment of a CTA may begin inside its request, the last may end inside
        const bool whole = n == total;
        const int part = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (at == 0 && b != r.b ? 1 : 0);
        for (long long base = 0; base < n; base += 32) {
            int code[2], count[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                code[u] = -1;
                count[u] = 0;
                if (base + lane < n) span_code(p, b, len, 2 * (at + base + lane) + u, code[u], count[u]);
            }
            const int m = static_cast<int>(min(32ll, n - base));
            for (int i = 0; i < m; ++i, ++k) {
                if (!warp_wait(kBarRingEmpty + k % kRing, ((k / kRing) & 1) ^ 1, p, lane)) return;
                if (lane == i) {
                    Tile t;
                    t.code[0] = code[0];
                    t.code[1] = code[1];
                    t.count[0] = count[0];
                    t.count[1] = count[1];
                    t.b = b;
                    t.flags = (base + i == 0 ? kFirst : 0) | (base + i == n - 1 ? kLast : 0);
                    t.part = part;
                    t.pad = 0;
                    sm_ring()[k % kRing] = t;
                    mbar_arrive(sm_bar(kBarRingFull + k % kRing));
                    // the rows head for L2 while the tiles before them are worked on
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        if (code[u] < 0) continue;
                        const uint8_t *rows = token_row(p.cache, code[u] * kSpan);
                        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(rows), "r"(count[u] * kRowBytes)
                                     : "memory");
                        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(token_scales(p.cache, code[u] * kSpan)),
                                     "r"((count[u] * kScaleRowBytes + 15) & ~15)
                                     : "memory");
                    }
                }
                __syncwarp();
            }
        }
    }
    if (!warp_wait(kBarRingEmpty + k % kRing, ((k / kRing) & 1) ^ 1, p, lane)) return;
    if (lane == 0) {
        sm_ring()[k % kRing].b = -1;
        mbar_arrive(sm_bar(kBarRingFull + k % kRing));
    }
}

// ------------------------------------------------------------------ dequantisation
// Thread t works on the tokens (t >> 3) + 32 j (j = 0..3, the first two in the first span).
// Dims chunks 0..2 (128 nope dims): 16-byte unit t & 7 of each token; chunk 3: nope unit
// 24 + (t & 3) of two of them, and rope unit t & 7 of each.
struct Rows {
    uint4 nope[3][4];
    uint4 nope3[2];
    uint4 rope[4];
    uint2 scales[4];
};

struct Source {
    const uint8_t *row[2];  // first token row of each span
    const uint8_t *scale[2];
    int count[2];
};

__device__ __forceinline__ Source tile_source(const Params &p, const Tile &t) {
    Source s;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int code = max(0, t.code[u]) * kSpan;
        s.row[u] = token_row(p.cache, code);
        s.scale[u] = token_scales(p.cache, code);
        s.count[u] = t.count[u];
    }
    return s;
}

__device__ __forceinline__ void load_chunk(int c, int t, const Source &s, Rows &r) {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int tok = (t >> 3) + 32 * (j & 1);
        const bool valid = tok < s.count[j >> 1];
        const uint8_t *row = s.row[j >> 1] + tok * kRowBytes + 16 * (t & 7);
        if (c < 3)
            r.nope[c][j] = valid ? ld_stream_v4(row + 128 * c) : zero;
        else
            r.rope[j] = valid ? ld_stream_v4(row + kNope) : zero;
        if (c == 3) r.scales[j] = valid ? ld_stream_v2(s.scale[j >> 1] + tok * kScaleRowBytes) : make_uint2(0u, 0u);
    }
    if (c == 3) {
        const int h = (t >> 2) & 1;  // lanes 4..7 of a group take the second span's tokens
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int tok = (t >> 3) + 32 * k;
            const uint8_t *row = (h ? s.row[1] : s.row[0]) + tok * kRowBytes + 384 + 16 * (t & 3);
            r.nope3[k] = tok < (h ? s.count[1] : s.count[0]) ? ld_stream_v4(row) : zero;
        }
    }
}

// 16 e4m3 bytes into token row r of K-block kb, 16-byte units oc and oc + 1 of its bf16 row.  Odd
// K-blocks store their high half first, so that the 8 lanes of a store phase hit 8 bank groups.
__device__ __forceinline__ void store_nope(uint32_t kv, int r, int kb, int oc, const uint4 raw, uint32_t scale,
                                           bool high_first) {
    uint4 lo, hi;
    dequant16(raw, scale, lo, hi);
    const uint32_t row = kv + kb * (kTile * 128) + r * 128;
    const int sw = r & 7, f = high_first ? 1 : 0;
    sts_v4(row + (((oc + f) ^ sw) << 4), f ? hi : lo);
    sts_v4(row + (((oc + 1 - f) ^ sw) << 4), f ? lo : hi);
}

__device__ __forceinline__ void store_chunk(int c, int t, const Rows &r) {
    const uint32_t kv = smem_addr(g_smem + kSmemKV);
    const int k8 = t & 7, k4 = t & 3, h = (t >> 2) & 1;
    if (c < 3) {
        const int kb = 2 * c + h;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            store_nope(kv, (t >> 3) + 32 * j, kb, 2 * k4, r.nope[c][j], scale_byte(r.scales[j], kb), h != 0);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint2 sc = h ? r.scales[2 + k] : r.scales[k];
            store_nope(kv, (t >> 3) + 64 * h + 32 * k, 6, 2 * k4, r.nope3[k], scale_byte(sc, 6), h != 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = (t >> 3) + 32 * j;
            sts_v4(kv + 7 * (kTile * 128) + row * 128 + ((k8 ^ (row & 7)) << 4), r.rope[j]);
        }
    }
}

__device__ __forceinline__ void dequant_role(const Params &p, int t, int lane) {
    Rows rows;
    if (!warp_wait(kBarRingFull, 0, p, lane)) return;
    Tile tile = sm_ring()[0];
    if (tile.b < 0) return;
    {
        const Source s = tile_source(p, tile);
#pragma unroll
        for (int c = 0; c < 4; ++c) load_chunk(3 - c, t, s, rows);
    }
    for (int k = 0;; ++k) {
        // the next tile's pages; this tile's loads are all issued
        __syncwarp();
        if (lane == 0) mbar_arrive(sm_bar(kBarRingEmpty + k % kRing));
        if (!warp_wait(kBarRingFull + (k + 1) % kRing, ((k + 1) / kRing) & 1, p, lane)) return;
        tile = sm_ring()[(k + 1) % kRing];
        const bool more = tile.b >= 0;
        const Source s = tile_source(p, tile);
        const bool live = more;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (k > 0 && !warp_wait(kBarKvFree + c, (k - 1) & 1, p, lane)) return;
            store_chunk(c, t, rows);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(sm_bar(kBarKvFull + c));
            // chunk 3's load also replaces the scales, which chunks 0..3 of this tile have used by then
            if (live) load_chunk(c, t, s, rows);
        }
        if (!more) return;
    }
}

// ------------------------------------------------------------------ MMA issue (one thread)
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t a_lo, uint32_t b_lo, bool accumulate) {
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {  // 16 tokens a step, 2 KB apart in the MN-major V^T and P^T
        const uint32_t o = ks * (2048 >> 4);
        if (ks == 0 && !accumulate)
            mma_bf16_ss(d, desc_from(a_lo, kDescHi), desc_from(b_lo, kDescHi), kIdescPV, 0u);
        else
            mma_bf16_ss_acc(d, desc_from(a_lo + o, kDescHi), desc_from(b_lo + o, kDescHi), kIdescPV);
    }
}

__device__ __forceinline__ void load_q(const CUtensorMap *tmap_q, int b) {
    mbar_arrive_expect_tx(sm_bar(kBarQ), kHeads * kDim * 2);
#pragma unroll
    for (int kb = 0; kb < 8; ++kb)
        tma_load_2d(g_smem + kSmemQ + kb * 8192, tmap_q, 64 * kb, kHeads * b, sm_bar(kBarQ));
}

__device__ __forceinline__ void mma_role(const Params &p, const CUtensorMap *tmap_q, uint32_t tmem) {
    const uint32_t kv = smem_addr(g_smem + kSmemKV);
    const uint32_t qk_a = desc_lo(kv, 16), qk_b = desc_lo(smem_addr(g_smem + kSmemQ), 16);
    const uint32_t pv_a = desc_lo(kv, kTile * 128), pv_b = desc_lo(smem_addr(g_smem + kSmemP), 8192);
    bool ok = wait_bar(kBarRingFull, 0, p), spare_used = false;
    int flags = 0, segments = 0;  // segments: Q loads issued
    if (ok) {
        const int b = sm_ring()[0].b;
        flags = sm_ring()[0].flags;
        mbar_arrive(sm_bar(kBarRingEmpty));
        if (b < 0) ok = false;
        if (ok) {
            load_q(tmap_q, b);
            segments = 1;
        }
    }
    bool q_pending = segments > 0;
    for (int k = 0; ok; ++k) {
        const uint32_t par = k & 1;
        if (flags & kFirst) {
            ok = wait_bar(kBarQ, (segments - 1) & 1, p);
            if (!ok) break;
            q_pending = false;
        }
#pragma unroll 1
        for (int c = 0; c < 4 && ok; ++c) {
            ok = wait_bar(kBarKvFull + c, par, p);
            if (!ok) break;
            tc_fence_after_sync();
            issue_qk_chunk(tmem + kTmemS, qk_a + c * 2 * ((kTile * 128) >> 4), qk_b + c * 2 * (8192 >> 4), c == 0);
        }
        if (!ok) break;
        const bool hook = k == 0 && (p.debug_flags & SMLA_DEBUG_SKIP_FIRST_COMMIT);
        mma_commit(sm_bar(hook ? kBarSpare : kBarS));
        spare_used = spare_used || hook;
        // the next tile; a new request's Q is fetched as soon as this tile's scores are done
        ok = wait_bar(kBarRingFull + (k + 1) % kRing, ((k + 1) / kRing) & 1, p);
        if (!ok) break;
        const int next_b = sm_ring()[(k + 1) % kRing].b, next_flags = sm_ring()[(k + 1) % kRing].flags;
        mbar_arrive(sm_bar(kBarRingEmpty + (k + 1) % kRing));
        if (next_b >= 0 && (next_flags & kFirst)) {
            ok = wait_bar(kBarS, par, p);
            if (!ok) break;
            load_q(tmap_q, next_b);
            ++segments;
            q_pending = true;
        }
        ok = wait_bar(kBarP, par, p);
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            issue_pv(tmem + 64 * c, pv_a + c * 2 * ((kTile * 128) >> 4), pv_b, !(flags & kFirst));
            mma_commit(sm_bar(kBarKvFree + c));
        }
        if (next_b < 0) break;
        flags = next_flags;
    }
    // every MMA and copy issued must be complete before tensor and shared memory are released
    if (spare_used) (void)mbar_wait(sm_bar(kBarSpare), 0, p.timeout_ns);
    if (q_pending) (void)mbar_wait(sm_bar(kBarQ), (segments - 1) & 1, p.timeout_ns);
    mma_commit(sm_bar(kBarDrain));
    (void)mbar_wait(sm_bar(kBarDrain), 0, p.timeout_ns);
}

// ------------------------------------------------------------------ softmax and epilogue
// Warp q (0..3) owns tensor-memory lanes 32q..: tokens of S^T, dims of an O^T chunk.
// Verdicts that the four warps must share go through their named barrier.

// Raises the references to the tile's maxima and rescales what was accumulated by
// 2^(m_old - m_new): on a segment's first tile, and when a score passes m by more than
// kRescaleThreshold.
__device__ __noinline__ void raise_max(const Params &p, uint32_t tmem_lane, int q, int lane, bool valid, bool first) {
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        float y[32];
        tmem_ld32(tmem_lane + kTmemS + 32 * half, y);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 32; ++h) y[h] = valid ? y[h] * p.scale_log2 : -INFINITY;
        sm_red()[q * 64 + 32 * half + lane] = warp_transpose_reduce<true, 32>(y, lane);
    }
    named_barrier_sync(kBarIdSoftmax, kSoftmaxThreads);
    const int t = 32 * q + lane;
    if (t < kHeads) {
        const float *red = sm_red();
        const float tm = fmaxf(fmaxf(red[t], red[64 + t]), fmaxf(red[128 + t], red[192 + t]));
        const float mo = first ? -INFINITY : sm_head_m()[t];
        const float mn = fmaxf(mo, tm);
        sm_alpha()[t] = (mo == -INFINITY) ? 0.0f : exp2f(mo - mn);
        sm_head_m()[t] = mn;
    }
    named_barrier_sync(kBarIdSoftmax, kSoftmaxThreads);
    if (first) return;  // nothing accumulated yet
    // the PV of the tile before is complete: the commit of this tile's scores covers it
#pragma unroll 1
    for (int g = 0; g < 20; ++g) {  // 16 columns at a time: O^T and then L
        const uint32_t col = tmem_lane + (g < 16 ? 16 * g : kTmemL + 16 * (g - 16));
        float al[16], o[16];
        load16(sm_alpha() + 16 * (g & 3), al);
        tmem_ld16(col, o);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 16; ++h) o[h] *= al[h];
        tmem_st16(col, o);
    }
    tmem_wait_st();
}

// L per head over the 128 lanes -> 1/L, and the segment's log-sum-exps.
__device__ __noinline__ void finish_sums(const Params &p, uint32_t tmem_lane, int q, int lane, int b, int part) {
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        float y[32];
        tmem_ld32(tmem_lane + kTmemL + 32 * half, y);
        tmem_wait_ld();
        sm_red()[q * 64 + 32 * half + lane] = warp_transpose_reduce<false, 32>(y, lane);
    }
    named_barrier_sync(kBarIdSoftmax, kSoftmaxThreads);
    const int t = 32 * q + lane;
    if (t < kHeads) {
        const float *red = sm_red();
        const float l = (red[t] + red[64 + t]) + (red[128 + t] + red[192 + t]);
        // l = 0: no valid token; NaN goes through
        const float lambda = l == 0.0f ? -INFINITY : sm_head_m()[t] + log2f(l);
        if (part >= 0)
            p.part_lambda[static_cast<size_t>(part) * kHeads + t] = lambda;
        else
            p.lse[static_cast<size_t>(b) * kHeads + t] = lambda * 0.69314718055994531f;
        sm_alpha()[t] = l == 0.0f ? 0.0f : 1.0f / l;
    }
    named_barrier_sync(kBarIdSoftmax, kSoftmaxThreads);
}

// O^T / L: dim 128c + 32q + lane of every head; a warp's stores of a head are contiguous.
__device__ __noinline__ void write_out(const Params &p, uint32_t tmem_lane, int q, int lane, int b, int part) {
    const size_t first = static_cast<size_t>(part >= 0 ? part : b) * kHeads * kDim + 32 * q + lane;
#pragma unroll 1
    for (int g = 0; g < 16; ++g) {  // dims chunk g / 4, heads 16 (g % 4)..
        float o[16], inv[16];
        tmem_ld16(tmem_lane + 16 * g, o);
        load16(sm_alpha() + 16 * (g & 3), inv);
        tmem_wait_ld();
        const size_t at = first + 128 * (g >> 2) + static_cast<size_t>(16 * (g & 3)) * kDim;
        if (part >= 0) {
#pragma unroll
            for (int h = 0; h < 16; ++h) p.part_o[at + h * kDim] = o[h] * inv[h];
        } else {
#pragma unroll
            for (int h = 0; h < 16; ++h) p.out[at + h * kDim] = static_cast<uint16_t>(pack_bf16x2(o[h] * inv[h], 0.0f));
        }
    }
}

__device__ __forceinline__ void softmax_role(const Params &p, uint32_t tmem, int q, int lane) {
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const int r = 32 * q + lane;  // token row
    const uint32_t prow = smem_addr(g_smem + kSmemP) + r * 128;
    const float c = p.scale_log2;
    for (int k = 0;; ++k) {
        const uint32_t par = k & 1;
        bool ok = warp_wait(kBarRingFull + k % kRing, (k / kRing) & 1, p, lane);
        const Tile tile = sm_ring()[k % kRing];
        const bool done = ok && tile.b < 0;  // leaves through the barriers below: another warp's wait may have failed
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(sm_bar(kBarRingEmpty + k % kRing));
        const bool first = tile.flags & kFirst;
        const bool valid = (r & 63) < tile.count[(r >> 6) & 1];
        ok = ok && !done && warp_wait(kBarS, par, p, lane);
        tc_fence_after_sync();
        float x[64];
        bool over = first || !ok;
        if (ok) {
            tmem_ld32(lane_addr + kTmemS, x);
            tmem_ld32(lane_addr + kTmemS + 32, x + 32);
            tmem_wait_ld();
        }
        if (!over) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float m[16];
                load16(sm_head_m() + 16 * g, m);
#pragma unroll
                for (int h = 0; h < 16; ++h) {
                    x[16 * g + h] = valid ? fmaf(x[16 * g + h], c, -m[h]) : -INFINITY;
                    over |= x[16 * g + h] > kRescaleThreshold;
                }
            }
        }
        if (barrier_or(kBarIdSoftmax, kSoftmaxThreads, over)) {
            if (barrier_or(kBarIdSoftmax, kSoftmaxThreads, !ok)) return;
            raise_max(p, lane_addr, q, lane, valid, first);
            tmem_ld32(lane_addr + kTmemS, x);
            tmem_ld32(lane_addr + kTmemS + 32, x + 32);
            tmem_wait_ld();
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float m[16];
                load16(sm_head_m() + 16 * g, m);
#pragma unroll
                for (int h = 0; h < 16; ++h) x[16 * g + h] = valid ? fmaf(x[16 * g + h], c, -m[h]) : -INFINITY;
            }
        }
#pragma unroll
        for (int h = 0; h < 64; ++h) x[h] = fast_exp2(x[h]);
#pragma unroll
        for (int g = 0; g < 8; ++g)
            sts_v4(prow + ((g ^ (r & 7)) << 4),
                   make_uint4(pack_bf16x2(x[8 * g], x[8 * g + 1]), pack_bf16x2(x[8 * g + 2], x[8 * g + 3]),
                              pack_bf16x2(x[8 * g + 4], x[8 * g + 5]), pack_bf16x2(x[8 * g + 6], x[8 * g + 7])));
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm_bar(kBarP));
        // L += p, after the hand-over: the PV does not read it
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            if (!first) {
                float l[16];
                tmem_ld16(lane_addr + kTmemL + 16 * g, l);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < 16; ++h) x[16 * g + h] += l[h];
            }
            tmem_st16(lane_addr + kTmemL + 16 * g, x + 16 * g);
        }
        tmem_wait_st();
        if (tile.flags & kLast) {
            ok = warp_wait(kBarKvFree + 3, par, p, lane);  // commits complete in order: every chunk of O^T is final
            if (barrier_or(kBarIdSoftmax, kSoftmaxThreads, !ok)) return;
            tc_fence_after_sync();
            finish_sums(p, lane_addr, q, lane, tile.b, tile.part);
            write_out(p, lane_addr, q, lane, tile.b, tile.part);
            tc_fence_before_sync();
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    span_decode_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tmap_q) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // The tiles need a 1024-byte aligned base (128-byte swizzle); the base is the same for every
    // CTA of a launch.
    const bool misplaced = (smem_addr(g_smem) & 1023u) != 0;
    const Range range = find_range(p, tid);
    if (misplaced || range.begin >= range.end) {  // nothing to do, or the join writes NaN
        if (tid == 0) {
            p.failed[blockIdx.x] = misplaced ? 1 : 0;
            if (misplaced) atomicOr(p.err, SMLA_FLAG_SMEM);
        }
        return;
    }
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(g_smem + kSmemTmemSlot);
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    } else if (warp == kWalkWarp && lane == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(sm_bar(kBarRingFull + i), 1);
            mbar_init(sm_bar(kBarRingEmpty + i), kDequantWarps + kSoftmaxWarps + 1);
        }
        mbar_init(sm_bar(kBarQ), 1);
        for (int c = 0; c < 4; ++c) {
            mbar_init(sm_bar(kBarKvFull + c), kDequantWarps);
            mbar_init(sm_bar(kBarKvFree + c), 1);
        }
        mbar_init(sm_bar(kBarS), 1);
        mbar_init(sm_bar(kBarP), kSoftmaxWarps);
        mbar_init(sm_bar(kBarDrain), 1);
        mbar_init(sm_bar(kBarSpare), 1);
        *sm_abort() = 0;
        fence_barrier_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp < kDequantWarps) {
        dequant_role(p, tid, lane);
    } else if (warp < kMmaWarp) {
        softmax_role(p, tmem, warp - kDequantWarps, lane);
    } else if (warp == kMmaWarp) {
        if (lane == 0) mma_role(p, &tmap_q, tmem);
        __syncwarp();
    } else if (warp == kWalkWarp) {
        walk(p, range, lane);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (tid == 0) p.failed[blockIdx.x] = *sm_abort();
}

// ------------------------------------------------------------------ the join
// Block (x, b) finishes heads [x heads_per, ..) of request b: zeros and -inf for a request without
// tiles, NaN where a CTA gave up, nothing for a request that one CTA wrote whole, and
// otherwise the parts, in the order of the CTAs, with weights 2^(lambda - max).
__global__ void __launch_bounds__(kCombineThreads)
    join_kernel(const __grid_constant__ Params p, int grid, int heads_per) {
    const int b = blockIdx.y, t = threadIdx.x;
    const long long begin = p.prefix[b], n = p.prefix[b + 1] - begin, total = p.prefix[p.B];
    const long long per = max(1ll, (total + grid - 1) / grid);
    const int h0 = blockIdx.x * heads_per;
    const int c0 = static_cast<int>(begin / per), c1 = n > 0 ? static_cast<int>((begin + n - 1) / per) : c0 - 1;
    int bad = 0;
    for (int c = c0 + t; c <= c1; c += kCombineThreads) bad |= p.failed[c];
    bad = __syncthreads_or(bad);
    if (c0 == c1 && !bad) return;
    uint32_t *out = reinterpret_cast<uint32_t *>(p.out + (static_cast<size_t>(b) * kHeads) * kDim);
    for (int h = h0; h < h0 + heads_per; ++h) {
        float top = -INFINITY, sum = 0.0f, x = 0.0f, y = 0.0f;
        if (bad) {
            x = y = NAN;
        } else {
            auto part = [&](int c) { return 2 * c + (c == c0 && begin > c * per ? 1 : 0); };
            for (int c = c0; c <= c1; ++c) {
                const float v = p.part_lambda[static_cast<size_t>(part(c)) * kHeads + h];
                top = (isnan(v) || isnan(top)) ? NAN : fmaxf(top, v);
            }
            if (top != -INFINITY) {
#pragma unroll 4
                for (int c = c0; c <= c1; ++c) {
                    const size_t at = static_cast<size_t>(part(c)) * kHeads + h;
                    const float w = exp2f(p.part_lambda[at] - top);
                    const float2 o = reinterpret_cast<const float2 *>(p.part_o + at * kDim)[t];
                    sum += w;
                    x += w * o.x;
                    y += w * o.y;
                }
                x /= sum;
                y /= sum;
            }
        }
        out[h * (kDim / 2) + t] = pack_bf16x2(x, y);
        if (t == 0)
            p.lse[static_cast<size_t>(b) * kHeads + h] =
                bad ? NAN : top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
    }
}

}  // namespace span_decode
}  // namespace smla

namespace {

using namespace smla::span_decode;

// Workspace after the header: failed [grid], prefix [B + 1], part_lambda, part_o.
struct Layout {
    size_t failed, prefix, lambda, o, bytes;
};
Layout layout_for(int B, int grid) {
    using smla::host::round256;
    Layout l;
    l.failed = SMLA_WORKSPACE_HEADER;
    l.prefix = l.failed + round256(static_cast<size_t>(grid) * 4);
    l.lambda = l.prefix + round256((static_cast<size_t>(B) + 1) * 8);
    l.o = l.lambda + round256(static_cast<size_t>(2 * grid) * SMLA_HEADS * 4);
    l.bytes = l.o + static_cast<size_t>(2 * grid) * SMLA_HEADS * SMLA_DIM * 4;
    return l;
}

int prepare_kernel(int dev) {
    static std::mutex mutex;
    static bool ready[smla::host::kMaxDevices] = {};
    std::lock_guard<std::mutex> lock(mutex);
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(span_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
            cudaSuccess)
            return SMLA_ERR_CUDA;
        ready[dev] = true;
    }
    return SMLA_OK;
}

}  // namespace

extern "C" {

size_t smla_decode_spans_workspace_bytes(int B) {
    if (B < 1 || B > 65535) return 0;
    int dev = 0, sms = 0;
    if (smla::host::current_device(dev, sms) != SMLA_OK) return 0;
    return layout_for(B, sms).bytes;
}

int smla_decode_spans(const void *q, const uint8_t *kv_cache, const int32_t *block_table, const int32_t *spans,
                      int nsel, const int32_t *seq_lens, float sm_scale, void *out, float *lse, int B, int H,
                      int max_blocks, int num_pages, void *workspace, size_t workspace_bytes,
                      const smla_options *opts, void *stream) {
    using smla::host::aligned;
    if (!q || !kv_cache || !block_table || !seq_lens || !out || !lse || !workspace) return SMLA_ERR_INVALID;
    if (B < 1 || B > 65535 || H != SMLA_HEADS || max_blocks < 1 || num_pages < 1 || num_pages >= (1 << 23))
        return SMLA_ERR_INVALID;
    if (spans ? (nsel < 1 || nsel > SMLA_MAX_NSEL) : nsel != 0) return SMLA_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(workspace, 256) ||
        !aligned(block_table, 4) || !aligned(spans, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4))
        return SMLA_ERR_INVALID;
    if (!std::isfinite(sm_scale) || (opts && (opts->nsplit != 0 || opts->out_bf16 == 0))) return SMLA_ERR_INVALID;
    int dev = 0, sms = 0;
    int rc = smla::host::current_device(dev, sms);
    if (rc != SMLA_OK) return rc;
    const Layout l = layout_for(B, sms);
    if (workspace_bytes < l.bytes) return SMLA_ERR_INVALID;
    rc = prepare_kernel(dev);
    if (rc != SMLA_OK) return rc;
    alignas(64) CUtensorMap tmap_q;
    rc = smla::host::encode_q_map(&tmap_q, q, B);
    if (rc != SMLA_OK) return rc;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    Params p{};
    p.cache = kv_cache;
    p.block_table = block_table;
    p.spans = spans;
    p.seq_lens = seq_lens;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.part_o = reinterpret_cast<float *>(ws + l.o);
    p.part_lambda = reinterpret_cast<float *>(ws + l.lambda);
    p.prefix = reinterpret_cast<long long *>(ws + l.prefix);
    p.failed = reinterpret_cast<int32_t *>(ws + l.failed);
    p.err = reinterpret_cast<uint32_t *>(ws);
    p.num_pages = num_pages;
    p.timeout_ns = (opts && opts->wait_timeout_ns) ? opts->wait_timeout_ns : 1000000000ull;
    p.B = B;
    p.max_blocks = max_blocks;
    p.nsel = nsel;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    p.debug_flags = opts ? opts->debug_flags : 0u;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    (void)cudaGetLastError();
    span_decode_kernel<<<static_cast<unsigned>(sms), kThreads, kSmemBytes, st>>>(p, tmap_q);
    if (cudaGetLastError() != cudaSuccess) return SMLA_ERR_LAUNCH;
    const int heads_per = B >= 32 ? 8 : 1;
    join_kernel<<<dim3(SMLA_HEADS / heads_per, static_cast<unsigned>(B)), kCombineThreads, 0, st>>>(p, sms, heads_per);
    return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

}  // extern "C"
