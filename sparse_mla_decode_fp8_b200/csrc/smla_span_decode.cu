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
// Roles (28 warps): four warpgroups dequantise, one 128-dim chunk of the tile each; two run the
// softmax and the epilogue; of the last, one warp issues the MMAs and one walks the CTA's range and
// publishes a tile's pages in a ring.
//
// What bounds it (64 requests of 65536 tokens, 860 to 917 us from one GPU to the other at the 1 kW cap: 2.68 to
// 2.86 TB/s, 600 to 640 TFLOP/s; a tile takes about 7,100 cycles): the chain of one tile.  Q, one converted
// tile and P^T fill shared memory, so a chunk is stored when the second product of the tile before has
// released it.  By clock stamps, from the hand-over
// of P^T: second product 1,950 cycles, the last chunk stored 1,000 later (the first pair's MMAs run by
// then), scores complete 2,000 after that, weights handed over 1,700 after that.  Under the chain lies shared
// memory's port: the MMAs read 128 bytes a cycle for 3,100 cycles, the conversions store for 1,000, and the
// loads of raw nope rows take the same pipe a cycle for 32 bytes, 1,800 (without row loads a tile
// took 5,900).  Tried and slower: 96-token tiles with all raw rows by TMA 13 %, chunk 1 by TMA through
// the place of P^T 16 %, row loads held back until P^T is done 14 %; the last nope group by TMA through
// 8 KB of its own gains nothing, rope values by TMA straight into the tile 3 %.  With few tokens a start
// of 15,000 cycles counts: cold instructions, the lookups, one tile's chain of loads and barriers; and a
// part's 128 KB, stored in 5,000 cycles and read again by the join.  The join has a warp per (request, head), which walks
// the request's parts in turn: with one long request that is 64 warps on 8 SMs for up to 148 parts, and most of the
// call (one request of 32,768 tokens 66 us, of 131,072 95 us).  With a list every two entries are a tile, -1 or not: 64
// requests of 300 tokens with 64 entries take 73 us.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "smla_device.cuh"
#include "smla_host.cuh"
#include "smla_range.cuh"
#include "smla_tile.cuh"

namespace smla {
namespace span_decode {

constexpr int kSpan = SMLA_SPAN_TOKENS;
constexpr int kChunks = 4;                        // dims chunks of 128, a dequantising warpgroup each
constexpr int kDequantWarps = 4 * kChunks;
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kMmaWarp = kDequantWarps + kSoftmaxWarps;  // 24
constexpr int kWalkWarp = kMmaWarp + 1;                  // 25
constexpr int kThreads = 32 * (kDequantWarps + kSoftmaxWarps + 4);
// Registers a thread: 72 at launch (896 threads); the control warps give to those that dequantise.
constexpr int kRegsLaunch = 72, kRegsNope = 80, kRegsTail = 80, kRegsSoftmax = 72, kRegsControl = 40;
static_assert(32 * ((kDequantWarps - 4) * kRegsNope + 4 * kRegsTail + kSoftmaxWarps * kRegsSoftmax + 4 * kRegsControl) <=
                  kThreads * kRegsLaunch && kThreads * kRegsLaunch <= 65536,
              "the shares are drawn from what the block was launched with");
constexpr int kRing = 4;                                 // tiles published ahead
// The chunks' order in both products, two at a time in the first: chunk 3 first, since its rope values are
// copied in when the second product of the tile before has released it.
__device__ constexpr int chunk_at(int i) { return (i + 3) % kChunks; }
__device__ constexpr int pair_of(int c) { return (c + 1) % kChunks / 2; }
static_assert(chunk_at(0) == 3 && pair_of(chunk_at(1)) == 0 && pair_of(chunk_at(2)) == 1, "3, 0 and 1, 2");
constexpr uint32_t kBarIdSoftmax = 1;                    // named barrier of the softmax warps
constexpr float kRescaleThreshold = 64.0f;               // log2 units
constexpr int kJoinWarps = 8;

// Dynamic shared memory map (bytes from a 1024-aligned base).
constexpr int kSmemQ = 0;                          // 64 KB: 8 K-blocks x [64 heads x 128 B], TMA-written
constexpr int kSmemKV = kSmemQ + 65536;            // 128 KB: 8 K-blocks x [128 tokens x 128 B]
constexpr int kSmemP = kSmemKV + 131072;           // 16 KB: P^T [128 tokens x 64 heads] bf16
constexpr int kSmemRing = kSmemP + 16384;          // [kRing] Tile
constexpr int kSmemScales = kSmemRing + kRing * 32;  // [kRing][128] scale rows of 8 bytes
constexpr int kSmemRed = kSmemScales + kRing * 1024;   // [4][64] f32: per-quadrant maxima or sums
constexpr int kSmemHeadM = kSmemRed + 1024;        // [64] m per head
constexpr int kSmemAlpha = kSmemHeadM + 256;       // [64] rescale factors; 1/L in the epilogue
constexpr int kSmemNegM = kSmemAlpha + 256;        // [64] -m per head
constexpr int kSmemScan = kSmemNegM + 256;        // block scan of the tile counts (a row per warp), the range's start
constexpr int kSmemBars = kSmemScan + 8 * (kThreads / 32 + 2);
enum Bar : int {
    kBarRingFull = 0,               // + slot
    kBarRingEmpty = kRing,          // + slot: dequant warps, softmax warps and the MMA thread are done with it
    kBarQ = 2 * kRing,              // Q of the current request landed
    kBarRope = kBarQ + 1,           // rope values of the tile landed
    kBarKvFull = kBarRope + 1,      // + i: the chunks of pair i written (8 warps)
    kBarKvFree = kBarKvFull + 2,    // + c: the PV of chunk c is done
    kBarS = kBarKvFree + 4,         // S^T of the tile complete
    kBarP = kBarS + 1,              // P^T written (8 warps)
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
constexpr uint32_t kTmemPark = 384;  // converted rows of the next tile, 32 columns a warp

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
__device__ __forceinline__ float *sm_neg_m() { return reinterpret_cast<float *>(g_smem + kSmemNegM); }
__device__ __forceinline__ float *sm_alpha() { return reinterpret_cast<float *>(g_smem + kSmemAlpha); }
__device__ __forceinline__ long long *sm_scan() { return reinterpret_cast<long long *>(g_smem + kSmemScan); }
__device__ __forceinline__ volatile int *sm_abort() { return reinterpret_cast<volatile int *>(g_smem + kSmemAbort); }

// Bounded wait on an mbarrier phase: false when the CTA has been aborted or the time is out
// (which aborts it and sets the error word).
__device__ __forceinline__ bool wait_slow(uint64_t *bar, uint32_t parity, const Params &p) {
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        if (mbar_try_wait_for(bar, parity, 1000000u)) return true;  // suspends for a bounded time
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
// Every lane waits; a uniform verdict.
__device__ __forceinline__ bool all_wait(int bar, uint32_t parity, const Params &p) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, p)) != 0;
}

// Number of tiles of request b.
__device__ __forceinline__ long long tiles_of(const Params &p, int b) {
    const int len = p.seq_lens[b];
    if (len <= 0) return 0;
    if (p.spans) return (p.nsel + 1) / 2;
    const long long n = min(static_cast<long long>(len), static_cast<long long>(p.max_blocks) * kPageTokens);
    return (n + kTile - 1) / kTile;
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
        j = p.spans[static_cast<size_t>(b) * p.nsel + slot];
    }
    if (j < 0 || j * kSpan >= len || j / (kPageTokens / kSpan) >= p.max_blocks) return;
    const int page = p.block_table[static_cast<size_t>(b) * p.max_blocks + j / (kPageTokens / kSpan)];
    if (page < 0 || page >= p.num_pages) {
        atomicOr(p.err, SMLA_FLAG_BAD_PAGE);
        return;
    }
    code = page * (kPageTokens / kSpan) + static_cast<int>(j % (kPageTokens / kSpan));
    count = static_cast<int>(min(static_cast<long long>(kSpan), len - j * kSpan));
}

// The tiles whose scale rows may still be on their way when the CTA is aborted, [from, to) in shared memory (the scan's,
// which is over): registers would be held by every warp of the kernel.
__device__ __forceinline__ void set_published(int from, int to, int lane) {
    if (lane == 0) reinterpret_cast<int2 *>(sm_scan())[0] = make_int2(max(0, from), to);
}
__device__ __forceinline__ void drain_published() {
    const int2 tiles = reinterpret_cast<const int2 *>(sm_scan())[0];
    for (int i = tiles.x; i < tiles.y; ++i) (void)mbar_wait(sm_bar(kBarRingFull + i % kRing), (i / kRing) & 1, kDrainNs);
}

__device__ __forceinline__ void walk(const Params &p, const Range &r, int lane) {
    long long left = r.end - r.begin;
    long long at = r.at;
    int k = 0;  // tiles published
    for (int b = r.b; left > 0; ++b, at = 0) {
        const long long total = tiles_of(p, b);
        const int len = p.seq_lens[b];
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
                if (!all_wait(kBarRingEmpty + k % kRing, ((k / kRing) & 1) ^ 1, p)) return set_published(k - kRing, k, lane);
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
                    // the scale rows come with the tile; the token rows head for L2 while the tiles
                    // before them are worked on
                    uint32_t bytes[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) bytes[u] = (count[u] * kScaleRowBytes + 15) & ~15;
                    mbar_arrive_expect_tx(sm_bar(kBarRingFull + k % kRing), bytes[0] + bytes[1]);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        if (code[u] < 0) continue;
                        bulk_load(smem_addr(g_smem + kSmemScales) + (k % kRing) * 1024 + u * 512,
                                  token_scales(p.cache, code[u] * kSpan), bytes[u], sm_bar(kBarRingFull + k % kRing));
                        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(token_row(p.cache, code[u] * kSpan)),
                                     "r"(count[u] * kRowBytes)
                                     : "memory");
                    }
                }
                __syncwarp();
            }
        }
    }
    if (!all_wait(kBarRingEmpty + k % kRing, ((k / kRing) & 1) ^ 1, p)) return set_published(k - kRing, k, lane);
    if (lane == 0) {
        sm_ring()[k % kRing].b = -1;
        mbar_arrive(sm_bar(kBarRingFull + k % kRing));
    }
    set_published(k - kRing + 1, k, lane);  // the end took the place of tile k - kRing, which was read
}

// ------------------------------------------------------------------ dequantisation
// Warpgroup c writes dims [128c, 128c + 128) of every tile: of c = 0..2 two nope groups, of c = 3
// the last nope group, and it has the rope values copied in.  Thread t (0..127) of it works on the token
// rows own + 32 j (j = 0..3, the first two in the first span) and the 32 bytes u = t & 3 of the chunk's
// 128; for c = 3 on 32 nope bytes of the two rows in span h = u >> 1.
//
// own: a store phase is 8 lanes with 16 bytes each; the four lanes of a row would hit each
// bank group twice (u and u + 2 write the same columns of two K-blocks), as would the next row's.
// Lanes with h = 1 therefore take the row of the other parity, and the second four lanes a
// row that differs in bits 0 and 1: 8 bank groups of the swizzled tile.
//
// One chunk per warpgroup and not all four in turn: a warp that converts a chunk with loads for the
// next just issued was measured to wait for those (12,500 cycles a tile).
struct Source {
    const uint8_t *row[2];  // first token row of each span
    uint32_t scales;        // shared memory: the spans' scale rows, 512 bytes each
    int count[2];
};

__device__ __forceinline__ int half_of(int t) { return (t >> 1) & 1; }
__device__ __forceinline__ int own_row(int t) {
    const int g = t >> 2;
    return (g & ~3) | (((g & 1) * 3) ^ ((g >> 1) & 1) ^ half_of(t));
}

__device__ __forceinline__ Source tile_source(const Params &p, int slot) {
    const Tile &t = sm_ring()[slot];
    Source s;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        s.row[u] = token_row(p.cache, max(0, t.code[u]) * kSpan);
        s.count[u] = t.count[u];
    }
    s.scales = smem_addr(g_smem + kSmemScales) + slot * (kTile * kScaleRowBytes);
    return s;
}

// 32 e4m3 bytes times 2^(s-127) -> 32 bf16 as four 16-byte units.  A byte sign-extended to 16 bits and
// moved up by 4 has its sign, exponent and mantissa in bf16's places (0x87F0) and reads there as
// the value times 2^-120, subnormals included; one multiplication by 2^(s-7) then gives the product
// exactly (see smla.h for its range).  Three integer operations for two values: their pipe is
// what bounds the conversion.  Above s = 134 that factor is no bf16, and a second one follows.
__device__ __forceinline__ void convert_nope(const Bytes32 &raw, uint32_t s, uint4 (&v)[4]) {
    const uint32_t m = (min(s, 134u) + 120u) * 0x00800080u;  // bf16 2^(s-7) in both halves
    const uint32_t w[8] = {raw.a.x, raw.a.y, raw.a.z, raw.a.w, raw.b.x, raw.b.y, raw.b.z, raw.b.w};
    uint32_t o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        uint32_t two;  // prmt selectors with bit 3 set repeat the byte's sign
        if (i & 1)
            asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(two) : "r"(w[i >> 1]));
        else
            asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(two) : "r"(w[i >> 1]));
        o[i] = bf16x2_mul((two << 4) & 0x87F087F0u, m);
    }
    if (s > 134u) {
        const uint32_t m2 = s == 255u ? 0x7FC07FC0u : (s - 7u) * 0x00800080u;  // NaN, or 2^(s-134)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = bf16x2_mul(o[i], m2);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
}
// Units 4n..4n+3 of the row at shared address `row`, whose swizzle is `sw`.
__device__ __forceinline__ void store_nope(uint32_t row, int n, int sw, const uint4 (&v)[4]) {
    const uint32_t first = row + (((4 * n) ^ sw) << 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) sts_v4(first ^ (q << 4), v[q]);
}

__device__ __forceinline__ Bytes32 load32(const uint8_t *src, bool valid) {
    if (valid) return ld_stream_v8(src);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    return Bytes32{zero, zero};
}

__device__ __forceinline__ uint32_t load_scale(const Source &s, int half, int tok, int g, bool valid) {
    uint32_t v = 0;
    if (valid)
        asm volatile("ld.shared.u8 %0, [%1];"
                     : "=r"(v)
                     : "r"(s.scales + half * (kSpan * kScaleRowBytes) + tok * kScaleRowBytes + g));
    return v;
}

// Dims chunks 0..2.  A tile is converted a tile ahead: right after the tile before it is stored,
// while the tensor core works through its scores (the conversions of 12 warps next to the softmax
// made that 900 cycles longer), and half of the converted rows wait in tensor memory (32 columns a
// warp), which leaves the registers for the loads of the tile after.  Between the release of a
// chunk and its hand-over there are only stores.
struct NopePart {
    Bytes32 raw[4];
    uint32_t scale[4];
    uint4 v[2][4];  // of rows j = 0, 1; those of j = 2, 3 are in tensor memory

    __device__ __forceinline__ void load(int c, int t, const Source &s) {
        const int own = own_row(t);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int tok = own + 32 * (j & 1);
            raw[j] = load32(s.row[j >> 1] + tok * kRowBytes + 128 * c + 32 * (t & 3), tok < s.count[j >> 1]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int tok = own + 32 * (j & 1);
            scale[j] = load_scale(s, j >> 1, tok, 2 * c + half_of(t), tok < s.count[j >> 1]);
        }
    }
    __device__ __forceinline__ void convert(uint32_t park) {
#pragma unroll
        for (int j = 0; j < 2; ++j) convert_nope(raw[2 + j], scale[2 + j], v[j]);
        tmem_st32(park, reinterpret_cast<const float *>(v));
#pragma unroll
        for (int j = 0; j < 2; ++j) convert_nope(raw[j], scale[j], v[j]);
        tmem_wait_st();
    }
    __device__ __forceinline__ void store(int c, int t, uint32_t park) {
        const int own = own_row(t);
        const uint32_t row = smem_addr(g_smem + kSmemKV) + (2 * c + half_of(t)) * (kTile * 128) + own * 128;
#pragma unroll
        for (int j = 0; j < 2; ++j) store_nope(row + 32 * 128 * j, t & 1, own & 7, v[j]);
        tmem_ld32(park, reinterpret_cast<float *>(v));
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 2; ++j) store_nope(row + 32 * 128 * (2 + j), t & 1, own & 7, v[j]);
    }
};

__device__ __forceinline__ void nope_role(const Params &p, uint32_t tmem, int c, int t, int q, int lane) {
    const uint32_t park = tmem + (static_cast<uint32_t>(32 * q) << 16) + kTmemPark + 32 * c;
    NopePart part;
    // loads tile k, if there is one: 1, none: 0, a wait failed: -1
    auto fetch = [&](int k) {
        if (!all_wait(kBarRingFull + k % kRing, (k / kRing) & 1, p)) return -1;
        if (sm_ring()[k % kRing].b < 0) return 0;
        part.load(c, t, tile_source(p, k % kRing));
        __syncwarp();
        if (lane == 0) mbar_arrive(sm_bar(kBarRingEmpty + k % kRing));
        return 1;
    };
    if (fetch(0) <= 0) return;
    part.convert(park);
    for (int k = 0;; ++k) {
        const int more = fetch(k + 1);
        if (more < 0) return;
        if (k > 0 && !all_wait(kBarKvFree + c, (k - 1) & 1, p)) return;
        part.store(c, t, park);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm_bar(kBarKvFull + pair_of(c)));
        if (!more) return;
        part.convert(park);
    }
}

// Dims chunk 3: the last nope group, loaded once the tile before is stored, and the rope values, which
// TMA puts in place once the PV of the tile before has released them.  A box is a span's 64 rows:
// those behind the span's count come along (they are inside the page) and are zeroed afterwards.
// Returns the number of tiles whose rope values it has asked for.
__device__ __forceinline__ uint32_t tail_role(const Params &p, const CUtensorMap *tmap_rope, int t, int lane) {
    const int own = own_row(t), h = half_of(t), sw = own & 7;
    const uint32_t kb6 = smem_addr(g_smem + kSmemKV) + 6 * (kTile * 128);
    Source s;
    int code[2];
    if (!all_wait(kBarRingFull, 0, p) || sm_ring()[0].b < 0) return 0;
    s = tile_source(p, 0);
    code[0] = sm_ring()[0].code[0];
    code[1] = sm_ring()[0].code[1];
    for (int k = 0;; ++k) {
        Bytes32 raw[2];
        uint32_t scale[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int tok = own + 32 * j;
            const bool valid = tok < (h ? s.count[1] : s.count[0]);
            raw[j] = load32((h ? s.row[1] : s.row[0]) + tok * kRowBytes + 384 + 32 * (t & 1), valid);
            scale[j] = load_scale(s, h, tok, 6, valid);
        }
        const int count[2] = {s.count[0], s.count[1]}, now[2] = {code[0], code[1]};
        __syncwarp();
        if (lane == 0) mbar_arrive(sm_bar(kBarRingEmpty + k % kRing));
        // the next tile's pages: what its loads need is in registers before this tile is stored
        if (!all_wait(kBarRingFull + (k + 1) % kRing, ((k + 1) / kRing) & 1, p)) return k;
        const Tile &next = sm_ring()[(k + 1) % kRing];
        const bool more = next.b >= 0;
        s = tile_source(p, (k + 1) % kRing);
        code[0] = next.code[0];
        code[1] = next.code[1];
        uint4 v[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) convert_nope(raw[j], scale[j], v[j]);
        if (k > 0 && !all_wait(kBarKvFree + 3, (k - 1) & 1, p)) return k;
        if (t == 0) {
            mbar_arrive_expect_tx(sm_bar(kBarRope), ((now[0] >= 0 ? 1u : 0u) + (now[1] >= 0 ? 1u : 0u)) * kSpan * 128u);
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (now[u] >= 0)
                    tma_load_3d(g_smem + kSmemKV + 7 * (kTile * 128) + u * (kSpan * 128), tmap_rope, kNope,
                                (now[u] & 3) * kSpan, now[u] >> 2, sm_bar(kBarRope));
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 2; ++j) store_nope(kb6 + (64 * h + 32 * j + own) * 128, t & 1, sw, v[j]);
        if (count[0] < kSpan || count[1] < kSpan) {  // uniform over the warpgroup
            if (!all_wait(kBarRope, k & 1, p)) return k + 1;
            if ((t & 63) >= ((t >> 6) ? count[1] : count[0]))
#pragma unroll
                for (int i = 0; i < 8; ++i) sts_v4(kb6 + kTile * 128 + t * 128 + 16 * i, make_uint4(0u, 0u, 0u, 0u));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm_bar(kBarKvFull + pair_of(3)));
        if (!more) return k + 1;
    }
}

// ------------------------------------------------------------------ MMA issue (one warp)
// The warp walks its loop converged, so that descriptors stay in uniform registers, and one
// elected lane issues: 50 cycles an MMA, 80 to 100 by one lane of divergent code.  Loops over the chunks
// are unrolled (rolled ones: 7 % more time for the whole kernel).
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t a_lo, uint32_t b_lo, bool accumulate) {
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {  // 16 tokens a step, 2 KB apart in the MN-major V^T and P^T
        const uint32_t o = ks * (2048 >> 4);
        mma_bf16_ss(d, desc_from(a_lo + o, kDescHi), desc_from(b_lo + o, kDescHi), kIdescPV,
                    (ks > 0 || accumulate) ? 1u : 0u);
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
    const bool leader = elect_one();
    bool spare_used = false, q_pending = false;
    int flags = 0, segments = 0;  // segments: Q loads issued
    bool ok = all_wait(kBarRingFull, 0, p) && sm_ring()[0].b >= 0;
    if (ok) {
        flags = sm_ring()[0].flags;
        if (leader) load_q(tmap_q, sm_ring()[0].b);
        __syncwarp();
        if (leader) mbar_arrive(sm_bar(kBarRingEmpty));
        segments = 1;
        q_pending = true;
    }
    for (int k = 0; ok; ++k) {
        const uint32_t par = k & 1;
        if (flags & kFirst) {
            ok = all_wait(kBarQ, (segments - 1) & 1, p);
            if (!ok) break;
            q_pending = false;
        }
        // two chunks at a time, with one barrier for both: a look at a barrier takes hundreds of cycles while
        // MMAs run, more than the MMAs that are queued by then (single chunks, or 1 + 2 + 1: 4 % slower)
#pragma unroll
        for (int i = 0; i < kChunks; i += 2) {
            ok = (i > 0 || all_wait(kBarRope, par, p)) && all_wait(kBarKvFull + i / 2, par, p);
            if (!ok) break;
            tc_fence_after_sync();
            if (leader) {
#pragma unroll
                for (int j = i; j < i + 2; ++j) {
                    const int e = chunk_at(j);
                    issue_qk_chunk(tmem + kTmemS, qk_a + e * 2 * ((kTile * 128) >> 4), qk_b + e * 2 * (8192 >> 4), j == 0);
                }
            }
            __syncwarp();
        }
        if (!ok) break;
        const bool hook = k == 0 && (p.debug_flags & SMLA_DEBUG_SKIP_FIRST_COMMIT);
        if (leader) mma_commit(sm_bar(hook ? kBarSpare : kBarS));
        __syncwarp();
        spare_used = spare_used || hook;
        // the next tile; a new request's Q is fetched as soon as this tile's scores are done
        ok = all_wait(kBarRingFull + (k + 1) % kRing, ((k + 1) / kRing) & 1, p);
        if (!ok) break;
        const int next_b = sm_ring()[(k + 1) % kRing].b, next_flags = sm_ring()[(k + 1) % kRing].flags;
        __syncwarp();
        if (leader) mbar_arrive(sm_bar(kBarRingEmpty + (k + 1) % kRing));
        if (next_b >= 0 && (next_flags & kFirst)) {
            ok = all_wait(kBarS, par, p);
            if (!ok) break;
            if (leader) load_q(tmap_q, next_b);
            ++segments;
            q_pending = true;
        }
        ok = all_wait(kBarP, par, p);
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = chunk_at(i);
            if (leader) {
                issue_pv(tmem + 64 * c, pv_a + c * 2 * ((kTile * 128) >> 4), pv_b, !(flags & kFirst));
                mma_commit(sm_bar(kBarKvFree + c));
            }
            __syncwarp();
        }
        if (next_b < 0) break;
        flags = next_flags;
    }
    // every MMA and copy issued must be complete before tensor and shared memory are released
    if (leader) {
        if (spare_used) (void)mbar_wait(sm_bar(kBarSpare), 0, kDrainNs);
        if (q_pending) (void)mbar_wait(sm_bar(kBarQ), (segments - 1) & 1, kDrainNs);
        mma_commit(sm_bar(kBarDrain));
        (void)mbar_wait(sm_bar(kBarDrain), 0, kDrainNs);
    }
    __syncwarp();
}

// ------------------------------------------------------------------ softmax and epilogue
// Warp (q, hf) of the 8 owns tensor-memory lanes 32q.. (tokens of S^T, dims of an O^T chunk) and
// heads 32 hf...  Verdicts that the 8 warps must share go through their named barrier.

// Raises the references to the tile's maxima and rescales what was accumulated by
// 2^(m_old - m_new): on a segment's first tile, and when a score passes m by more than
// kRescaleThreshold.
__device__ __forceinline__ void raise_max(const Params &p, uint32_t tmem_lane, int q, int hf, int lane, bool valid,
                                          bool first) {
    {
        float y[32];
        tmem_ld32(tmem_lane + kTmemS + 32 * hf, y);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 32; ++h) y[h] = valid ? y[h] * p.scale_log2 : -INFINITY;
        sm_red()[q * 64 + 32 * hf + lane] = warp_transpose_reduce<true, 32>(y, lane);
    }
    named_barrier_sync(kBarIdSoftmax, kSoftmaxThreads);
    if (q == 0) {
        const int t = 32 * hf + lane;
        const float *red = sm_red();
        const float tm = fmaxf(fmaxf(red[t], red[64 + t]), fmaxf(red[128 + t], red[192 + t]));
        const float mo = first ? -INFINITY : sm_head_m()[t];
        const float mn = fmaxf(mo, tm);
        sm_alpha()[t] = (mo == -INFINITY) ? 0.0f : exp2f(mo - mn);
        sm_head_m()[t] = mn;
        // no score above -inf yet: one that is -inf itself has to give 2^-inf and not 2^NaN, any other to raise m
        sm_neg_m()[t] = mn == -INFINITY ? FLT_MAX : -mn;
    }
    named_barrier_sync(kBarIdSoftmax, kSoftmaxThreads);
    if (first) return;  // nothing accumulated yet
    // the PV of the tile before is complete: the commit of this tile's scores covers it
#pragma unroll 1
    for (int g = 0; g < 10; ++g) {  // 16 columns at a time: the four chunks of O^T, then L
        const uint32_t col = tmem_lane + 64 * (g >> 1) + 32 * hf + 16 * (g & 1) + (g < 8 ? 0u : kTmemL - 256u);
        float al[16], o[16];
        load16(sm_alpha() + 32 * hf + 16 * (g & 1), al);
        tmem_ld16(col, o);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 16; ++h) o[h] *= al[h];
        tmem_st16(col, o);
    }
    tmem_wait_st();
}

// L per head over the 128 lanes -> 1/L, and the segment's log-sum-exps.
__device__ __forceinline__ void finish_sums(const Params &p, uint32_t tmem_lane, int q, int hf, int lane, int b,
                                            int part) {
    {
        float y[32];
        tmem_ld32(tmem_lane + kTmemL + 32 * hf, y);
        tmem_wait_ld();
        sm_red()[q * 64 + 32 * hf + lane] = warp_transpose_reduce<false, 32>(y, lane);
    }
    named_barrier_sync(kBarIdSoftmax, kSoftmaxThreads);
    if (q == 0) {
        const int t = 32 * hf + lane;
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

// O^T / L: dim 128c + 32q + lane of this warp's heads; a warp's stores of a head are contiguous.
__device__ __forceinline__ void write_out(const Params &p, uint32_t tmem_lane, int q, int hf, int lane, int b,
                                          int part) {
    const size_t first = static_cast<size_t>(part >= 0 ? part : b) * kHeads * kDim + 32 * q + lane;
#pragma unroll 1
    for (int g = 0; g < 8; ++g) {  // dims chunk g / 2, heads 32 hf + 16 (g % 2)..
        const int h0 = 32 * hf + 16 * (g & 1);
        float o[16], inv[16];
        tmem_ld16(tmem_lane + 64 * (g >> 1) + h0, o);
        load16(sm_alpha() + h0, inv);
        tmem_wait_ld();
        const size_t at = first + 128 * (g >> 1) + static_cast<size_t>(h0) * kDim;
        if (part >= 0) {
#pragma unroll
            for (int h = 0; h < 16; ++h) p.part_o[at + h * kDim] = o[h] * inv[h];
        } else {
#pragma unroll
            for (int h = 0; h < 16; ++h) p.out[at + h * kDim] = static_cast<uint16_t>(pack_bf16x2(o[h] * inv[h], 0.0f));
        }
    }
}

// (three inputs to a maximum and two products an instruction: 1 % of the kernel's time)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// (a, b) = (a, b) * c + (x, y)
__device__ __forceinline__ void fma2(float &a, float &b, float c, float x, float y) {
    asm("{\n.reg .b64 u, v, w;\nmov.b64 u, {%0, %1};\nmov.b64 v, {%2, %2};\nmov.b64 w, {%3, %4};\nfma.rn.f32x2 u, u, v, w;\nmov.b64 {%0, %1}, u;\n}"
        : "+f"(a), "+f"(b) : "f"(c), "f"(x), "f"(y));
}
// Scores of this warp's heads in log2 units less the references (-inf for a masked token) and
// their maximum.
__device__ __forceinline__ float load_scores(uint32_t lane_addr, int hf, float c, bool whole, bool valid,
                                             float (&x)[32]) {
    tmem_ld32(lane_addr + kTmemS + 32 * hf, x);
    tmem_wait_ld();
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        const float4 m = reinterpret_cast<const float4 *>(sm_neg_m() + 32 * hf)[g];
        fma2(x[4 * g], x[4 * g + 1], c, m.x, m.y);
        fma2(x[4 * g + 2], x[4 * g + 3], c, m.z, m.w);
    }
    if (!whole) {  // a tile with masked tokens: uniform over the warps
#pragma unroll
        for (int h = 0; h < 32; ++h) x[h] = valid ? x[h] : -INFINITY;
    }
    float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int h = 4; h < 28; h += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = max3(top[i], x[h + 2 * i], x[h + 2 * i + 1]);
    return max3(max3(top[0], top[1], x[28]), max3(top[2], top[3], x[29]), fmaxf(x[30], x[31]));
}

__device__ __forceinline__ void softmax_role(const Params &p, uint32_t tmem, int q, int hf, int lane) {
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const int r = 32 * q + lane;  // token row
    const uint32_t prow = smem_addr(g_smem + kSmemP) + r * 128;
    for (int k = 0;; ++k) {
        const uint32_t par = k & 1;
        bool ok = all_wait(kBarRingFull + k % kRing, (k / kRing) & 1, p);
        const Tile tile = sm_ring()[k % kRing];
        const bool done = ok && tile.b < 0;  // leaves through the barriers below: another warp's wait may have failed
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(sm_bar(kBarRingEmpty + k % kRing));
        const bool first = tile.flags & kFirst;
        const bool whole = tile.count[0] == kSpan && tile.count[1] == kSpan;
        const bool valid = (r & 63) < ((r >> 6) ? tile.count[1] : tile.count[0]);
        ok = ok && !done && all_wait(kBarS, par, p);
        tc_fence_after_sync();
        // the weights before the verdict on the references (3 % less time than after it): those of a tile that
        // passes them are computed again
        float x[32];
#pragma unroll
        for (int h = 0; h < 32; ++h) x[h] = 0.0f;
        bool over = first || !ok;
        if (!over) over = load_scores(lane_addr, hf, p.scale_log2, whole, valid, x) > kRescaleThreshold;
#pragma unroll
        for (int h = 0; h < 32; ++h) x[h] = fast_exp2(x[h]);
        if (barrier_or(kBarIdSoftmax, kSoftmaxThreads, over)) {
            if (barrier_or(kBarIdSoftmax, kSoftmaxThreads, !ok)) return;
            raise_max(p, lane_addr, q, hf, lane, valid, first);
            (void)load_scores(lane_addr, hf, p.scale_log2, whole, valid, x);
#pragma unroll
            for (int h = 0; h < 32; ++h) x[h] = fast_exp2(x[h]);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g)
            sts_v4(prow + (((4 * hf + g) ^ (r & 7)) << 4),
                   make_uint4(pack_bf16x2(x[8 * g], x[8 * g + 1]), pack_bf16x2(x[8 * g + 2], x[8 * g + 3]),
                              pack_bf16x2(x[8 * g + 4], x[8 * g + 5]), pack_bf16x2(x[8 * g + 6], x[8 * g + 7])));
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm_bar(kBarP));
        // L += p, after the hand-over: the PV does not read it
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const uint32_t col = lane_addr + kTmemL + 32 * hf + 16 * g;
            if (!first) {
                float l[16];
                tmem_ld16(col, l);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < 16; ++h) x[16 * g + h] += l[h];
            }
            tmem_st16(col, x + 16 * g);
        }
        tmem_wait_st();
        if (tile.flags & kLast) {
            ok = all_wait(kBarKvFree + chunk_at(3), par, p);  // commits complete in order: every chunk of O^T is final
            if (barrier_or(kBarIdSoftmax, kSoftmaxThreads, !ok)) return;
            tc_fence_after_sync();
            finish_sums(p, lane_addr, q, hf, lane, tile.b, tile.part);
            write_out(p, lane_addr, q, hf, lane, tile.b, tile.part);
            tc_fence_before_sync();
        }
    }
}

template <int kRegs>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__global__ void __launch_bounds__(kThreads, 1)
    span_decode_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_rope) {
    // Launched while the kernel before it drains (2 us a call).  No load in here is of the read-only kind, which
    // holds only for data older than the kernel's launch.
    wait_for_prior_kernel();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // The tiles need a 1024-byte aligned base (128-byte swizzle); the base is the same for every
    // CTA of a launch.
    const bool misplaced = (smem_addr(g_smem) & 1023u) != 0;
    const Range range = find_range<kThreads>([&](int b) { return tiles_of(p, b); }, p.B, sm_scan(), p.prefix);
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
        mbar_init(sm_bar(kBarRope), 1);
        for (int c = 0; c < 4; ++c) {
            if (c < 2) mbar_init(sm_bar(kBarKvFull + c), kDequantWarps / 2);
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
        if (warp < kDequantWarps - 4) {
            more_registers<kRegsNope>();
            nope_role(p, tmem, warp >> 2, tid & 127, warp & 3, lane);
        } else {
            more_registers<kRegsTail>();
            const uint32_t copies = tail_role(p, &tmap_rope, tid & 127, lane);
            if (tid == 32 * (kDequantWarps - 4) && copies)  // the last copy asked for
                (void)mbar_wait(sm_bar(kBarRope), (copies - 1) & 1, kDrainNs);
            __syncwarp();
        }
    } else if (warp < kMmaWarp) {
        softmax_role(p, tmem, warp & 3, (warp - kDequantWarps) >> 2, lane);
    } else {
        fewer_registers<kRegsControl>();
        if (warp == kMmaWarp)
            mma_role(p, &tmap_q, tmem);
        else if (warp == kWalkWarp)
            walk(p, range, lane);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
    // of an aborted CTA, nobody else has waited for the scale rows
    if (warp == kWalkWarp && lane == 0 && *sm_abort()) drain_published();
    if (tid == 0) p.failed[blockIdx.x] = *sm_abort();
}

// ------------------------------------------------------------------ the join
// One warp per (request, head); blockIdx.x is the request and kJoinWarps heads.  Zeros and -inf for
// a request without tiles, NaN where a CTA gave up, nothing for a request that one CTA wrote
// whole, and otherwise the parts, in the order of the CTAs, with weights 2^(lambda - max).
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Params p, int grid) {
    wait_for_prior_kernel();
    const int b = blockIdx.x / (kHeads / kJoinWarps);
    const int h = blockIdx.x % (kHeads / kJoinWarps) * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const long long begin = p.prefix[b], n = p.prefix[b + 1] - begin, total = p.prefix[p.B];
    const long long per = max(1ll, (total + grid - 1) / grid);
    const int c0 = static_cast<int>(begin / per), c1 = n > 0 ? static_cast<int>((begin + n - 1) / per) : c0 - 1;
    // part c of the request: lane c - c0 - 32 i looks at it
    auto index = [&](int c) { return static_cast<size_t>(2 * c + (c == c0 && begin > c * per ? 1 : 0)) * kHeads + h; };
    bool bad = false;
    float top = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) {
        bad |= p.failed[c] != 0;
        const float v = c0 < c1 ? p.part_lambda[index(c)] : 0.0f;
        bad |= isnan(v);
        top = fmaxf(top, v);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (c0 == c1 && !bad) return;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = bad ? NAN : 0.0f;
    float sum = 0.0f;
    if (!bad && top != -INFINITY) {
#pragma unroll 2
        for (int c = c0; c <= c1; ++c) {
            const size_t at = index(c);
            const float4 *src = reinterpret_cast<const float4 *>(p.part_o + at * kDim) + lane;
            float4 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = src[32 * i];
            const float w = exp2f(p.part_lambda[at] - top);
            sum += w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[4 * i] += w * o[i].x;
                x[4 * i + 1] += w * o[i].y;
                x[4 * i + 2] += w * o[i].z;
                x[4 * i + 3] += w * o[i].w;
            }
        }
        const float inv = 1.0f / sum;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= inv;
    }
    uint2 *dst = reinterpret_cast<uint2 *>(p.out + (static_cast<size_t>(b) * kHeads + h) * kDim) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        dst[32 * i] = make_uint2(pack_bf16x2(x[4 * i], x[4 * i + 1]), pack_bf16x2(x[4 * i + 2], x[4 * i + 3]));
    if (lane == 0)
        p.lse[static_cast<size_t>(b) * kHeads + h] =
            bad ? NAN : top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
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

// The cache as [num_pages][256][576] bytes; boxes of a span's 64 rows x 128 bytes.
int encode_cache_map(CUtensorMap *map, const uint8_t *cache, int num_pages) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    const int rc = smla::host::tensor_map_encoder(fn);
    if (rc != SMLA_OK) return rc;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(smla::kRowBytes), static_cast<cuuint64_t>(smla::kPageTokens),
                          static_cast<cuuint64_t>(num_pages)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(smla::kRowBytes), static_cast<cuuint64_t>(smla::kPageBytes)};
    cuuint32_t box[3] = {128, kSpan, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(cache), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SMLA_OK : SMLA_ERR_INVALID;
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
    if (!aligned(q, 16) || !aligned(kv_cache, 32) || !aligned(out, 16) || !aligned(workspace, 256) ||
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
    alignas(64) CUtensorMap tmap_q, tmap_rope;
    rc = smla::host::encode_q_map(&tmap_q, q, B);
    if (rc == SMLA_OK) rc = encode_cache_map(&tmap_rope, kv_cache, num_pages);
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
    if (smla::host::launch_after(span_decode_kernel, dim3(static_cast<unsigned>(sms)), kThreads, kSmemBytes, st, p, tmap_q, tmap_rope) !=
        cudaSuccess)
        return SMLA_ERR_LAUNCH;
    // launched while the first kernel drains: 2 to 3 us a call
    const dim3 grid(static_cast<unsigned>(B) * (SMLA_HEADS / kJoinWarps));
    if (smla::host::launch_after(join_kernel, grid, 32 * kJoinWarps, 0, st, p, sms) != cudaSuccess) return SMLA_ERR_LAUNCH;
    return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

}  // extern "C"
