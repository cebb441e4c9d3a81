// smla_range.cuh -- work split of the persistent kernels: the tiles of all requests as one sequence,
// cut into equal contiguous ranges, one per CTA, by lengths that only the device knows.
#pragma once

#include <cstdint>

namespace smla {

// A CTA's range of tiles [begin, end) and where it begins.
struct Range {
    long long begin, end, per;
    int b;         // request of tile `begin`
    long long at;  // its first tile's index inside that request
};

// Called by every thread of the CTA.  tiles_of(b) is the number of tiles of request b < B; the counts are
// scanned over the block (scan: kThreads / 32 + 2 entries of shared memory).  CTA 0 writes
// the sums before each request to prefix[0..B] (if not null) for a kernel that follows.
template <int kThreads, class Tiles>
__device__ __forceinline__ Range find_range(Tiles tiles_of, int B, long long *scan, long long *prefix) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (B + kThreads - 1) / kThreads;
    const int b0 = min(B, tid * each), b1 = min(B, b0 + each);
    // with one request a thread (B <= kThreads) its length is read once
    const long long head = b0 < b1 ? tiles_of(b0) : 0;
    long long mine = head;
    for (int b = b0 + 1; b < b1; ++b) mine += tiles_of(b);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
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
        for (long long n = head; r.begin >= at + n; n = tiles_of(++b)) at += n;
        scan[kThreads / 32] = b;
        scan[kThreads / 32 + 1] = r.begin - at;
    }
    if (prefix && blockIdx.x == 0) {
        long long at = before;
        for (int b = b0; b < b1; ++b) {
            prefix[b] = at;
            if (b + 1 < b1) at += b == b0 ? head : tiles_of(b);
        }
        if (tid == 0) prefix[B] = total;
    }
    __syncthreads();
    r.b = r.begin < r.end ? static_cast<int>(scan[kThreads / 32]) : B;
    r.at = r.begin < r.end ? scan[kThreads / 32 + 1] : 0;
    return r;
}

}  // namespace smla
