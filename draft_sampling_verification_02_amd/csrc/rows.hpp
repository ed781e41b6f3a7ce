// rows.hpp -- packed rows and where they go: the request of a row, its position,
// its slot of a paged cache, and the scale of an 8-bit row (cache.hip,
// rotary.hip).
#pragma once

#include "attend.hpp"
#include "internal.hpp"

namespace dspark {

constexpr int kCacheThreads = 256;  // of a workgroup

struct RowPlace {
    long long slot;  // (page * Hkv * page_size + offset in the page), -1: none
    long long pos;   // position of the row, -1: its request takes no part
    int inside;      // the row belongs to a request
};

// The requests of rows r0 and r1 (r0 <= r1): how many requests end at or
// before each row.  Workgroup-wide; red holds two words a wave.
__device__ __forceinline__ void find_requests(const int32_t *off, int B, int r0, int r1, int *red, int &b0, int &b1) {
    int c0 = 0, c1 = 0;
    for (int b = threadIdx.x; b < B; b += kCacheThreads) {
        const int end = off[b + 1];
        c0 += end <= r0;
        c1 += end <= r1;
    }
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) {
        c0 += __shfl_xor(c0, s);
        c1 += __shfl_xor(c1, s);
    }
    if ((threadIdx.x & 63) == 0) {
        red[threadIdx.x >> 6] = c0;
        red[4 + (threadIdx.x >> 6)] = c1;
    }
    __syncthreads();
    b0 = red[0] + red[1] + red[2] + red[3];
    b1 = red[4] + red[5] + red[6] + red[7];
}

// Where row r lies, its request being one of b0 .. b1.
__device__ __forceinline__ RowPlace place_row(const CacheArgs &a, int pshift, int r, int b0, int b1) {
    RowPlace p{-1, -1, 0};
    int b = r, first = r;
    if (a.row_offsets) {
        int lo = b0, hi = b1;  // the first request in [b0, b1] that ends past r (b1 at the latest)
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.row_offsets[mid + 1] <= r)
                lo = mid + 1;
            else
                hi = mid;
        }
        b = lo;
        if (b >= a.B) return p;
        // clamped as everywhere (its end needs no clamp: r is a row of the call)
        first = max(a.row_offsets[b], 0);
        if (first > r) return p;
    }
    if (b < 0 || b >= a.B) return p;
    p.inside = 1;
    const int start = a.start ? a.start[b] : 0;
    if (start < 0) return p;  // the request takes no part
    const long long pos = (long long)start + (r - first);
    p.pos = pos;
    const long long pi = pos >> pshift;
    if (pi >= a.max_pages) return p;
    const int page = a.page_table[(long long)b * a.max_pages + pi];
    if (page < 0 || page >= a.n_pages) return p;
    p.slot = (((long long)page * a.n_kv_heads) << pshift) + (pos & ((1 << pshift) - 1));
    return p;
}

// exponent e of the scale: the smallest e >= -126 with amax <= 448 2^e
// (448 = 1.75 * 2^8)
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int ex = int(u >> 23) - 127;  // amax = 1.f * 2^ex (subnormal values: ex = -127, clamped below)
    const int e = ex - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < -126 ? -126 : e;
}

}  // namespace dspark
