// cache.hip -- rows into the paged key-value cache (kv_write) and back out
// (kv_read).
//
// A cache is [n_pages, Hkv, page_size, D]: the tokens of a page that belong to
// one head are one contiguous run, which is what the attention streams.  Row i
// of request b stands at position pos = start_b + i, in page
// page_table[b][pos / page_size], slot pos % page_size.  In an 8-bit cache the
// D values of one (token, head) are x 2^-e rounded to e4m3 (to nearest, ties to
// even: off by at most 2^-4 of the value, or by 2^-10 2^e below 2^-6 2^e, where
// the steps are 2^-9 2^e), e the smallest integer >= -126 with max|x| <= 448 2^e.
// A power of two moves only exponents: the scaling is exact, so the value's own
// rounding is the only one, and a scale is one byte (e + 127).
//
// Both kernels are bound by memory: every row is read once and written once.
// A work item is 16 bytes of the 16-bit side (8 values); a workgroup takes a
// contiguous run of items in (row, K or V, head, chunk) order, finds the
// requests its rows belong to, and writes whole 128- or 256-byte runs.  (Items
// ordered by head over 16 rows, for 2-4 KiB runs in the cache, measured the
// same.)  Many rows take four items a thread, so that a wave has enough loads
// in flight; few rows one, for the shorter chain.
//
// Measured (MI355X, 8 heads, D = 128): 37,700 prompt rows into 8 bits 51 us
// (232 MB, 4.6 TB/s; a large copy reaches 4.7), into bfloat16 60 us (309 MB,
// 5.1 TB/s); 167,000 rows read back 267 us (1.37 GB, 5.1 TB/s); 64 single rows
// 3 us, the verify rows of 256 requests into 8 bits 5 us.
#include "attend.hpp"
#include "dspark.h"
#include "internal.hpp"

namespace dspark {

namespace {

constexpr int kCacheThreads = 256;
constexpr int kCacheItems = 4;  // items of a thread when there are many

struct CacheParams {
    CacheArgs a;
    long long items;  // 2 * n_rows * Hkv * (D / 8)
    int per_row;      // 2 * Hkv * (D / 8)
    int C, cshift;    // D / 8 and its logarithm
    int pshift;
    int per_block;    // items of a workgroup
};

struct RowPlace {
    long long slot;  // (page * Hkv * page_size + offset in the page), -1: none
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
    RowPlace p{-1, 0};
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
    const long long pi = pos >> pshift;
    if (pi >= a.max_pages) return p;
    const int page = a.page_table[(long long)b * a.max_pages + pi];
    if (page < 0 || page >= a.n_pages) return p;
    p.slot = (((long long)page * a.n_kv_heads) << pshift) + (pos & ((1 << pshift) - 1));
    return p;
}

constexpr int kMaxRowsPerBlock = kCacheThreads * kCacheItems / 16 + 2;  // a row has at least 2 * 1 * 8 items

// exponent e of the scale: the smallest e >= -126 with amax <= 448 2^e
// (448 = 1.75 * 2^8)
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int ex = int(u >> 23) - 127;  // amax = 1.f * 2^ex (subnormal values: ex = -127, clamped below)
    const int e = ex - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < -126 ? -126 : e;
}

// Maximum over the C neighbouring lanes (8, 16 or 32; items in order) that hold
// one (row, head).
__device__ __forceinline__ uint32_t group_max(uint32_t u, int C) {
    u = max(u, uint32_t(__builtin_amdgcn_mov_dpp(int(u), 0xB1, 0xF, 0xF, true)));   // lanes l ^ 1
    u = max(u, uint32_t(__builtin_amdgcn_mov_dpp(int(u), 0x4E, 0xF, 0xF, true)));   // l ^ 2
    u = max(u, uint32_t(__builtin_amdgcn_mov_dpp(int(u), 0x141, 0xF, 0xF, true)));  // the eight lanes mirrored
    if (C >= 16) u = max(u, uint32_t(__builtin_amdgcn_mov_dpp(int(u), 0x140, 0xF, 0xF, true)));  // the sixteen
    if (C >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        u = max(uint32_t(r[0]), uint32_t(r[1]));
    }
    return u;
}

// Two pairs of 16-bit floats, divided by a power of two, as four e4m3 values
// (none of them past 448).
template <typename T>
__device__ __forceinline__ int to_e4m3(uint32_t a, uint32_t b, float scale) {
    typedef short s16x2_t __attribute__((ext_vector_type(2)));
    s16x2_t r = {0, 0};
    if constexpr (std::is_same<T, TypeBf16>::value) {
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, a), scale, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, b), scale, true);
    } else {
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(f16x2_t, a), scale, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(f16x2_t, b), scale, true);
    }
    return __builtin_bit_cast(int, r);
}

struct Item {
    int row, head, chunk;  // row relative to the workgroup's first
    bool v;
};
// item `rel` counted from the first item of the workgroup's first row
__device__ __forceinline__ Item item_of(const CacheParams &p, int rel) {
    Item r;
    r.row = unsigned(rel) / unsigned(p.per_row);
    int rest = rel - r.row * p.per_row;
    r.chunk = rest & (p.C - 1);
    rest >>= p.cshift;
    r.v = rest >= p.a.n_kv_heads;
    r.head = r.v ? rest - p.a.n_kv_heads : rest;
    return r;
}

// The workgroup's items: `count` of them, from item rel0 of its first row.
struct Run {
    int row0, row1, rel0, count;
};
__device__ __forceinline__ Run run_of(const CacheParams &p) {
    const long long it0 = (long long)blockIdx.x * p.per_block;
    Run r;
    r.count = int(min((long long)p.per_block, p.items - it0));
    r.row0 = int(it0 / p.per_row);
    r.rel0 = int(it0 - (long long)r.row0 * p.per_row);
    r.row1 = r.row0 + unsigned(r.rel0 + r.count - 1) / unsigned(p.per_row);
    return r;
}

// The places of rows row0 .. row1, in LDS.
__device__ __forceinline__ void place_rows(const CacheParams &p, int row0, int row1, long long *slots, int *inside,
                                           int *red) {
    int b0 = 0, b1 = 0;
    if (p.a.row_offsets) find_requests(p.a.row_offsets, p.a.B, row0, row1, red, b0, b1);
    for (int t = threadIdx.x; t <= row1 - row0; t += kCacheThreads) {
        const RowPlace pl = place_row(p.a, p.pshift, row0 + t, b0, b1);
        slots[t] = pl.slot;
        if (inside) inside[t] = pl.inside;
    }
    __syncthreads();
}

template <typename T, bool E4, int ITEMS>
__global__ __launch_bounds__(kCacheThreads) void kv_write_kernel(CacheParams p) {
    __shared__ long long slots[kMaxRowsPerBlock];
    __shared__ int red[8];
    const CacheArgs &a = p.a;
    const Run run = run_of(p);
    const int row0 = run.row0;
    // the rows go out first: their addresses need no request
    Item im[ITEMS];
    u32x4v_t x[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        im[j] = item_of(p, run.rel0 + min(int(threadIdx.x) + j * kCacheThreads, run.count - 1));
        const uint8_t *src = static_cast<const uint8_t *>(im[j].v ? a.v : a.k);
        const long long stride = im[j].v ? a.v_stride : a.k_stride;
        // read once: non-temporal (measured with the row's conversion at 37,700 rows
        // of 8 heads, D = 128, into 8 bits: 58 us against 65)
        x[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4v_t *>(
            src + 2 * ((row0 + im[j].row) * stride + ((long long)im[j].head * p.C + im[j].chunk) * 8)));
    }
    place_rows(p, row0, run.row1, slots, nullptr, red);
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const bool live = int(threadIdx.x) + j * kCacheThreads < run.count;
        const long long slot = slots[im[j].row];
        const long long rowat = slot + ((long long)im[j].head << p.pshift);  // row of the cache, D values each
        uint8_t *cache = static_cast<uint8_t *>(im[j].v ? a.v_cache : a.k_cache);
        if constexpr (!E4) {
            if (live && slot >= 0) *reinterpret_cast<u32x4v_t *>(cache + (rowat * p.C + im[j].chunk) * 16) = x[j];
        } else {
            // magnitudes of 16-bit floats order as their bits do
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max_u16x2(top, x[j][i] & 0x7fff7fffu);
            top = max(top & 0xffffu, top >> 16);
            const bool odd = __any(top >= T::kInf);
            if (odd) {
                // infinities or NaN: the scale is that of the finite values
                top = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) top = max_u16x2(top, finite_pair<T>(x[j][i]) & 0x7fff7fffu);
                top = max(top & 0xffffu, top >> 16);
            }
            const int e = scale_exponent(widen<T>(group_max(top, p.C)).x);
            int lo, hi;
            if (!odd) {
                const float scale = __uint_as_float(uint32_t(e + 127) << 23);  // e in -126 .. 120
                lo = to_e4m3<T>(x[j][0], x[j][1], scale);
                hi = to_e4m3<T>(x[j][2], x[j][3], scale);
            } else {
                const float inv = __uint_as_float(uint32_t(127 - e) << 23);
                float f[8];
                widen4<T>(u32x2_t{x[j][0], x[j][1]}, f);
                widen4<T>(u32x2_t{x[j][2], x[j][3]}, f + 4);
                lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * inv, f[1] * inv, 0, false);
                lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * inv, f[3] * inv, lo, true);
                hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4] * inv, f[5] * inv, 0, false);
                hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6] * inv, f[7] * inv, hi, true);
            }
            if (live && slot >= 0) {
                *reinterpret_cast<int2 *>(cache + (rowat * p.C + im[j].chunk) * 8) = make_int2(lo, hi);
                if (im[j].chunk == 0) (im[j].v ? a.v_scale : a.k_scale)[rowat] = uint8_t(e + 127);
            }
        }
    }
}

// finite values past the type's largest become the largest (an amax just below
// it may round up to the next power of two)
template <typename T>
__device__ __forceinline__ uint32_t narrow2(float x, float y) {
    constexpr bool bf = std::is_same<T, TypeBf16>::value;
    const float top = bf ? __uint_as_float(0x7f7f0000u) : 65504.f;
    x = x > top ? top : (x < -top ? -top : x);
    y = y > top ? top : (y < -top ? -top : y);
    if constexpr (bf)
        return __builtin_bit_cast(uint32_t, bf16x2_t{__bf16(x), __bf16(y)});
    else
        return __builtin_bit_cast(uint32_t, f16x2_t{_Float16(x), _Float16(y)});
}

template <typename T, bool E4, int ITEMS>
__global__ __launch_bounds__(kCacheThreads, 8) void kv_read_kernel(CacheParams p) {
    __shared__ long long slots[kMaxRowsPerBlock];
    __shared__ int inside[kMaxRowsPerBlock];
    __shared__ int red[8];
    const CacheArgs &a = p.a;
    const Run run = run_of(p);
    const int row0 = run.row0;
    place_rows(p, row0, run.row1, slots, inside, red);
    Item im[ITEMS];
    u32x4v_t x[ITEMS];
    float sc[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        im[j] = item_of(p, run.rel0 + min(int(threadIdx.x) + j * kCacheThreads, run.count - 1));
        const long long slot = slots[im[j].row];
        const long long rowat = max(slot, 0LL) + ((long long)im[j].head << p.pshift);
        const uint8_t *cache = static_cast<const uint8_t *>(im[j].v ? a.v_cache : a.k_cache);
        x[j] = u32x4v_t{0, 0, 0, 0};
        sc[j] = 0.f;
        if (slot < 0) continue;
        if constexpr (E4) {
            const u32x2_t t = *reinterpret_cast<const u32x2_t *>(cache + (rowat * p.C + im[j].chunk) * 8);
            x[j][0] = t[0];
            x[j][1] = t[1];
            sc[j] = scale_of((im[j].v ? a.v_scale : a.k_scale)[rowat]);
        } else {
            x[j] = *reinterpret_cast<const u32x4v_t *>(cache + (rowat * p.C + im[j].chunk) * 16);
        }
    }
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        if (int(threadIdx.x) + j * kCacheThreads >= run.count || !inside[im[j].row]) continue;
        u32x4v_t o = x[j];
        if constexpr (E4) {
            float f[8];
            e4m3_to4(x[j][0], f);
            e4m3_to4(x[j][1], f + 4);
            const bool none = slots[im[j].row] < 0;  // zeros, whatever the scale
            o[0] = none ? 0u : narrow2<T>(f[0] * sc[j], f[1] * sc[j]);
            o[1] = none ? 0u : narrow2<T>(f[2] * sc[j], f[3] * sc[j]);
            o[2] = none ? 0u : narrow2<T>(f[4] * sc[j], f[5] * sc[j]);
            o[3] = none ? 0u : narrow2<T>(f[6] * sc[j], f[7] * sc[j]);
        }
        uint8_t *dst = static_cast<uint8_t *>(im[j].v ? a.v_out : a.k_out);
        *reinterpret_cast<u32x4v_t *>(
            dst + 2 * (((long long)(row0 + im[j].row) * a.n_kv_heads + im[j].head) * p.C + im[j].chunk) * 8) = o;
    }
}

template <typename T, bool E4>
void launch_cache_typed(const CacheParams &p, bool write, bool many, int blocks, hipStream_t s) {
    const dim3 grid(blocks), block(kCacheThreads);
    if (write) {
        if (many)
            launch_kernel("kv_write", kv_write_kernel<T, E4, kCacheItems>, grid, block, s, p);
        else
            launch_kernel("kv_write", kv_write_kernel<T, E4, 1>, grid, block, s, p);
    } else {
        if (many)
            launch_kernel("kv_read", kv_read_kernel<T, E4, kCacheItems>, grid, block, s, p);
        else
            launch_kernel("kv_read", kv_read_kernel<T, E4, 1>, grid, block, s, p);
    }
}

}  // namespace

hipError_t launch_cache(const CacheArgs &a, bool write, hipStream_t s) {
    CacheParams p{};
    p.a = a;
    p.C = a.head_dim / 8;
    p.cshift = log2_of(p.C);
    p.per_row = 2 * a.n_kv_heads * p.C;
    p.items = (long long)a.n_rows * p.per_row;
    p.pshift = log2_of(a.page_size);
    // Us with one / four items a thread (8 heads, D = 128: 256 items a row), a
    // bfloat16 write and an 8-bit write with its read: 2048 rows 6.0 / 4.9 and
    // 14.1 / 15.2, 4096 rows 8.6 / 7.9 and 25.0 / 21.6, 8192 rows 17.5 / 11.9 and
    // 52.2 / 32.8; up to 1024 rows the same.
    const bool many = p.items >= 2048LL * kCacheThreads;
    p.per_block = many ? kCacheThreads * kCacheItems : kCacheThreads;
    const int blocks = int((p.items + p.per_block - 1) / p.per_block);
    const bool e4 = a.cache_dtype == DSPARK_E4M3;
    if (a.dtype == DSPARK_BF16)
        e4 ? launch_cache_typed<TypeBf16, true>(p, write, many, blocks, s)
           : launch_cache_typed<TypeBf16, false>(p, write, many, blocks, s);
    else
        e4 ? launch_cache_typed<TypeF16, true>(p, write, many, blocks, s)
           : launch_cache_typed<TypeF16, false>(p, write, many, blocks, s);
    return hipGetLastError();
}

}  // namespace dspark
