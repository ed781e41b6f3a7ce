// rotary.hip -- heads normed and turned by their positions: query and key rows
// (rotary), and the same with the keys and values going into the paged cache
// (kv_append).
//
// For a head x of D channels at position p:
//   y = x, or x w / sqrt(mean(x^2) + eps) with a norm of weights w,
//   (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a),  a = p f_m
// over the pairs (i, j) = (m, m + rot / 2), or neighbours (2 m, 2 m + 1), m <
// rot / 2; channels from rot on keep y.  Everything is in 32 bits and rounded
// once, to the rows' type or to the 8-bit cache's (the scale then is that of the
// 32-bit values).  An angle is far larger than what matters of it: its turns p f /
// 2 pi are taken in 64 bits, off by 2^-51 of them at most (two products and a
// constant, each rounded), and so are the cosine and sine of their fraction.  A workgroup takes each angle once, whatever the number of
// heads.
//
// Bound by memory: every row is read once and written once.  A work item is 16
// values, two chunks of 8 that hold each other's pairs, so a rotation stays in
// its lane; D / 16 neighbouring lanes hold a head, and its norm and scale are
// sums and maxima over lane permutes.  A lane loads only what it stores itself:
// rows may be turned in place.
//
// Measured (MI355X, 32/8 heads, D = 128, bfloat16): 37,800 rows normed and turned
// 146-158 us over cards (774 MB, 4.9 to 5.3 TB/s; a large copy reaches 4.75); 64 rows
// 3.6 us, 64 appended 4.9; 853 normed rows of 256 requests into 8 bits 9.3 us; 50,000
// rows of 16/4 heads, D = 64, into a float16 cache 68 us (307 MB, 4.5 TB/s).
#include <algorithm>

#include "dspark.h"
#include "rows.hpp"

namespace dspark {

namespace {

constexpr int kTableFloats = 4096;  // cosines and sines of a workgroup's rows
constexpr int kRotaryItems = 2;     // items of a thread
constexpr int kManyItems = 4;       // where many go into a cache

struct RotaryParams {
    RotaryArgs a;
    long long items;  // n_rows * heads * (D / 16)
    int per_row;      // heads * (D / 16), heads = n_heads + n_kv_heads, + n_kv_heads with a cache
    int per_block;    // items of a workgroup
    int pshift;
};

template <int D>
constexpr int kRotaryRows = kTableFloats / D;  // rows a workgroup touches at most

enum { kToRows, kToCache, kToCache8 };

// Sum and maximum over the LANES (4, 8 or 16) neighbouring lanes of a head.
template <int LANES>
__device__ __forceinline__ float head_sum(float x) {
    auto add = [&](auto ctrl) __device__ {
        x += __uint_as_float(uint32_t(__builtin_amdgcn_mov_dpp(int(__float_as_uint(x)), decltype(ctrl)::value, 0xF, 0xF, true)));
    };
    add(std::integral_constant<int, 0xB1>{});   // lanes l ^ 1
    add(std::integral_constant<int, 0x4E>{});   // l ^ 2
    if constexpr (LANES >= 8) add(std::integral_constant<int, 0x141>{});   // the eight lanes mirrored
    if constexpr (LANES >= 16) add(std::integral_constant<int, 0x140>{});  // the sixteen
    return x;
}
template <int LANES>
__device__ __forceinline__ float head_max(float x) {
    auto top = [&](auto ctrl) __device__ {
        x = fmaxf(x, __uint_as_float(uint32_t(__builtin_amdgcn_mov_dpp(int(__float_as_uint(x)), decltype(ctrl)::value, 0xF, 0xF, true))));
    };
    top(std::integral_constant<int, 0xB1>{});
    top(std::integral_constant<int, 0x4E>{});
    if constexpr (LANES >= 8) top(std::integral_constant<int, 0x141>{});
    if constexpr (LANES >= 16) top(std::integral_constant<int, 0x140>{});
    return x;
}

// Cosine and sine of an angle of -1/2 to 1/2 turns, off by half a step of float32 and
// 2^-32: the Taylor series in 64 bits over an eighth of a turn to either side of the
// nearest quarter, where what is left out is below x^13 / 13! = 7e-12 and x^12 / 12! =
// 1.2e-10.
__device__ __forceinline__ float2 cos_sin(double turn) {
    const double q = rint(4. * turn), x = __builtin_fma(q, -0.25, turn) * 6.283185307179586, y = x * x;
    double s = __builtin_fma(y, -1. / 39916800., 1. / 362880.);
    s = __builtin_fma(y, s, -1. / 5040.);
    s = __builtin_fma(y, s, 1. / 120.);
    s = __builtin_fma(y, s, -1. / 6.);
    s = __builtin_fma(x * y, s, x);
    double c = __builtin_fma(y, -1. / 3628800., 1. / 40320.);
    c = __builtin_fma(y, c, -1. / 720.);
    c = __builtin_fma(y, c, 1. / 24.);
    c = __builtin_fma(y, c, -1. / 2.);
    c = __builtin_fma(y, c, 1.);
    const int k = int(q) & 3;  // quarters: (c, s), (-s, c), (-c, -s), (s, -c)
    const float a = float(k & 1 ? s : c), b = float(k & 1 ? c : s);
    return make_float2(k == 1 || k == 2 ? -a : a, k >= 2 ? -b : b);
}

template <typename T>
__device__ __forceinline__ void widen8(u32x4v_t w, float *f) {
    widen4<T>(u32x2_t{w[0], w[1]}, f);
    widen4<T>(u32x2_t{w[2], w[3]}, f + 4);
}
template <typename T>
__device__ __forceinline__ u32x4v_t narrow8(const float *f) {
    using E = typename T::E;
    typedef E e8_t __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(u32x4v_t, e8_t{E(f[0]), E(f[1]), E(f[2]), E(f[3]), E(f[4]), E(f[5]), E(f[6]), E(f[7])});
}
// eight values, none past 448, as e4m3
__device__ __forceinline__ int2 to_e4m3x8(const float *f, float inv) {
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * inv, f[1] * inv, 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * inv, f[3] * inv, lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4] * inv, f[5] * inv, 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6] * inv, f[7] * inv, hi, true);
    return make_int2(lo, hi);
}

template <typename T, int D, int MODE, int ITEMS>
__global__ __launch_bounds__(kCacheThreads) void rotary_kernel(RotaryParams p) {
    constexpr int LANES = D / 16, R = kRotaryRows<D>;
    __shared__ __attribute__((aligned(16))) float table[kTableFloats];  // row: rot / 2 cosines, rot / 2 sines
    __shared__ __attribute__((aligned(16))) float weight[2][D];         // of queries and keys
    __shared__ long long slots[R], at[R];
    __shared__ int red[8];
    const RotaryArgs &a = p.a;
    const CacheArgs &c = a.c;
    const int tid = threadIdx.x, half = a.rot / 2;

    // the workgroup's items: `count` of them, from item rel0 of row row0
    const long long it0 = (long long)blockIdx.x * p.per_block;
    const int count = int(min((long long)p.per_block, p.items - it0));
    const int row0 = int(it0 / p.per_row), rel0 = int(it0 - (long long)row0 * p.per_row);
    const int rows = int(unsigned(rel0 + count - 1) / unsigned(p.per_row)) + 1;

    struct Item {
        int row, kind, head, c0, c1;  // row from row0 on; 0 query, 1 key, 2 value; its chunks
        bool turned;
    };
    Item im[ITEMS];
    u32x4v_t x[ITEMS][2];
    // the rows go out first: their addresses need no request
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const int rel = rel0 + min(tid + j * kCacheThreads, count - 1);
        Item &t = im[j];
        t.row = int(unsigned(rel) / unsigned(p.per_row));
        const int rest = rel - t.row * p.per_row, l = rest & (LANES - 1);
        t.head = rest / LANES;
        t.kind = 0;
        if (t.head >= a.n_heads) {
            t.head -= a.n_heads;
            t.kind = 1;
            if (MODE != kToRows && t.head >= c.n_kv_heads) {
                t.head -= c.n_kv_heads;
                t.kind = 2;
            }
        }
        // a lane of the turned channels holds chunks l and l + rot / 16, where the pairs of both kinds
        // lie; the others share the rest
        t.turned = t.kind < 2 && l < a.rot / 16;
        if (t.kind == 2) {
            t.c0 = l;
            t.c1 = l + LANES;
        } else if (t.turned) {
            t.c0 = l;
            t.c1 = l + a.rot / 16;
        } else {
            t.c0 = l + a.rot / 16;
            t.c1 = l + LANES;
        }
        const uint8_t *src = static_cast<const uint8_t *>(t.kind == 0 ? a.q : t.kind == 1 ? c.k : c.v);
        const long long stride = t.kind == 0 ? a.q_stride : t.kind == 1 ? c.k_stride : c.v_stride;
        src += 2 * ((row0 + t.row) * stride + (long long)t.head * D);
        x[j][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4v_t *>(src) + t.c0);
        x[j][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4v_t *>(src) + t.c1);
    }
    // norm weights, and each row's position and slot
    for (int i = tid; i < 2 * D; i += kCacheThreads) {
        const void *w = i < D ? a.q_norm : a.k_norm;
        const int ch = i & (D - 1);
        if (w) {
            float f;
            if (a.norm_dtype == DSPARK_F32) {
                f = static_cast<const float *>(w)[ch];
            } else {
                const uint32_t pair = static_cast<const uint16_t *>(w)[ch];
                f = widen<T>(pair).x;
            }
            weight[i / D][ch] = f;
        }
    }
    int b0 = 0, b1 = 0;
    if (c.row_offsets) find_requests(c.row_offsets, c.B, row0, row0 + rows - 1, red, b0, b1);
    for (int t = tid; t < rows; t += kCacheThreads) {
        const RowPlace pl = place_row(c, p.pshift, row0 + t, b0, b1);
        slots[t] = pl.slot;
        at[t] = pl.pos;
    }
    __syncthreads();
    for (int i = tid; i < rows * half; i += kCacheThreads) {
        const int r = int(unsigned(i) / unsigned(half)), m = i - r * half;
        const double turns = double(at[r]) * double(a.inv_freq[m]) * 0.15915494309189535;  // 1 / 2 pi
        const float2 cs = cos_sin(turns - rint(turns));
        table[r * a.rot + m] = cs.x;
        table[r * a.rot + half + m] = cs.y;
    }
    __syncthreads();

#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const Item &t = im[j];
        const bool live = tid + j * kCacheThreads < count;
        const bool taken = live && at[t.row] >= 0;  // (a row of no request has no position)
        float f[16];
        widen8<T>(x[j][0], f);
        widen8<T>(x[j][1], f + 8);
        bool changed = false;
        const bool normed = t.kind < 2 && (t.kind ? a.k_norm : a.q_norm) != nullptr;
        if (__any(normed)) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) sum = __builtin_fmaf(f[i], f[i], sum);
            const float s = rsqrtf(head_sum<LANES>(sum) * (1.f / D) + a.eps);
            if (normed) {
                const float *w = weight[t.kind];
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const f32x4_t y = *reinterpret_cast<const f32x4_t *>(w + (i < 8 ? t.c0 * 8 : t.c1 * 8 - 8) + i);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i + k] = y[k];
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = f[i] * s * v[i];
                changed = true;
            }
        }
        if (t.turned) {
            changed = true;
            float co[8], si[8];
            if (!a.neighbours) {
                const float *row = table + t.row * a.rot + 8 * t.c0;
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const f32x4_t y = *reinterpret_cast<const f32x4_t *>(row + i), z = *reinterpret_cast<const f32x4_t *>(row + half + i);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        co[i + k] = y[k];
                        si[i + k] = z[k];
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = f[i], v = f[8 + i];
                    f[i] = __builtin_fmaf(u, co[i], -(v * si[i]));
                    f[8 + i] = __builtin_fmaf(v, co[i], u * si[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float *row = table + t.row * a.rot + 4 * (i ? t.c1 : t.c0);
                    const f32x4_t y = *reinterpret_cast<const f32x4_t *>(row), z = *reinterpret_cast<const f32x4_t *>(row + half);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        co[i + k] = y[k];
                        si[i + k] = z[k];
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = f[2 * i], v = f[2 * i + 1];
                    f[2 * i] = __builtin_fmaf(u, co[i], -(v * si[i]));
                    f[2 * i + 1] = __builtin_fmaf(v, co[i], u * si[i]);
                }
            }
        }
        const u32x4v_t y0 = changed ? narrow8<T>(f) : x[j][0], y1 = changed ? narrow8<T>(f + 8) : x[j][1];
        if (MODE == kToRows || t.kind == 0) {
            uint8_t *dst = static_cast<uint8_t *>(t.kind == 0 ? a.q_out : c.k_out);
            const long long stride = t.kind == 0 ? a.q_out_stride : a.k_out_stride;
            dst += 2 * ((row0 + t.row) * stride + (long long)t.head * D);
            if (taken) {
                reinterpret_cast<u32x4v_t *>(dst)[t.c0] = y0;
                reinterpret_cast<u32x4v_t *>(dst)[t.c1] = y1;
            }
        }
        if constexpr (MODE != kToRows) {
            const long long slot = slots[t.row];
            const long long rowat = slot + ((long long)t.head << p.pshift);  // row of the cache, D values each
            const bool stored = taken && slot >= 0 && t.kind > 0;
            uint8_t *cache = static_cast<uint8_t *>(t.kind == 2 ? c.v_cache : c.k_cache);
            if constexpr (MODE == kToCache) {
                if (stored) {
                    u32x4v_t *dst = reinterpret_cast<u32x4v_t *>(cache + rowat * (2 * D));
                    dst[t.c0] = y0;
                    dst[t.c1] = y1;
                }
            } else {
                // infinities and NaN become NaN, the scale is that of the finite values
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, is_finite(f[i]) ? fabsf(f[i]) : 0.f);
                const int e = scale_exponent(head_max<LANES>(top));
                const float inv = __uint_as_float(uint32_t(127 - e) << 23);  // e in -126 .. 120
                if (stored) {
                    int2 *dst = reinterpret_cast<int2 *>(cache + rowat * D);
                    dst[t.c0] = to_e4m3x8(f, inv);
                    dst[t.c1] = to_e4m3x8(f + 8, inv);
                    if (t.c0 == 0) (t.kind == 2 ? c.v_scale : c.k_scale)[rowat] = uint8_t(e + 127);
                }
            }
        }
    }
}

template <typename T, int D, int MODE>
void launch_rotary_items(const RotaryParams &p, bool many, int blocks, hipStream_t s) {
    const char *name = MODE == kToRows ? "rotary" : "kv_append";
    if constexpr (MODE != kToRows)
        if (many) return launch_kernel(name, rotary_kernel<T, D, MODE, kManyItems>, dim3(blocks), dim3(kCacheThreads), s, p);
    launch_kernel(name, rotary_kernel<T, D, MODE, kRotaryItems>, dim3(blocks), dim3(kCacheThreads), s, p);
}

template <typename T, int D>
void launch_rotary_mode(const RotaryParams &p, bool many, int blocks, hipStream_t s) {
    if (!p.a.c.k_cache)
        launch_rotary_items<T, D, kToRows>(p, many, blocks, s);
    else if (p.a.c.cache_dtype == DSPARK_E4M3)
        launch_rotary_items<T, D, kToCache8>(p, many, blocks, s);
    else
        launch_rotary_items<T, D, kToCache>(p, many, blocks, s);
}

template <typename T>
void launch_rotary_dim(const RotaryParams &p, bool many, int blocks, hipStream_t s) {
    switch (p.a.c.head_dim) {
        case 64: return launch_rotary_mode<T, 64>(p, many, blocks, s);
        case 128: return launch_rotary_mode<T, 128>(p, many, blocks, s);
        default: return launch_rotary_mode<T, 256>(p, many, blocks, s);
    }
}

}  // namespace

// A workgroup takes whole heads, and no more rows than its table of angles holds.
// Us a call in 2 / 4 items a thread, captured (packed rows of 64 requests, normed):
// rotation (32/8 heads, D = 128) of 64 rows 5.0 / 6.4, 1000 7.3 / 8.4, 4000 19.8 / 21.0,
// 37,800 147 / 150 (one item 161); appends of the same heads to 8 bits, 1000 rows 8.0 /
// 9.5, 2000 15.0 / 13.2, 16,000 81.7 / 76.3; appends of 16/4 heads, D = 64, in float16,
// 4000 rows 8.1 / 9.6, 16,000 26.6 / 24.7, 50,000 68.6 / 64.6.
RotaryPlan rotary_plan(long long n_rows, int heads, int head_dim, bool to_cache) {
    RotaryPlan p{};
    p.per_row = heads * (head_dim / 16);
    p.items = n_rows * p.per_row;
    p.many = to_cache && p.items >= 2048LL * kCacheThreads;
    p.per_block = std::min(kCacheThreads * (p.many ? kManyItems : kRotaryItems), (kTableFloats / head_dim - 1) * p.per_row);
    p.blocks = (p.items + p.per_block - 1) / p.per_block;
    return p;
}

hipError_t launch_rotary(const RotaryArgs &a, const RotaryPlan &plan, hipStream_t s) {
    RotaryParams p{};
    p.a = a;
    p.items = plan.items;
    p.per_row = plan.per_row;
    p.per_block = plan.per_block;
    p.pshift = a.c.k_cache ? log2_of(a.c.page_size) : 0;
    if (a.c.dtype == DSPARK_BF16)
        launch_rotary_dim<TypeBf16>(p, plan.many, int(plan.blocks), s);
    else
        launch_rotary_dim<TypeF16>(p, plan.many, int(plan.blocks), s);
    return hipGetLastError();
}

}  // namespace dspark
