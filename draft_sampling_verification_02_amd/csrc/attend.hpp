// attend.hpp -- building blocks of the attention kernels (paged.hip,
// prompt.hip): element types, matrix products, transposed LDS reads, direct
// loads into LDS and the cross-lane maximum and sum of a softmax.
//
// Both kernels compute the scores transposed, S^T = K Q^T: the A operand is a
// block of cache rows (tokens), the B operand the queries, so that a lane owns
// one query (the accumulator column) and its registers run over tokens.  The
// exponentials of those registers are then already the B operand of
// O^T = V^T P^T -- the order of the contraction index is free, so the tokens a
// lane happens to hold define it -- and the probabilities never leave the
// registers.  V^T comes from the row-major V tile by transposing LDS reads.
#pragma once

#include "device_common.hpp"

namespace dspark {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v_t __attribute__((ext_vector_type(4)));

// Element types of rows and caches: storage is 16 bits, E names the value type.
// kInf is the bit pattern of infinity: magnitudes from it on are not finite.
struct TypeBf16 {
    using E = __bf16;
    using V8 = bf16x8_t;
    static constexpr uint32_t kInf = 0x7f80;
};
struct TypeF16 {
    using E = _Float16;
    using V8 = f16x8_t;
    static constexpr uint32_t kInf = 0x7c00;
};

// the larger of each of two 16-bit halves, unsigned
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}

__device__ __forceinline__ f32x4_t mma16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma16(f16x8_t a, f16x8_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mma32(bf16x8_t a, bf16x8_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mma32(f16x8_t a, f16x8_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// ---------------------------------------------------------------- LDS access
// (`off`, a constant at the call, goes into the instruction)
typedef __attribute__((address_space(3))) uint8_t *LdsBytes;
template <typename T>
__device__ __forceinline__ T lds_read(uint32_t at, int off = 0) {
    return *reinterpret_cast<__attribute__((address_space(3))) const T *>(reinterpret_cast<LdsBytes>(at) + off);
}
template <typename T>
__device__ __forceinline__ void lds_write(uint32_t at, T v) {
    *reinterpret_cast<__attribute__((address_space(3))) T *>(at) = v;
}
__device__ __forceinline__ uint32_t lds_addr(const void *p) {
    return uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)p));
}
// Transposing reads.  Each group of 16 lanes reads a small matrix and every
// lane gets one of its 16 columns.  tr16: 4 rows of 16 16-bit values, lane
// 4 i + c addressing row i, columns 4 c .. 4 c + 3 (8 bytes).  tr8: 8 rows of
// 16 bytes, lane 2 j + c addressing row j, bytes 8 c .. 8 c + 7.
__device__ __forceinline__ s16x4_t lds_read_tr16(uint32_t at, int off = 0) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        reinterpret_cast<__attribute__((address_space(3))) s16x4_t *>(reinterpret_cast<LdsBytes>(at) + off));
}
__device__ __forceinline__ u32x2_t lds_read_tr8(uint32_t at, int off = 0) {
    return __builtin_bit_cast(
        u32x2_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                     reinterpret_cast<__attribute__((address_space(3))) i32x2_t *>(reinterpret_cast<LdsBytes>(at) + off)));
}
template <typename V8>
__device__ __forceinline__ V8 join4(s16x4_t a, s16x4_t b) {
    return __builtin_bit_cast(V8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Direct global-to-LDS loads, lane i writing 16 (or 4) bytes at lds + 16 i
// (4 i) from base + voff.  They go through asm because the compiler, told of
// such a load, makes every later LDS read wait for all of them; here the
// kernels wait themselves, by count (vm_wait).  The asm has no register
// outputs.  Extra loads in flight only make the compiler's own counted waits
// stricter.  M0, the LDS base, is written right before each load; nothing else
// in these kernels uses it.  lds and base are uniform.
__device__ __forceinline__ void dma16(uint32_t lds, uint32_t voff, const void *base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(voff), "s"(base)
                 : "memory");
}
// the same with an address a lane
__device__ __forceinline__ void dma16(uint32_t lds, const void *lane_src) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(lane_src) : "memory");
}
__device__ __forceinline__ void dma4(uint32_t lds, const void *lane_src) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" : : "s"(lds), "v"(lane_src) : "memory");
}
// Waits until at most N of this wave's vector memory operations are in flight.
template <int N>
__device__ __forceinline__ void vm_wait() {
    static_assert(N >= 0 && N < 64, "vmcnt is a 6-bit count");
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// Every LDS read of this wave has returned: its buffers may be refilled.
__device__ __forceinline__ void lds_drain() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

// Workgroup barrier that leaves the direct loads in flight: this wave's LDS
// accesses are done, and none moves across it.
__device__ __forceinline__ void wg_barrier() {
    lds_drain();
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(u));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(uint32_t(u >> 32));
    return reinterpret_cast<const uint8_t *>(uint64_t(hi) << 32 | lo);
}

// ---------------------------------------------------------------- cross-lane
// Over lanes l and l ^ 32, and l ^ 16: a swap of register halves leaves the
// two partners' values in the two results.
__device__ __forceinline__ float max_x32(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_x32(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float max_x16(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_x16(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The value again, opaque to the compiler: what is derived from it is made
// anew here instead of being held in registers across a loop.
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
    asm volatile("" : "+v"(x));
    return x;
}

// ---------------------------------------------------------------- values
template <typename T>
__device__ __forceinline__ float2 widen(uint32_t w) {
    if constexpr (std::is_same<T, TypeBf16>::value) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        const f16x2_t h = __builtin_bit_cast(f16x2_t, w);
        return make_float2(float(h[0]), float(h[1]));
    }
}
template <typename T>
__device__ __forceinline__ void widen4(u32x2_t w, float *v) {
    const float2 a = widen<T>(w[0]), b = widen<T>(w[1]);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}
__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) < __builtin_huge_valf(); }
// a pair of 16-bit values, and four e4m3 values, with zeros in the place of what is not finite
template <typename T>
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
    if ((w & 0x7fffu) >= T::kInf) w &= 0xffff0000u;
    if (((w >> 16) & 0x7fffu) >= T::kInf) w &= 0xffffu;
    return w;
}
// an infinity in the pair
template <typename T>
__device__ __forceinline__ bool has_infinity(uint32_t w) {
    return (w & 0x7fffu) == T::kInf || ((w >> 16) & 0x7fffu) == T::kInf;
}
__device__ __forceinline__ uint32_t finite_e4m3(uint32_t w) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        if (((w >> i) & 0x7fu) == 0x7fu) w &= ~(0xffu << i);
    return w;
}

// ---------------------------------------------------------------- e4m3
__device__ __forceinline__ void e4m3_to4(uint32_t w, float *v) {
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
    v[0] = a[0];
    v[1] = a[1];
    v[2] = b[0];
    v[3] = b[1];
}
// Eight e4m3 values (two words) as 16-bit floats; every e4m3 value is exact in
// both types.
__device__ __forceinline__ void e4m3_to8(u32x2_t w, bf16x8_t &o) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], 1.f, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], 1.f, true);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], 1.f, false);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], 1.f, true);
    o = bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ void e4m3_to8(u32x2_t w, f16x8_t &o) {
    const f16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[0], 1.f, false);
    const f16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[0], 1.f, true);
    const f16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[1], 1.f, false);
    const f16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[1], 1.f, true);
    o = f16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// 2^(byte - 127), the power-of-two scale of one (token, head)
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// Exponents of a softmax are fma(score, c, -m), the product unrounded, which is
// one instruction; m is itself a rounded product, so that the largest exponent
// is not 0 but m's rounding error: half a step of m.  From kFar on (half a step:
// 1/16) that would grow past any range of the probabilities, to zeros or
// infinities for all: there the products are rounded first.
constexpr float kFar = 1048576.f;
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kFar && m != kNegInf; }
__device__ __forceinline__ float far_exponent(float score, float c, float m) {
#pragma clang fp contract(off)
    const float product = score * c;
    return product - (m == kNegInf ? 0.f : m);
}

// The reference of a softmax whose probabilities are of type T: the maximum, for
// float16, whose range is narrow, lowered by `lift` (far from zero that would be
// lost in the maximum's own rounding).
template <typename T>
__device__ __forceinline__ float lowered(float mx, float lift) {
    if constexpr (std::is_same<T, TypeF16>::value)
        return fabsf(mx) < kFar ? mx - lift : mx;
    else
        return mx;
}

// The natural logsumexp from the reference (base-2 units) and the sum.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? kNegInf : (m + fast_log2(l)) * kLn2;
}

// Four channels of one output row (row * heads + head = at), normalised: out =
// o / l, zeros where nothing is visible; lse from the maximum and sum.
template <typename T>
__device__ __forceinline__ void store_row(void *out, float *lse, long long at, int c4, int D, f32x4_t o, float m, float l) {
    using E = typename T::E;
    typedef E e4_t __attribute__((ext_vector_type(4)));
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const e4_t x = l == 0.f ? e4_t{} : e4_t{E(o[0] * inv), E(o[1] * inv), E(o[2] * inv), E(o[3] * inv)};
    *reinterpret_cast<e4_t *>(static_cast<E *>(out) + at * D + 4 * c4) = x;
    if (lse && c4 == 0) lse[at] = lse_of(m, l);
}

// Adds a partial result (maximum m2, sum l2, products o2) to (m, l, o).
__device__ __forceinline__ void merge_partial(float &m, float &l, f32x4_t &o, float m2, float l2, f32x4_t o2) {
    const float mn = fmaxf(m, m2), ms = mn == kNegInf ? 0.f : mn;
    const float f1 = fast_exp2(m - ms), f2 = fast_exp2(m2 - ms);
    l = l * f1 + l2 * f2;
    o = o * f1 + o2 * f2;
    m = mn;
}

}  // namespace dspark
