// rules.hip -- penalties for repeated tokens, biases and grammar masks on the
// logits of a round's target rows, written as the float32 rows that the
// verification reads.
//
// Row j of a request, token v, whose text holds v c times as generated (the
// drafts x_1 .. x_j in front of the row among them) and possibly in its prompt:
//   z = l_v;  seen: z > 0 ? z / rho : z rho;  z -= phi c + pi [c > 0];
//   z += the biases of v;  -inf where the row's mask forbids v.
//
// Bound by memory: a row is read once and written once, 6 bytes an entry for
// 16-bit logits.  A workgroup takes one slice of the vocabulary for all rows of
// a request: it counts the request's text within the slice in LDS once, adds a
// draft from row to row, and streams the rows' slices through.  Counts are
// integers and biases are added in the order of their list, so that results do
// not depend on timing.  An entry that its mask forbids is not read.
#include <algorithm>

#include "dspark.h"
#include "rows.hpp"

namespace dspark {

namespace {

struct RulesParams {
    RulesArgs a;
    int slices;
};

constexpr long long kManySlices = 512;        // slices of 4096 entries that fill the chip
constexpr uint32_t kInPrompt = 0x80000000u;  // beside a token's count

// Four entries of a row as floats.
template <typename L>
__device__ __forceinline__ f32x4_t load4(const L *p) {
    if constexpr (sizeof(L) == 4) {
        return __builtin_nontemporal_load(reinterpret_cast<const f32x4_t *>(p));
    } else {
        using T = typename std::conditional<std::is_same<L, __bf16>::value, TypeBf16, TypeF16>::type;
        float f[4];
        widen4<T>(__builtin_nontemporal_load(reinterpret_cast<const u32x2_t *>(p)), f);
        return f32x4_t{f[0], f[1], f[2], f[3]};
    }
}

// A workgroup of NT threads, each with E entries of the slice: V4 four
// neighbouring ones at a time (rows 16-byte aligned), else one at a time.
template <typename L, int NT, int E, bool V4>
__global__ __launch_bounds__(NT) void rules_kernel(RulesParams p) {
    constexpr int S = NT * E, W = V4 ? 4 : 1, N = E / W;  // entries of the slice, of a load, loads
    __shared__ __attribute__((aligned(16))) uint32_t count[S];
    __shared__ __attribute__((aligned(16))) float bias[S];
    const RulesArgs &a = p.a;
    const int tid = threadIdx.x;
    const int b = int(blockIdx.x / unsigned(p.slices)), v0 = int(blockIdx.x - unsigned(b) * unsigned(p.slices)) * S;
    const int size = min(S, a.V - v0);  // entries there are
    int r0 = b, r1 = b + 1;
    if (a.row_offsets) {
        r0 = min(max(a.row_offsets[b], 0), a.n_rows);
        r1 = min(max(a.row_offsets[b + 1], 0), a.n_rows);
    }
    if (r0 >= r1) return;

    const float rho = a.repetition ? a.repetition[b] : 1.f;
    const float phi = a.frequency ? a.frequency[b] : 0.f, pi = a.presence ? a.presence[b] : 0.f;
    const bool counted = !(rho == 1.f && phi == 0.f && pi == 0.f);
    int e0 = 0, e1 = 0;
    if (a.bias_offsets) {
        e0 = min(max(a.bias_offsets[b], 0), a.n_biases);
        e1 = min(max(a.bias_offsets[b + 1], 0), a.n_biases);
    }
    const bool biased = e0 < e1;
    for (int i = tid; i < S; i += NT) {
        count[i] = 0;
        bias[i] = 0.f;
    }
    __syncthreads();
    // ---- biases: NT of the list at a time; of those with one token the first is added first
    for (int e = e0; e < e1; e += NT) {
        int i = -1;
        if (e + tid < e1) {
            i = a.bias_ids[e + tid] - v0;
            if (unsigned(i) >= unsigned(size)) i = -1;
        }
        while (__syncthreads_or(i >= 0)) {
            if (i >= 0) atomicMax(&count[i], uint32_t(NT - tid));
            __syncthreads();
            const bool first = i >= 0 && count[i] == uint32_t(NT - tid);
            if (first) bias[i] += a.bias_values[e + tid];
            __syncthreads();
            if (first) {
                count[i] = 0;
                i = -1;
            }
        }
    }
    // ---- the text
    if (counted && a.history) {
        const int32_t *text = a.history + (long long)b * a.max_history;
        const int len = min(max(a.history_len[b], 0), a.max_history);
        const int given = a.prompt_len ? a.prompt_len[b] : 0;
        constexpr int FLY = 8;
        for (int t0 = 0; t0 < len; t0 += NT * FLY) {
            int tok[FLY];
#pragma unroll
            for (int k = 0; k < FLY; ++k) {
                const int t = t0 + k * NT + tid;
                tok[k] = t < len ? text[t] : -1;
            }
#pragma unroll
            for (int k = 0; k < FLY; ++k) {
                const int i = tok[k] < 0 ? -1 : tok[k] - v0;
                if (unsigned(i) < unsigned(size)) {
                    if (t0 + k * NT + tid < given)
                        atomicOr(&count[i], kInPrompt);
                    else
                        atomicAdd(&count[i], 1u);
                }
            }
        }
        __syncthreads();
    }

    // ---- the rows
    auto entry = [&](int k) __device__ { return (k * NT + tid) * W; };  // first entry of load k
    for (int r = r0; r < r1; ++r) {
        if (r > r0 && counted && a.drafts && r - r0 - 1 < a.gamma) {
            const int i = a.drafts[(long long)b * a.gamma + (r - r0 - 1)] - v0;
            if (unsigned(i) < unsigned(size)) {
                __syncthreads();
                if (tid == 0) count[i] += 1;
                __syncthreads();
            }
        }
        const L *row = static_cast<const L *>(a.logits) + r * a.stride + v0;
        float *out = a.out + r * a.out_stride + v0;
        const int m = a.mask_index ? a.mask_index[r] : -1;
        const bool masked = m >= 0 && m < a.n_masks;
        const int32_t *bits = masked ? a.masks + (long long)m * a.mask_stride + v0 / 32 : nullptr;
        uint32_t keep[N];
        float z[N][W];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = entry(k);
            keep[k] = i < size ? (1u << W) - 1 : 0u;
            if (masked && i < size) keep[k] &= uint32_t(bits[i / 32]) >> (i & 31);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
#pragma unroll
            for (int w = 0; w < W; ++w) z[k][w] = 0.f;
            if (keep[k]) {
                if constexpr (V4) {
                    const f32x4_t x = load4<L>(row + entry(k));
#pragma unroll
                    for (int w = 0; w < 4; ++w) z[k][w] = x[w];
                } else {
                    z[k][0] = float(row[entry(k)]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = entry(k);
            if (i >= size) continue;
            if (counted) {
                uint32_t c[W], any = 0;
#pragma unroll
                for (int w = 0; w < W; ++w) any |= c[w] = count[i + w];
                if (any) {
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        if (c[w]) {
                            const float n = float(c[w] & ~kInPrompt);
                            float x = z[k][w];
                            x = x > 0.f ? x / rho : x * rho;
                            z[k][w] = x - (phi * n + (n > 0.f ? pi : 0.f));
                        }
                }
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (biased) z[k][w] += bias[i + w];
                if (!((keep[k] >> w) & 1)) z[k][w] = kNegInf;
            }
            if constexpr (V4)
                __builtin_nontemporal_store(f32x4_t{z[k][0], z[k][1], z[k][2], z[k][3]}, reinterpret_cast<f32x4_t *>(out + i));
            else
                out[i] = z[k][0];
        }
    }
}

template <typename L, int NT, int E>
void launch_rules_slices(RulesParams p, bool v4, hipStream_t s) {
    p.slices = (p.a.V + NT * E - 1) / (NT * E);
    const dim3 grid(unsigned(p.slices) * unsigned(p.a.B));
    if (v4)
        launch_kernel("logit_rules", rules_kernel<L, NT, E, true>, grid, dim3(NT), s, p);
    else
        launch_kernel("logit_rules", rules_kernel<L, NT, E, false>, grid, dim3(NT), s, p);
}

template <typename L>
void launch_rules_typed(const RulesParams &p, bool v4, hipStream_t s) {
    if ((long long)p.a.B * p.a.V >= kManySlices * 4096LL)
        launch_rules_slices<L, 512, 8>(p, v4, s);
    else
        launch_rules_slices<L, 256, 4>(p, v4, s);
}

}  // namespace

hipError_t launch_rules(const RulesArgs &a, hipStream_t s) {
    RulesParams p{};
    p.a = a;
    const size_t elt = a.dtype == DSPARK_F32 ? 4 : 2;
    // rows of four entries: the vocabulary, the strides and the buffers allow it
    const bool v4 = a.V % 4 == 0 && a.stride % 4 == 0 && a.out_stride % 4 == 0 &&
                    reinterpret_cast<uintptr_t>(a.logits) % (4 * elt) == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
    switch (a.dtype) {
        case DSPARK_F32: launch_rules_typed<float>(p, v4, s); break;
        case DSPARK_BF16: launch_rules_typed<__bf16>(p, v4, s); break;
        default: launch_rules_typed<_Float16>(p, v4, s); break;
    }
    return hipGetLastError();
}

}  // namespace dspark
