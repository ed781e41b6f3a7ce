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
//
// Measured (MI355X): 852 bfloat16 rows of 129,280 of 256 requests with texts up to
// 4096, biases and masks 144-155 us (664 MB, 4.3 to 4.6 TB/s); one float16 row 4.9 us; 76
// float32 rows of 50,257 with texts up to 60,000 27 us, of which the texts, read by
// every slice's workgroup, take 9, five rows one after another 10.
#include "dspark.h"
#include "rows.hpp"

namespace dspark {

namespace {

struct RulesParams {
    RulesArgs a;
    int slices;
};

constexpr uint32_t kInPrompt = 0x80000000u;  // beside a token's count
constexpr int kTurns = 4;                    // of a part of the bias list, an entry of each token

// W entries of a row as they come, and as floats.
template <typename L, int W>
struct Piece {
    typedef L type __attribute__((ext_vector_type(W)));
    static_assert(W == 4, "one entry is a type of its own");
};
template <typename L>
struct Piece<L, 1> {
    typedef L type;
};
template <typename L, int W>
__device__ __forceinline__ float piece_at(const typename Piece<L, W>::type &x, int w) {
    if constexpr (W == 1)
        return float(x);
    else
        return float(x[w]);
}

// A workgroup of NT threads, each with E entries of the slice: V4 four
// neighbouring ones at a time (rows 16-byte aligned), else one at a time.
//
// What a row needs comes on the way one row ahead, and its mask two: the mask
// says which entries are read.  (An entry that is not reads the slice's first one
// instead, one line for all of them: a load without a branch, so that the ones
// before it can be waited for by count.)
template <typename L, int NT, int E, bool V4>
__global__ __launch_bounds__(NT) void rules_kernel(RulesParams p) {
    constexpr int S = NT * E, W = V4 ? 4 : 1, N = E / W;  // entries of the slice, of a load, loads
    using X = typename Piece<L, W>::type;
    __shared__ __attribute__((aligned(16))) uint32_t count[S];
    __shared__ __attribute__((aligned(16))) float bias[S];
    __shared__ __attribute__((aligned(16))) int32_t ids[NT];  // entries of the bias list
    __shared__ __attribute__((aligned(16))) float values[NT];
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

    // ---- what is on its way first: the text, the first rows' masks, the first row
    const float rho = a.repetition ? a.repetition[b] : 1.f;
    const float phi = a.frequency ? a.frequency[b] : 0.f, pi = a.presence ? a.presence[b] : 0.f;
    const bool counted = !(rho == 1.f && phi == 0.f && pi == 0.f);
    const int32_t *text = a.history ? a.history + (long long)b * a.max_history : nullptr;
    const int len = counted && text ? min(max(a.history_len[b], 0), a.max_history) : 0;
    const int given = a.prompt_len ? a.prompt_len[b] : 0;
    constexpr int FLY = 8;  // tokens of a thread under way
    int tok[FLY];
    auto read_text = [&](int t0, int *to) __device__ {  // (past the end the last token again: not looked at)
#pragma unroll
        for (int k = 0; k < FLY; ++k) to[k] = text[min(t0 + k * NT + tid, len - 1)];
    };
    auto entry = [&](int k) __device__ { return (k * NT + tid) * W; };  // first entry of load k
    // which entries of row r the thread keeps, W bits a load (none of a row past the last one)
    auto read_mask = [&](int r, uint32_t *keep) __device__ {
        const int m = a.mask_index && r < r1 ? a.mask_index[r] : -1;
        const bool masked = m >= 0 && m < a.n_masks;
        const int32_t *bits = masked ? a.masks + (long long)m * a.mask_stride + v0 / 32 : nullptr;
#pragma unroll
        for (int k = 0; k < N; ++k) keep[k] = masked ? uint32_t(bits[min(entry(k), size - 1) / 32]) : r < r1 ? ~0u : 0u;
    };
    auto kept = [&](const uint32_t *keep, int k) __device__ {
        return entry(k) < size ? keep[k] >> (entry(k) & 31) & ((1u << W) - 1) : 0u;
    };
    auto read_row = [&](int r, const uint32_t *keep, X *x) __device__ {
        const L *row = static_cast<const L *>(a.logits) + min(r, r1 - 1) * a.stride + v0;
#pragma unroll
        for (int k = 0; k < N; ++k)
            x[k] = __builtin_nontemporal_load(reinterpret_cast<const X *>(row + (kept(keep, k) ? entry(k) : 0)));
    };
    uint32_t keep[N], keep_next[N];
    X x[N], x_next[N];
    if (len > 0) read_text(0, tok);
    read_mask(r0, keep);
    read_mask(r0 + 1, keep_next);
    int e0 = 0, e1 = 0;
    if (a.bias_offsets) {
        e0 = min(max(a.bias_offsets[b], 0), a.n_biases);
        e1 = min(max(a.bias_offsets[b + 1], 0), a.n_biases);
    }
    const bool biased = e0 < e1;
    read_row(r0, keep, x);

    if (counted || biased) {
        for (int i = tid; i < S; i += NT) count[i] = 0;
        if (biased)
            for (int i = tid; i < S; i += NT) bias[i] = 0.f;
        __syncthreads();
    }
    // ---- biases: NT of the list at a time; of those with one token the first is added first, an entry of each token
    // a turn, and after kTurns of them the first that is left adds the others too.  (Us a call on one row, turns
    // alone / now: 4096 entries of the whole vocabulary 17 / 17, of 64 tokens 77 / 91, of one token 2068 / 102.)
    for (int e = e0; e < e1; e += NT) {
        int i = -1, turn = 0;
        if (e + tid < e1) {
            i = a.bias_ids[e + tid] - v0;
            if (unsigned(i) >= unsigned(size)) i = -1;
        }
        while (__syncthreads_or(i >= 0)) {
            const bool all = turn++ == kTurns;
            float value = 0.f;
            if (i >= 0) {
                atomicMax(&count[i], uint32_t(NT - tid));
                value = a.bias_values[e + tid];
            }
            if (all) {
                ids[tid] = i;
                values[tid] = value;
            }
            __syncthreads();
            const bool first = i >= 0 && count[i] == uint32_t(NT - tid);
            if (first) {
                float sum = bias[i];
                if (all) {  // (it is the first: none stands before it.  x + -0 is x, and no branch)
#pragma unroll 4
                    for (int k = tid & -64; k < NT; k += 4) {
                        const u32x4v_t other = *reinterpret_cast<const u32x4v_t *>(ids + k);
                        const f32x4_t y = *reinterpret_cast<const f32x4_t *>(values + k);
#pragma unroll
                        for (int w = 0; w < 4; ++w) sum += int(other[w]) == i ? y[w] : -0.f;
                    }
                } else {
                    sum += value;
                }
                bias[i] = sum;
            }
            __syncthreads();
            if (first) count[i] = 0;
            if (first || all) i = -1;
        }
    }
    // ---- the text
    for (int t0 = 0; t0 < len; t0 += NT * FLY) {
        int next[FLY];
        read_text(t0 + NT * FLY, next);
#pragma unroll
        for (int k = 0; k < FLY; ++k) {
            // (ids outside the vocabulary are in no slice, negative ones far above all as unsigned numbers)
            const uint32_t i = uint32_t(tok[k]) - uint32_t(v0);
            const int t = t0 + k * NT + tid;
            if (t < len && i < uint32_t(size)) {
                if (t < given)
                    atomicOr(&count[i], kInPrompt);
                else
                    atomicAdd(&count[i], 1u);
            }
            tok[k] = next[k];
        }
    }
    if (counted || biased) __syncthreads();

    // ---- the rows
    for (int r = r0; r < r1; ++r) {
        uint32_t keep_later[N];
        read_row(r + 1, keep_next, x_next);
        read_mask(r + 2, keep_later);
        if (r > r0 && counted && a.drafts && r - r0 - 1 < a.gamma) {
            const int i = a.drafts[(long long)b * a.gamma + (r - r0 - 1)] - v0;
            if (unsigned(i) < unsigned(size)) {
                __syncthreads();
                if (tid == 0) count[i] += 1;
                __syncthreads();
            }
        }
        float *out = a.out + r * a.out_stride + v0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = entry(k);
            if (i < size) {
                float z[W];
                uint32_t c[W] = {};
#pragma unroll
                for (int w = 0; w < W; ++w) z[w] = piece_at<L, W>(x[k], w);
                if (counted) {
                    uint32_t any = 0;
#pragma unroll
                    for (int w = 0; w < W; ++w) any |= c[w] = count[i + w];
                    if (any) {
#pragma unroll
                        for (int w = 0; w < W; ++w)
                            if (c[w]) {
                                const float n = float(c[w] & ~kInPrompt);
                                const float y = z[w] > 0.f ? z[w] / rho : z[w] * rho;
                                z[w] = n > 0.f ? y - (phi * n + pi) : y;  // (an infinite phi times none would be NaN)
                            }
                    }
                }
                const uint32_t bits = kept(keep, k);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    if (biased) z[w] += bias[i + w];
                    if (!((bits >> w) & 1)) z[w] = kNegInf;
                }
                if constexpr (V4)
                    __builtin_nontemporal_store(f32x4_t{z[0], z[1], z[2], z[3]}, reinterpret_cast<f32x4_t *>(out + i));
                else
                    out[i] = z[0];
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            x[k] = x_next[k];
            keep[k] = keep_next[k];
            keep_next[k] = keep_later[k];
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

// The slices.  Few entries in all take small slices, for more workgroups; long
// texts, which every slice of a request reads, take more threads a workgroup and
// larger slices.  Us a call of 1 to 6 bfloat16 rows a request, V = 129280, in 256
// threads of 8 entries / 512 of 8 / 1024 of 4 / 256 of 4, > < the rule's:
//   256 requests, texts up to  4096  >149< / 158  / 233  / 200
//                             16384   178 />176< / 242  / 235
//                             60000   259 />222< / 279  / 361
//   16 requests, 600          >19.2< / 21.3 / 22.2 / 20.6
//   8                          13.7 / 13.7 / 13.2 />12.3<
//   1, one row                  5.5 /  5.9 /  6.3 /> 4.9<
//   2, texts up to 16384       15.1 / 14.7 / 12.9 />11.8<
//                  32768       18.5 / 15.9 />13.8</ 15.9
constexpr long long kFewEntries = 1500000;
constexpr int kLongText = 16384, kLongTextFew = 24576;

template <typename L>
void launch_rules_typed(const RulesParams &p, bool v4, hipStream_t s) {
    const int text = p.a.history ? p.a.max_history : 0;
    if ((long long)p.a.B * p.a.V >= kFewEntries)
        text < kLongText ? launch_rules_slices<L, 256, 8>(p, v4, s) : launch_rules_slices<L, 512, 8>(p, v4, s);
    else
        text < kLongTextFew ? launch_rules_slices<L, 256, 4>(p, v4, s) : launch_rules_slices<L, 1024, 4>(p, v4, s);
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
