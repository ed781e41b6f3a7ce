// prompt.hip -- attention over whole prompts: packed sequences of different
// lengths, grouped heads, causal or not.
//
// For query row i of a sequence with R rows and L keys and head h:
//   s_t = scale q . k_t over t < L, and t <= L - R + i if causal (the rows are
//   the last R positions; L = R for a prompt on its own, L > R behind a prefix),
//   out = sum_t exp(s_t - lse) v_t,  lse = log sum_t exp(s_t).
// The running maximum and sum of the softmax and the products are held in 32
// bits; probabilities are rounded to 16 bits as they enter the V product.
//
// What bounds it: 4 D flops for every (query, key) pair against 16-bit K and V
// tiles that a whole workgroup shares -- the matrix units, with the
// exponentials of the softmax beside them, and the clock, which falls to
// 1.7 GHz under this load (as it does under a large library product).  A
// workgroup of four waves takes 32 queries a wave: a query is a (row, head of
// the group) pair, heads fastest, so that the heads of a group share the K and
// V tiles and a workgroup covers few rows (the causal diagonal wastes little).
// Tiles of 64 tokens come in by direct loads, two K and two V buffers, one
// barrier a tile.  The products of tile j + 1 with the queries are taken
// beside the exponentials of tile j in one instruction stream, in steps laid
// out by hand (the compiler's own order left the matrix units waiting on LDS
// reads); two workgroups share a compute unit, so that one's start and end run
// beside the other's middle.  Workgroups of one key-value head are neighbours
// modulo the XCDs where the head count allows it, and the last rows of a
// sequence, which see the most keys, go first.  Where the query blocks do not
// fill the chip, their keys are split and prompt_join merges the parts.
//
// Measured (MI355X, bfloat16, 32 query and 8 key-value heads, D = 128): one
// prompt of 16384 tokens 1895-2008 us over several cards, 1095 to 1161 TFLOP/s,
// matrix units busy 64% of 1.72 GHz (a 16384-cubed library product reaches 1386
// TFLOP/s, 73% of 1.71 GHz); 16 prompts of 100 to 4100 tokens 931-1040 us over
// the cards, 910 to 1018 TFLOP/s, the rest being starts, ends and diagonal
// tiles.  16/4 heads at 8192 tokens: D = 64 163-170 us, 808 to
// 843 TFLOP/s; D = 256 564-624 us, 880 to 975 TFLOP/s (one wave a SIMD: the accumulators take half
// its registers).
#include <algorithm>

#include "attend.hpp"
#include "dspark.h"
#include "internal.hpp"

namespace dspark {

namespace {

constexpr int kKeys = 64;      // tokens of a tile
constexpr int kPromptWaves = 4;                      // of a workgroup
constexpr int kPromptQueries = 32 * kPromptWaves;    // queries of a workgroup
constexpr int kMinTiles = 2;                         // tiles of a split at least
// Growth of the running maximum that is left alone, base-2 units; and how far
// the softmax's reference lies below a float16 row's maximum.  Held 2^11 times as
// large, float16 probabilities keep their eleven bits down to 2^-25 of the
// largest instead of 2^-14, where the many small shares of a long prompt would be
// lost; with the slack they stay below 2^16.
template <typename T>
constexpr float kSlack = std::is_same<T, TypeF16>::value ? 4.f : 8.f;
constexpr float kLift = 11.f;

struct PromptParams {
    PromptArgs a;
    PromptWork w;
    int G, nsplit, slots;
    float c;  // scale * log2(e)
};

// Rows of RB = 2 D bytes in LDS, 16-byte chunk c of row r at c ^ k_swizzle(r)
// (K: 16 rows read at one chunk) or c ^ v_swizzle(r) (V: transposing reads
// take 4 rows of 64 bytes at a time).
template <int D>
struct KeyTile {
    static constexpr int RB = 2 * D;
    static constexpr int CPR = RB / 16;
    static constexpr int BYTES = kKeys * RB;
    static constexpr int PER = RB >= 256 ? 1 : 256 / RB;
    static constexpr int SW = CPR < 16 ? CPR : 16;
    __device__ static __forceinline__ int k_swizzle(int r) { return (r / PER) & (SW - 1); }
    __device__ static __forceinline__ int v_swizzle(int r) { return (((r & 3) / PER) * 4) & (SW - 1); }
};

template <int D>
struct PromptShape {
    using S = KeyTile<D>;
    static constexpr int NW = kPromptWaves, NT = 64 * NW;
    static constexpr int QB = kPromptQueries;
    static constexpr int LPT = kKeys * S::CPR / NT;          // loads a thread issues for K (and for V)
    static constexpr int LDS = 4 * S::BYTES;                  // two K tiles, two V tiles
    // Waves a SIMD.  (Three at D = 64 spill: 164 against 168 us at 8192 tokens, but
    // 13.3 against 11.2 us for 32 prompts of up to 200 rows, 16/4 heads.)
    static constexpr int EU = D >= 256 ? 1 : 2;
    static_assert(LPT * NT == kKeys * S::CPR && LDS <= 160 * 1024, "tile loads");
};

template <typename T, int D>
__global__ __launch_bounds__(64 * kPromptWaves, PromptShape<D>::EU) void prompt_kernel(PromptParams p) {
    using SH = PromptShape<D>;
    constexpr int NW = SH::NW;
    using S = KeyTile<D>;
    using V8 = typename T::V8;
    using E = typename T::E;
    constexpr int KS = D / 16, CB = D / 32;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[SH::LDS];
    __shared__ int found[5], found_bad, found_nan;

    const PromptArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n = lane & 31, h = lane >> 5;
    const uint32_t lds0 = lds_addr(lds);
    const int split = blockIdx.x % p.nsplit, unit = blockIdx.x / p.nsplit;
    const int kvh = unit % a.n_kv_heads;
    const int slot = p.slots - 1 - unit / a.n_kv_heads;

    // ---- the sequence and query block of this slot -----------------------
    // sequence b owns the slots from floor(off_b G / QB) + b on: enough for its
    // blocks, whatever the lengths, and found without a scan.  Every thread
    // tests its sequences with all it needs in one round of loads.
    auto clamped = [&](const int32_t *off, int i, int n_max) __device__ { return min(max(off[i], 0), n_max); };
    auto slot_of = [&](int off, int i) __device__ { return int((long long)off * p.G / SH::QB) + i; };
    if (tid == 0) {
        found[0] = -1;
        found_bad = found_nan = 0;
    }
    __syncthreads();
    for (int i = tid; i < a.B; i += SH::NT) {
        const int r0 = clamped(a.q_offsets, i, a.n_rows), r1 = clamped(a.q_offsets, i + 1, a.n_rows);
        int c0 = r0, c1 = r1;
        if (a.kv_offsets) {
            c0 = clamped(a.kv_offsets, i, a.n_kv_rows);
            c1 = clamped(a.kv_offsets, i + 1, a.n_kv_rows);
        }
        const int s0 = slot_of(r0, i);
        if (s0 <= slot && slot < slot_of(r1, i + 1)) {  // one sequence at most, as offsets do not decrease
            found[0] = slot - s0;
            found[1] = r0;
            found[2] = r1 - r0;
            found[3] = c0;
            found[4] = max(c1 - c0, 0);
        }
    }
    __syncthreads();
    // (the minima change nothing unless offsets decrease: then no row outside the arrays is touched)
    const int block = uniform(found[0]), q0 = uniform(found[1]), rows = min(uniform(found[2]), a.n_rows - q0);
    int k0 = uniform(found[3]), L = min(uniform(found[4]), a.n_kv_rows - k0);
    const int nq = rows * p.G;
    if (block < 0 || rows <= 0 || (long long)block * SH::QB >= nq) {
        if (p.nsplit > 1 && split == 0 && tid == 0) p.w.meta[unit] = make_int4(0, 0, 0, 0);
        return;
    }
    const int past = L - rows;
    auto limit_of = [&](int row) __device__ { return a.causal ? max(min(L, past + row + 1), 0) : L; };

    // this wave's queries
    const int wq0 = block * SH::QB + wave * 32;
    const int qi = wq0 + n;
    const int qrow = min(qi, nq - 1) / p.G, qhead = min(qi, nq - 1) - qrow * p.G;
    const int wlast = min(wq0 + 31, nq - 1);
    const int glast = min(block * SH::QB + SH::QB - 1, nq - 1);
    const int tiles = (uniform(limit_of(glast / p.G)) + kKeys - 1) / kKeys;  // that any query of the workgroup sees
    // this split's tiles; from here on keys count from its first
    const int per = max((tiles + p.nsplit - 1) / p.nsplit, p.nsplit > 1 ? kMinTiles : 0);
    const int parts = p.nsplit > 1 && per < tiles ? (tiles + per - 1) / per : 1;
    if (p.nsplit > 1 && split == 0 && tid == 0) p.w.meta[unit] = make_int4(parts, q0, nq, block);
    if (split >= parts) return;
    const int t0 = parts > 1 ? split * per * kKeys : 0;
    const int ntile = parts > 1 ? min(per, tiles - split * per) : tiles;
    k0 += t0;
    const int lim = (qi < nq ? limit_of(qrow) : 0) - t0;
    const int wmin = uniform(wq0 < nq ? limit_of(wq0 / p.G) : 0) - t0;
    const int wmax = uniform(wq0 < nq ? limit_of(wlast / p.G) : 0) - t0;
    const int gmin = uniform(limit_of(block * SH::QB / p.G)) - t0;
    L -= t0;

    // ---- loads of a tile ---------------------------------------------------
    const uint32_t kst = uint32_t(a.k_stride * 2), vst = uint32_t(a.v_stride * 2);
    // load j of a thread covers row j * RPL further down; the swizzles repeat
    // every 16 rows, so OFFS offsets serve all loads
    constexpr int RPL = SH::NT / S::CPR;
    constexpr int OFFS = RPL >= 16 ? 1 : 16 / RPL;
    uint32_t koff[OFFS], voff[OFFS];
#pragma unroll
    for (int j = 0; j < OFFS; ++j) {
        const int sl = (j * NW + wave) * 64 + lane, row = sl / S::CPR;
        koff[j] = row * kst + ((sl % S::CPR) ^ S::k_swizzle(row)) * 16;
        voff[j] = row * vst + ((sl % S::CPR) ^ S::v_swizzle(row)) * 16;
    }
    auto issue = [&](const void *src, long long stride, uint32_t st, const uint32_t *off, uint32_t dst, int t) __device__ {
        const uint8_t *base = uniform(static_cast<const uint8_t *>(src) + 2 * ((k0 + t) * stride + kvh * D));
        const int over = t + kKeys - L;
        if (over <= 0) {
#pragma unroll
            for (int j = 0; j < SH::LPT; ++j)
                dma16(uniform(dst + (j * NW + wave) * 1024), off[j % OFFS], uniform(base + size_t(j / OFFS * OFFS * RPL) * st));
        } else {
            // rows past the sequence repeat its last one: no query sees them
            // (offsets are unsigned, so a row's own offset is taken whole
            // before the rows it goes back are subtracted)
#pragma unroll
            for (int j = 0; j < SH::LPT; ++j) {
                const int row = ((j * NW + wave) * 64 + lane) / S::CPR;
                const uint32_t whole = off[j % OFFS] + uint32_t(j / OFFS * OFFS * RPL) * st;
                dma16(uniform(dst + (j * NW + wave) * 1024), whole - uint32_t(max(row + over - (kKeys - 1), 0)) * st, base);
            }
        }
    };
    auto issue_k = [&](int j) __device__ { issue(a.k, a.k_stride, kst, koff, lds0 + (j & 1) * S::BYTES, j * kKeys); };
    auto issue_v = [&](int j) __device__ { issue(a.v, a.v_stride, vst, voff, lds0 + (2 + (j & 1)) * S::BYTES, j * kKeys); };

    // ---- read addresses ----------------------------------------------------
    // K fragment (32 tokens from row r0, step k): chunk 2 k + h of row r0 + n;
    // V^T fragment (32 channels c, 16 tokens from row r0): rows r0 + 4 h + i and
    // r0 + 8 + 4 h + i.  The swizzles are XORs of chunk bits, so a step's chunk
    // is the first step's address with constant bits flipped.
    const uint32_t kread = n * S::RB + ((h ^ S::k_swizzle(n)) * 16);
    const int vrow = 4 * h + ((lane >> 2) & 3);
    const uint32_t vread = vrow * S::RB + (((((lane >> 4) & 1) * 2 + ((lane >> 1) & 1)) ^ S::v_swizzle(vrow)) * 16) + 8 * (lane & 1);
    // Held in registers for every step, except at D = 256, where there is no
    // room for them and they are made anew every tile.
    constexpr bool HELD = D < 256;
    uint32_t kheld[HELD ? KS : 1], vheld[HELD ? CB : 1];
    if constexpr (HELD) {
#pragma unroll
        for (int k = 0; k < KS; ++k) kheld[k] = kread ^ (32 * k);
#pragma unroll
        for (int c = 0; c < CB; ++c) vheld[c] = vread ^ (64 * c);
    }
    auto base_in = [&](uint32_t buf, uint32_t first) __device__ {
        if constexpr (HELD) return buf;
        uint32_t x = buf + first;
        asm volatile("" : "+v"(x));
        return x;
    };
    auto k_base = [&](uint32_t buf) __device__ { return base_in(buf, kread); };
    auto v_base = [&](uint32_t buf) __device__ { return base_in(buf, vread); };
    auto k_frag = [&](uint32_t base, int r0, int k) __device__ {
        return lds_read<V8>(HELD ? base + kheld[HELD ? k : 0] : base ^ (32 * k), r0 * S::RB);
    };
    auto v_frag = [&](uint32_t base, int r0, int c) __device__ {
        const uint32_t at = HELD ? base + vheld[HELD ? c : 0] : base ^ (64 * c);
        return join4<V8>(lds_read_tr16(at, r0 * S::RB), lds_read_tr16(at, (r0 + 8) * S::RB));
    };

    // ---- the first tiles and the queries, by way of the second K and V buffers
    // (whole rows a load; read straight into registers, every load touches 32
    // rows: 64 prompts of 200 to 300 rows 107 against 101 us, 32 of up to 200 rows
    // at D = 64 11.2 against 10.6).  A wave's 32 query rows fill half a buffer,
    // laid out as K rows are.
    V8 qf[KS];
    if (ntile > 0) {
        const int row0 = min(wq0, nq - 1) / p.G;
        const E *first = static_cast<const E *>(a.q) + (long long)(q0 + row0) * a.q_stride + (long long)kvh * p.G * D;
        const uint32_t own = uint32_t(qrow - row0) * uint32_t(a.q_stride * 2) + uint32_t(qhead * D * 2);
        const uint32_t qlds = lds0 + (wave < NW / 2 ? 1 : 3) * S::BYTES + wave % (NW / 2) * 32 * S::RB;
        constexpr int RPI = 1024 / S::RB;  // rows a load covers
#pragma unroll
        for (int j = 0; j < 32 / RPI; ++j) {
            const int row = j * RPI + lane / S::CPR;
            const uint32_t off = uint32_t(__shfl(int(own), row)) + ((lane % S::CPR) ^ S::k_swizzle(row)) * 16;
            dma16(uniform(qlds + j * 1024), off, uniform(reinterpret_cast<const uint8_t *>(first)));
        }
        issue_k(0);
        issue_v(0);
        vm_wait<SH::LPT>();
#pragma unroll
        for (int k = 0; k < KS; ++k) qf[k] = lds_read<V8>(qlds + (kread ^ (32 * k)));
        wg_barrier();  // K of tile 0 is in, every wave has its queries
        if (ntile > 1) issue_k(1);
    }

    float m, l, cs = p.c;  // maximum and sum; what scores are multiplied by
    bool far = false;      // the maximum of a query of the wave is far from zero
    f32x16_t o[CB];

    // ---- the walk, one tile ahead: while the scores of tile j become
    // probabilities and meet V, the products of tile j + 1 with the queries run
    // beside them in the same instruction stream
    f32x16_t s[2];  // s[tb][r] is token 32 tb + 8 (r / 4) + 4 h + r % 4 of the tile, query n
    auto scores = [&](int j, f32x16_t *x) __device__ {
        const uint32_t kb = k_base(lds0 + (j & 1) * S::BYTES);
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) x[tb] = f32x16_t{};
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) x[tb] = mma32(k_frag(kb, 32 * tb, k), qf[k], x[tb]);
    };
    auto hide = [&](int j, f32x16_t *x) __device__ {
        const int t = j * kKeys;
        if (t + kKeys <= wmin) return;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (t + 32 * tb + 8 * (r >> 2) + 4 * h + (r & 3) >= lim) x[tb][r] = kNegInf;
    };
    auto largest = [&](const f32x16_t *x) __device__ {
        float mx = fmaxf(x[0][0], x[1][0]);
#pragma unroll
        for (int r = 1; r < 16; ++r) mx = fmaxf(fmaxf(x[0][r], x[1][r]), mx);
        return lowered<T>(max_x32(mx) * p.c, kLift);
    };
    // the sums keep their scale until the maximum has grown by kSlack: probabilities
    // stay inside any type's range, and the products are rarely rescaled
    auto raise = [&](float mx, f32x16_t *x) __device__ {
        if (__any(mx > m + kSlack<T>)) {
            const float mn = fmaxf(m, mx);
            const float al = fast_exp2(m - (mn == kNegInf ? 0.f : mn));
            l *= al;
#pragma unroll
            for (int c = 0; c < CB; ++c) o[c] *= al;
            m = mn;
            far = __any(is_far(m));
        }
        // (scores far from zero become exponents at once)
        cs = far ? 1.f : p.c;
        if (far) {
#pragma unroll
            for (int tb = 0; tb < 2; ++tb)
#pragma unroll
                for (int r = 0; r < 16; ++r) x[tb][r] = far_exponent(x[tb][r], p.c, m);
        }
    };
    auto reference = [&]() __device__ { return far || m == kNegInf ? 0.f : m; };
    auto probabilities = [&](const f32x16_t *x, float ms, int f, V8 &pf) __device__ {
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = fast_exp2(__builtin_fmaf(x[f >> 1][8 * (f & 1) + i], cs, -ms));
        l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        pf = V8{E(e[0]), E(e[1]), E(e[2]), E(e[3]), E(e[4]), E(e[5]), E(e[6]), E(e[7])};
    };
    // K of tile j + 1 and V of tile j are in, and every wave is done with the
    // buffers that K of tile j + 2 and V of tile j + 1 go to
    auto turn = [&](int j) __device__ {
        vm_wait<0>();
        wg_barrier();
        if (j + 2 < ntile) issue_k(j + 2);
        if (j + 1 < ntile) issue_v(j + 1);
    };
    // What is not finite in a tile of V: the queries that see it get their share
    // of it here, and then it leaves the tile.  The share's probability is taken
    // anew in 32 bits: rounded to float16 it may be zero, and 0 * inf is NaN.  (What
    // is called twice and holds the sums has to be inlined, or they go to memory.)
    auto give_bad_shares = [&](int t, uint32_t vbuf) __device__ __attribute__((always_inline)) {
        const float ms = reference();
#pragma unroll 1
        for (int k = 0; k < kKeys; ++k) {
            // token k is s[k / 32][4 ((k / 8) % 4) + k % 4] of lane half (k / 4) % 2;
            // the lane holds channels 32 c + 8 i + 4 h .. + 3
            const int sw = S::v_swizzle(k), at = 16 * (k >> 5) + 4 * ((k >> 3) & 3) + (k & 3);
            float score = 0.f;
#pragma unroll
            for (int e = 0; e < 32; ++e) score = e == at ? s[e >> 4][e & 15] : score;
            const float pk = __shfl(fast_exp2(__builtin_fmaf(score, cs, -ms)), n + 32 * ((k >> 2) & 1));
            const bool sees = t + k < lim;
#pragma unroll
            for (int c = 0; c < CB; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    asm volatile("" : : : "memory");  // read four values at a time: registers are short
                    float v[4];
                    widen4<T>(lds_read<u32x2_t>(vbuf + k * S::RB + (((4 * c + i) ^ sw) * 16) + 8 * h), v);
                    if (__any(sees && !(is_finite(v[0]) && is_finite(v[1]) && is_finite(v[2]) && is_finite(v[3])))) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[c][4 * i + r] += sees && !is_finite(v[r]) ? pk * v[r] : 0.f;
                    }
                }
        }
    };
    // (every wave of the workgroup comes here)
    auto clean = [&](uint32_t vbuf) __device__ {
        wg_barrier();
#pragma unroll 1
        for (int i = tid; i < kKeys * S::CPR; i += SH::NT) {
            u32x4v_t w = lds_read<u32x4v_t>(vbuf + i * 16);
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = finite_pair<T>(w[q]);
            lds_write(vbuf + i * 16, w);
        }
        wg_barrier();
    };
    auto product = [&](uint32_t vb, const V8 *pf, int f) __device__ {
#pragma unroll
        for (int c = 0; c < CB; ++c) o[c] = mma32(v_frag(vb, 16 * f, c), pf[f], o[c]);
    };

    // nothing summed yet, the scores of tile 0
    auto begin = [&]() __device__ __attribute__((always_inline)) {
        m = kNegInf;
        l = 0.f;
        far = false;
#pragma unroll
        for (int c = 0; c < CB; ++c) o[c] = f32x16_t{};
        if (ntile > 0) {
            scores(0, s);
            hide(0, s);
            raise(largest(s), s);
        }
    };
    begin();
    // Tile j, which every query sees whole, with scores y; the next tile's scores
    // into x (HIDE: some of its keys may be hidden).  The two loops are the two halves of the work on
    // the matrix units; each step carries a share of the softmax and the LDS
    // reads of the steps to come, and the compiler keeps to the steps.
    auto step = [&](int jj, f32x16_t *y, f32x16_t *x, auto hide_tag) __device__ {
        constexpr bool HIDE = decltype(hide_tag)::value;
        turn(jj);
        const uint32_t kb = k_base(lds0 + ((jj + 1) & 1) * S::BYTES), vb = v_base(lds0 + (2 + (jj & 1)) * S::BYTES);
        const float ms = reference();
        // operands held: reads run one (K) and two (V) steps ahead (one more of each
        // is 1% slower at D = 128 and the same at D = 64)
        constexpr int KA = 2, VA = 3;
        V8 ka[KA][2], va[VA], pf[4];
        auto read_k = [&](int k) __device__ {
            ka[k % KA][0] = k_frag(kb, 0, k);
            ka[k % KA][1] = k_frag(kb, 32, k);
        };
        auto read_v = [&](int i) __device__ { va[i % VA] = v_frag(vb, 16 * (i / CB), i % CB); };
#pragma unroll
        for (int k = 0; k < KA - 1; ++k) read_k(k);
        x[0] = x[1] = f32x16_t{};
        constexpr int EPS = 32 / KS;  // probabilities a step
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            if (k + KA - 1 < KS) read_k(k + KA - 1);
            if (k + VA - 1 >= KS) read_v(k + VA - 1 - KS);
            x[0] = mma32(ka[k % KA][0], qf[k], x[0]);
            x[1] = mma32(ka[k % KA][1], qf[k], x[1]);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < EPS; ++i) {
                const int e = k * EPS + i;
                const float pr = fast_exp2(__builtin_fmaf(y[e >> 4][e & 15], cs, -ms));
                sum += pr;
                pf[e >> 3][e & 7] = E(pr);
            }
            l += sum;
            __builtin_amdgcn_sched_barrier(0);
        }
        constexpr int NP = 4 * CB;  // products with V
        float mx = kNegInf;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if (i + VA - 1 < NP) read_v(i + VA - 1);
            o[i % CB] = mma32(va[i % VA], pf[i / CB], o[i % CB]);
            if constexpr (!HIDE) {
#pragma unroll
                for (int r = i * 16 / NP; r < (i + 1) * 16 / NP; ++r) mx = fmaxf(fmaxf(x[0][r], x[1][r]), mx);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (HIDE) {
            hide(jj + 1, x);
            raise(largest(x), x);
        } else {
            raise(lowered<T>(max_x32(mx) * p.c, kLift), x);
        }
    };
    // The tiles from j on one after another (CAREFUL: with every one looked over).
    auto walk = [&](int j, auto careful_tag) __device__ __attribute__((always_inline)) {
        constexpr bool CAREFUL = decltype(careful_tag)::value;
        for (; j < ntile; ++j) {
            turn(j);
            const int t = j * kKeys;
            const uint32_t vbuf = lds0 + (2 + (j & 1)) * S::BYTES;
            // A V row that some queries must not see is harmless where it is finite,
            // as their probabilities are zero.  The workgroup looks its tile over,
            // a share a thread, for the rest.
            bool bad = false;
            if (CAREFUL || t + kKeys > gmin) {
                uint32_t top = 0;
                bool infinite = false;
#pragma unroll
                for (int i = 0; i < SH::LPT; ++i) {
                    const u32x4v_t w = lds_read<u32x4v_t>(vbuf + ((i * NW + wave) * 64 + lane) * 16);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        top = max_u16x2(top, w[q] & 0x7fff7fffu);
                        if constexpr (CAREFUL) infinite |= has_infinity<T>(w[q]);
                    }
                }
                const uint32_t inf = T::kInf;
                bool odd = (top & 0xffffu) >= inf || (top >> 16) >= inf;
                if (CAREFUL && t + kKeys <= gmin) odd = infinite;  // NaN that all see need no care
                if (__any(odd) && lane == 0) found_bad = j + 1;
                wg_barrier();
                bad = found_bad == j + 1;
            }
            if (t >= wmax) {
                // none of the wave's queries sees the tile, and s still holds an earlier one's
                // scores: they must not enter the sums again
                if (bad) clean(vbuf);
                continue;
            }
            if (bad) {
                give_bad_shares(t, vbuf);
                clean(vbuf);
            }
            const float ms = reference();
            V8 pf[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) probabilities(s, ms, f, pf[f]);
            const uint32_t vb = v_base(vbuf);
#pragma unroll
            for (int f = 0; f < 4; ++f) product(vb, pf, f);
            if (j + 1 < ntile && t + kKeys < wmax) {
                scores(j + 1, s);
                hide(j + 1, s);
                raise(largest(s), s);
            }
        }
    };
    // tiles that every query of the workgroup sees whole, then the rest
    const int nfull = min(max(gmin, 0) / kKeys, ntile);
    int j = 0;
    {
        f32x16_t x[2];
        for (; j + 2 < nfull; j += 2) {
            step(j, s, x, std::false_type{});
            step(j + 1, x, s, std::false_type{});
        }
        for (; j < nfull && j + 1 < ntile; ++j) {
            step(j, s, x, std::true_type{});
            s[0] = x[0];
            s[1] = x[1];
        }
    }
    walk(j, std::false_type{});

    l = sum_x32(l);
    // A small enough float16 probability is zero, and 0 * inf is NaN where the row
    // should be infinite.  A workgroup that finds NaN beside a good sum walks its
    // tiles again, all of them looked over.  (bfloat16 has the range of the sums.)
    if constexpr (std::is_same<T, TypeF16>::value) {
        bool nan = false;
#pragma unroll
        for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r) nan |= o[c][r] != o[c][r];
        if (__any(nan && is_finite(l) && qi < nq) && lane == 0) found_nan = 1;
        wg_barrier();  // and every wave is done with the tiles
        if (found_nan) {
            issue_k(0);
            issue_v(0);
            vm_wait<SH::LPT>();
            wg_barrier();
            if (ntile > 1) issue_k(1);
            begin();
            walk(0, std::true_type{});
            l = sum_x32(l);
        }
    }
    if (parts > 1) {
        if (qi >= nq) return;
        const long long part = (long long)unit * p.nsplit + split;
        const int q = wave * 32 + n;
        float *dst = p.w.o + (part * SH::QB + q) * D + 4 * h;
#pragma unroll
        for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                *reinterpret_cast<f32x4_t *>(dst + 32 * c + 2 * r) = f32x4_t{o[c][r], o[c][r + 1], o[c][r + 2], o[c][r + 3]};
        if (h == 0) {
            p.w.ml[part * 2 * SH::QB + q] = m;
            p.w.ml[part * 2 * SH::QB + SH::QB + q] = l;
        }
        return;
    }
    // out = o / l (zeros where nothing is visible), by way of LDS: a lane holds
    // pieces of a row, the stores are whole rows
    const int at = (q0 + qrow) * a.n_heads + kvh * p.G + qhead;
    if (a.lse && h == 0 && qi < nq) a.lse[at] = lse_of(m, l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const uint32_t rows_at = lds0 + wave * 32 * S::RB;
    typedef E e4_t __attribute__((ext_vector_type(4)));
    wg_barrier();  // every wave is done with the tiles
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const e4_t x = l == 0.f ? e4_t{}
                                    : e4_t{E(o[c][4 * i] * inv), E(o[c][4 * i + 1] * inv), E(o[c][4 * i + 2] * inv),
                                           E(o[c][4 * i + 3] * inv)};
            lds_write(rows_at + n * S::RB + (((4 * c + i) ^ S::k_swizzle(n)) * 16) + 8 * h, x);
        }
    lds_drain();
#pragma unroll
    for (int i = 0; i < 32 * S::CPR / 64; ++i) {
        const int row = (i * 64 + lane) / S::CPR, ch = lane % S::CPR;
        const u32x4v_t x = lds_read<u32x4v_t>(rows_at + row * S::RB + ((ch ^ S::k_swizzle(row)) * 16));
        const long long dst = __shfl(at, row);
        // not read again here: non-temporal (64 prompts of 512 rows: 252 -> 248 us)
        if (wq0 + row < nq) __builtin_nontemporal_store(x, reinterpret_cast<u32x4v_t *>(static_cast<E *>(a.out) + dst * D + 8 * ch));
    }
}

// The units whose keys were split: workgroup (unit, y) merges the partials of
// 1024 / D of its queries in their order, D / 4 threads a query, eight loads in
// flight.
template <typename T, int D>
__global__ __launch_bounds__(256) void prompt_join_kernel(PromptParams p) {
    constexpr int QB = kPromptQueries, TPQ = D / 4, FLY = 8;
    const int4 unit = p.w.meta[blockIdx.x];
    const int parts = unit.x;
    if (parts <= 1) return;
    const int c4 = threadIdx.x % TPQ, q = blockIdx.y * (256 / TPQ) + threadIdx.x / TPQ;
    const int qi = unit.w * QB + q;
    if (qi >= unit.z) return;
    float m = kNegInf, l = 0.f;
    f32x4_t o = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < parts; i0 += FLY) {
        float pm[FLY], pl[FLY];
        f32x4_t po[FLY];
#pragma unroll
        for (int i = 0; i < FLY; ++i) {
            const long long part = (long long)blockIdx.x * p.nsplit + min(i0 + i, parts - 1);
            pm[i] = p.w.ml[part * 2 * QB + q];
            pl[i] = p.w.ml[part * 2 * QB + QB + q];
            po[i] = *reinterpret_cast<const f32x4_t *>(p.w.o + (part * QB + q) * D + 4 * c4);
        }
#pragma unroll
        for (int i = 0; i < FLY; ++i)
            if (i0 + i < parts) merge_partial(m, l, o, pm[i], pl[i], po[i]);
    }
    const int row = qi / p.G, kvh = blockIdx.x % p.a.n_kv_heads;
    store_row<T>(p.a.out, p.a.lse, (long long)(unit.y + row) * p.a.n_heads + kvh * p.G + (qi - row * p.G), c4, D, o, m, l);
}

template <typename T, int D>
hipError_t launch_prompt_typed(const PromptParams &p, hipStream_t s) {
    const unsigned units = unsigned(p.slots) * p.a.n_kv_heads;
    launch_kernel("prompt_attention", prompt_kernel<T, D>, dim3(units * p.nsplit), dim3(64 * kPromptWaves), s, p);
    if (p.nsplit > 1)
        launch_kernel("prompt_join", prompt_join_kernel<T, D>, dim3(units, kPromptQueries * D / 1024), dim3(256), s, p);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_prompt_dim(const PromptParams &p, hipStream_t s) {
    switch (p.a.head_dim) {
        case 64: return launch_prompt_typed<T, 64>(p, s);
        case 128: return launch_prompt_typed<T, 128>(p, s);
        default: return launch_prompt_typed<T, 256>(p, s);
    }
}

}  // namespace

// Into how many ranges the keys of a query block are cut.  A chain of T tiles
// takes about 0.8, 1.2 or 2 us a tile (D = 64, 128, 256) while there are at most
// 512 blocks (the diagonal halves most), and in proportion more beyond; a cut
// adds a launch, 5 us, and writes and reads 64 KiB a part.  The cheapest cut is
// taken; the average sequence stands for all, as lengths are on the device.
// Measured, us a call in 1 / 2 / 3 / 4 / 8 / 16 parts, > < the rule's:
//   18 rows behind 4000 keys, 8/1 heads, D = 128   39.7 /  26.1  / 21.2 /  18.8  / 14.6 / 13.8 (32 parts 14.6, > 24 <: 15.7 in another run)
//   four times 64 rows behind 2000, 32/8 heads     32.8 /  25.4  / 24.0 / >23.7< / 27.1 / 36.7
//   one prompt of 2048 rows, 8/8 heads             37.8 / >31.0< / 28.6 /  29.3  / 40.8 / 58.8
//   of 4096                                        68.5 / >59.3< / 61.7 /  65.9
//   of 1024, 32/8 heads                           >24.3</  30.5  / 35.3 /  39.3
//   of 512, 32/8 heads                            >14.9</  18.1  / 19.3 /  19.7
//   of 4096, 8/8 heads, D = 64                     49.6 / >37.9< / 38.3 /  39.0  / 53.4
//   of 2048, 16/4 heads, D = 64                   >27.6</  26.5  / 28.5 /  30.6  / 49.6
//   of 4096, 8/1 heads, D = 256                     128 / > 109< /  121 /   136  /  201
//   of 1024, 8/8 heads, D = 256                    39.3 /  32.0  />29.0</  27.1  / 40.4
//   of 2048, 16/4 heads, D = 256                  >68.4</  72.5  / 86.9 /   106  /  166
// The rule's choice is up to 14% off the best measured one where 18 rows are all
// there is to do, and up to 8% elsewhere; and it cuts nothing where a batch of
// short prompts holds a long one.
PromptPlan prompt_plan(int B, int n_rows, int n_kv_rows, int n_heads, int n_kv_heads, int head_dim) {
    PromptPlan p{};
    p.slots = int((long long)n_rows * (n_heads / n_kv_heads) / kPromptQueries + B);
    const double units = (p.slots - 0.5 * B) * n_kv_heads;  // half of the last blocks are there on average
    const double tiles = double(n_kv_rows) / B / kKeys, wide = head_dim / 128.0;
    double best = 1e30;
    for (const int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
        if (s > 1 && tiles < s * kMinTiles) break;
        const double cost = (0.4 + 0.8 * wide) * tiles / s * std::max(1.0, units * s / 512) + (s > 1 ? 5 + 0.033 * wide * units * s : 0.0);
        if (cost < best) {
            best = cost;
            p.nsplit = s;
        }
    }
    return p;
}

PromptWork prompt_carve(void *ws, const PromptPlan &p, int n_kv_heads, int head_dim, size_t *bytes) {
    Carve c(ws);
    PromptWork w{};
    if (p.nsplit > 1) {
        const size_t units = size_t(p.slots) * n_kv_heads;
        w.meta = c.take<int4>(units);
        w.ml = c.take<float>(units * p.nsplit * 2 * kPromptQueries);
        w.o = c.take<float>(units * p.nsplit * kPromptQueries * head_dim);
    }
    if (bytes) *bytes = std::max(size_t(256), (c.off + 255) & ~size_t(255));
    return w;
}

hipError_t launch_prompt(const PromptArgs &a, const PromptPlan &plan, const PromptWork &w, hipStream_t s) {
    PromptParams p{};
    p.a = a;
    p.w = w;
    p.G = a.n_heads / a.n_kv_heads;
    p.nsplit = plan.nsplit;
    p.slots = plan.slots;
    p.c = a.scale * kLog2e;
    return a.dtype == DSPARK_BF16 ? launch_prompt_dim<TypeBf16>(p, s) : launch_prompt_dim<TypeF16>(p, s);
}

}  // namespace dspark
