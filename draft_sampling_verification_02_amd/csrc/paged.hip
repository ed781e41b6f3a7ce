// paged.hip -- attention of a few new rows a request over a paged key-value
// cache (the target forward of a verify step, a decoding step, the parallel
// stage of a draft).
//
// For row i of request b (position start_b + i) and head h:
//   s_t = scale q . k_t over the visible tokens t (t <= start_b + i if causal,
//   every token of the request otherwise),
//   out = sum_t exp(s_t - lse) v_t,  lse = log sum_t exp(s_t).
// One pass over the cache carries the running maximum and sum; everything is
// accumulated in 32 bits, and the probabilities are rounded to 16 bits (by up to
// 2^-8 of each for bfloat16, 2^-11 for float16) only as they enter the V product:
// outputs are 2.0e-3 from the definition on average, 1.6e-3 of it their own
// rounding (float16: 2.3e-4 and 2.0e-4).
//
// What bounds it: the cache is read once, 4 D bytes (2 D + 2 in 8 bits) a
// token and head against 4 D G flops for G queries -- memory, for any group a
// request of a round has.  So the kernel is built to keep loads in flight: a
// workgroup of four independent waves, each streaming tiles of 32 tokens
// through an LDS buffer of its own with direct loads (no registers held, no
// barriers), K refilled as soon as its scores are taken, V as soon as its
// product is; two to three workgroups share a compute unit, so that one wave's
// arithmetic runs under the others' loads.  (Two tiles a wave in flight and
// half the workgroups measured the same for single rows, and 470 against 413 us
// for the verify rows of 256 requests, whose arithmetic is longer.)  G query
// heads times the request's rows share every tile.
//
// Work is the concatenation of all (request, head, query group) segments, cut
// into units of 128 tokens and dealt to the workgroups in equal contiguous
// ranges, whatever the requests' lengths (each workgroup finds its range from
// the lengths on the device, so a captured call follows them).  A range may
// start or end inside a segment: it then leaves a partial result (maximum, sum,
// unnormalised product), and paged_join merges a segment's partials in an
// order that the split alone fixes, so results do not depend on timing.  Short
// tables are not split: a workgroup takes whole segments, and one launch does.
//
// Measured (MI355X; 32 query and 8 key-value heads, D = 128, pages of 16):
// 256 requests, one row, 16 to 8192 tokens, bfloat16: 726 us for 4.20 GB,
// 5.8 TB/s (no LDS bank conflicts); the same with 1 to 6 rows and up to 4096
// tokens 406 us for 2.05 GB, 5.0 TB/s; four requests of 60,000 to 131,000 tokens
// over 8 bits, 64 query heads: 119 us for 620 MB, 5.2 TB/s; one request of 500
// tokens 10 us, of 8000 tokens 11 + 4 us, where the chain of dependent loads
// (lengths, page, tile) is what there is to wait for: 7 us with a single token.
#include <algorithm>

#include "attend.hpp"
#include "dspark.h"
#include "internal.hpp"

namespace dspark {

namespace {

constexpr int kTokens = 32;       // tokens of a wave's tile
constexpr int kUnit = 128;        // tokens of a work unit: a tile for each of four waves
constexpr int kMinUnits = 2;      // units a workgroup takes at least
// Tables up to kWholeTokens are not split: a workgroup walks whole segments, of
// eight waves where there are at most kFewSegments of them.  Measured, us a call
// (32/8 heads, D = 128, one row, all requests of the length; split / whole by
// four waves / by eight):
//   8 segments:    500 tokens 11.9 / 10.8 / 9.3     1000: 12.5 / 15.6 / 12.4    2000: 12.2 / 24.7 / 18.1
//   64 segments:   500        12.4 / 11.5 / 10.1    1000: 14.3 / 16.6 / 13.5    2000: 18.8 / 26.3 / 18.9
//   256 segments:  500        19.1 / 15.5 / 16.1    1000: 32.7 / 28.0 / 28.2    2000: 54.9 / 49.3 / 49.6
//   1024 segments: 500        55.1 / 52.4 / 58.1    1000: 97.0 / 93.9 / 97.3    2000: 182 / 180 / 181
// and with lengths from 16 up to 1000 tokens: 256 segments 22.1 / 18.9 / 18.1,
// 1024 segments 67.8 / 61.8 / 62.4, 2048 segments 115.9 / 120.0 / 117.3; up to
// 500: 17.6 / 12.6 / 12.1, 41.3 / 34.7 / 40.1 and 78.1 / 69.2 / 76.7.
constexpr int kWholeTokens = 1024;
constexpr int kFewSegments = 128;

typedef __attribute__((address_space(4))) const int32_t *ConstInts;  // read by scalar loads

struct PagedParams {
    PagedArgs a;
    PagedWork w;
    int G, pshift, whole;
    int unit;  // tokens of a work unit
    float c;   // scale * log2(e)
};

struct Request {
    int row0, rows;  // its rows of q
    int past;        // position of the first one
    int L;           // tokens present (0: the request takes no part)
    int groups;      // query groups
    int T;           // units of one segment
};

template <int QB>
__device__ __forceinline__ Request request_of(const PagedParams &p, int b) {
    Request r;
    const PagedArgs &a = p.a;
    int r0 = b, r1 = b + 1;
    if (a.row_offsets) {
        r0 = min(max(a.row_offsets[b], 0), a.n_rows);
        r1 = min(max(a.row_offsets[b + 1], 0), a.n_rows);
    }
    r.row0 = r0;
    r.rows = max(r1 - r0, 0);
    r.past = min(a.start[b], 1 << 30);  // tables end at 2^30 tokens: no sum below overflows
    const long long cap = (long long)a.max_pages << p.pshift;
    r.L = r.past < 0 ? 0 : int(min((long long)r.past + r.rows, cap));
    r.groups = (r.rows * p.G + QB - 1) / QB;
    r.T = p.whole ? 1 : max(1, (r.L + p.unit - 1) / p.unit);
    return r;
}
// its units, over all heads and groups (the unit is chosen so that all fit 31 bits)
__device__ __forceinline__ int cost_of(const PagedParams &p, const Request &r) { return r.groups * p.a.n_kv_heads * r.T; }

// Layout of a wave's LDS tiles: rows of RB bytes in CPR chunks of 16, chunk c
// of row r at c ^ k_swizzle(r) (K) or c ^ v_swizzle(r) (V).  K is read 16 rows
// at one chunk, V transposed 4 rows (16-bit) or 8 rows (8-bit) of each of two
// lane groups at one 32- or 16-byte column: the swizzles put those in distinct
// banks.
template <bool E4, int D>
struct TileShape {
    static constexpr int RB = E4 ? D : 2 * D;
    static constexpr int CPR = RB / 16;
    static constexpr int BYTES = kTokens * RB;
    static constexpr int NI = BYTES / 1024;       // load instructions of a tile
    static constexpr int RPI = 1024 / RB;         // rows one of them covers (at most 16)
    static constexpr int PER = RB >= 256 ? 1 : 256 / RB;  // rows that span all banks
    static constexpr int SW = CPR < 16 ? CPR : 16;
    __device__ static __forceinline__ int k_swizzle(int r) { return (r / PER) & (SW - 1); }
    __device__ static __forceinline__ int v_swizzle(int r) {
        if constexpr (E4) {
            // rows 4 g .. 4 g + 3 and 16 + 4 g .. of two neighbouring g: bits 0-2 and 4
            constexpr int low = 8 / PER;  // distinct values of the low bits after PER rows share a line
            return ((r & 7) / PER) | (((r >> 4) & 1) * low);
        } else {
            return (((r & 7) / PER) * 2) & (SW - 1);
        }
    }
};

template <typename T, bool E4>
struct ProbType {
    using type = T;
};
template <typename T>
struct ProbType<T, true> {
    // 8-bit caches: the V scales multiply the probabilities, whose range then
    // needs bfloat16's exponent
    using type = TypeBf16;
};
// float16 rows over an 8-bit cache: bfloat16 would leave the probabilities
// three bits short of the rows' own rounding, so a second bfloat16 carries the
// rest of each (2^-16 in all) through a second product (the verify rows of 256
// requests, up to 4096 tokens, D = 128: 268 us, 258 for bfloat16 rows)
template <typename T, bool E4>
constexpr bool kTwoTerms = E4 && std::is_same<T, TypeF16>::value;

// float16 probabilities are held up to 2^14 times as large: relative to the
// largest, float16 then keeps its eleven bits down to 2^-28 instead of 2^-14,
// where a long cache's many small shares would be lost.
constexpr float kLift = 14.f;

// LDS of a workgroup of nw waves and how many share a compute unit.
constexpr int paged_body(bool e4, int d, int nq, int nw) {
    const int ring = nw * (2 * kTokens * (e4 ? d : 2 * d) + (e4 ? 256 : 0));
    const int join = nw * 16 * nq * (d + 6) * 4;
    return ring > join ? ring : join;
}
constexpr int paged_per_cu(bool e4, int d, int nq, int nw) {
    const int fit = 163840 / (paged_body(e4, d, nq, nw) + 16 * nq * d * 2 + 128);
    const int eu = nq == 1 && d <= 128 ? 3 : (nq <= 2 && d <= 128) || (nq == 4 && d == 64) ? 2 : 1;  // waves a SIMD, by registers
    const int most = eu * 4 / nw;
    return fit < most ? fit : most;
}

template <bool E4, int D, int NQ, int NW>
struct PagedShape {
    using S = TileShape<E4, D>;
    static constexpr int QB = 16 * NQ;
    static constexpr int SCALE = E4 ? 256 : 0;                // a tile's scales
    static constexpr int RING = 2 * S::BYTES + SCALE;         // bytes of a wave: K tile, V tile, scales
    static constexpr int OROW = D + 4;                        // padded floats of a joined row
    static constexpr int QBYTES = QB * D * 2;
    static constexpr int BODY = paged_body(E4, D, NQ, NW);    // the waves' tiles, or their results to be joined
    static constexpr int LDS = BODY + QBYTES;
    static constexpr int KL = S::NI + (E4 ? 1 : 0);           // loads of a tile's K (and scales)
    static constexpr int VL = S::NI;
    static constexpr int PER_CU = paged_per_cu(E4, D, NQ, NW);
    static constexpr int EU = PER_CU * NW / 4;                // waves a SIMD
    static_assert(PER_CU >= 1, "a workgroup fits a compute unit");
    static_assert(LDS <= 160 * 1024, "LDS of a workgroup");
};

template <typename T, bool E4, int D, int NQ, int NW>
__global__ __launch_bounds__(64 * NW, (PagedShape<E4, D, NQ, NW>::EU)) void paged_kernel(PagedParams p) {
    using SH = PagedShape<E4, D, NQ, NW>;
    constexpr int NT = 64 * NW;
    using S = TileShape<E4, D>;
    using V8 = typename T::V8;
    using PT = typename ProbType<T, E4>::type;
    using P8 = typename PT::V8;
    using QS = TileShape<false, D>;  // query rows in LDS are laid out as 16-bit K rows
    constexpr int QB = SH::QB, KS = D / 32, CB = D / 16;
    constexpr int KSTEP = S::RB / 64;  // 16-byte chunks of a K row a lane reads
    __shared__ __attribute__((aligned(1024))) uint8_t lds[SH::LDS];
    __shared__ int scan[NW];
    __shared__ int found[8];

    const PagedArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n = lane & 15, g = lane >> 4;
    const uint32_t lds0 = lds_addr(lds);
    const uint32_t ring = lds0 + wave * SH::RING;
    const uint32_t qlds = lds0 + SH::BODY;

    // ---- this workgroup's range of units, and the request it starts in -----
    // (one round of loads where a thread has one request)
    Request rq{};
    int mine = 0, all = 0;
    for (int i = tid; i < a.B; i += NT) {
        rq = request_of<QB>(p, i);
        mine = cost_of(p, rq);
        all += mine;
    }
    auto total_of = [&](int x) __device__ {  // over the workgroup; inclusive sums of x stay in `inc`
        int inc = x;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(inc, d);
            if (lane >= d) inc += up;
        }
        __syncthreads();
        if (lane == 63) scan[wave] = inc;
        __syncthreads();
        int sum = 0;
        for (int w = 0; w < NW; ++w) {
            if (w == wave) inc += sum;
            sum += scan[w];
        }
        return make_int2(inc, sum);
    };
    int2 sums = total_of(all);
    const int total = uniform(sums.y);
    const int per = max(int((unsigned(total) + gridDim.x - 1) / gridDim.x), p.whole ? 1 : kMinUnits);
    const int begin = int(min((long long)blockIdx.x * per, (long long)total)), end = int(min((long long)begin + per, (long long)total));
    if (tid == 0 && !p.whole) p.w.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (begin < 0 || begin >= end) return;
    if (tid == 0) found[0] = -1;
    __syncthreads();
    int before = 0;  // units of the requests before this chunk of NT
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        const int i = b0 + tid;
        if (a.B > NT) {
            mine = 0;
            if (i < a.B) {
                rq = request_of<QB>(p, i);
                mine = cost_of(p, rq);
            }
            sums = total_of(mine);
        }
        const int past_it = before + sums.x;
        if (i < a.B && begin < past_it && begin >= past_it - mine) {
            found[0] = i;
            found[1] = past_it - mine;
            found[2] = rq.row0;
            found[3] = rq.rows;
            found[4] = rq.past;
            found[5] = rq.L;
            found[6] = rq.groups;
            found[7] = rq.T;
        }
        before += sums.y;
        if (begin < before) break;
    }
    __syncthreads();
    int b = uniform(found[0]);
    if (b < 0) return;
    rq = Request{uniform(found[2]), uniform(found[3]), uniform(found[4]), uniform(found[5]), uniform(found[6]), uniform(found[7])};
    int at = begin;
    const int rest = begin - uniform(found[1]);      // units into the request
    int seg = uniform(int(unsigned(rest) / unsigned(rq.T)));  // (head, group) segment of the request
    int u0 = rest - seg * rq.T;

    // Fixed parts of the load and read addresses.  The swizzles are XORs of
    // chunk bits with row bits, so load j's offset is the first load's with
    // constant bits flipped, and so is a step's read address; they are made
    // anew where they are used, as registers are short.
    uint32_t kload, vload;
    {
        const int rin = lane / S::CPR, c = lane % S::CPR;  // row of the load, chunk
        kload = rin * S::RB + ((c ^ S::k_swizzle(rin)) * 16);
        vload = rin * S::RB + ((c ^ S::v_swizzle(rin)) * 16);
    }
    const uint32_t kread = n * S::RB + ((g ^ S::k_swizzle(n)) * 16);
    // transposing reads: 16-bit, row 4 g + i of a half; 8-bit, rows 4 g + i of both halves
    const int vrow = E4 ? ((lane >> 1) & 3) + 4 * g + ((lane & 8) ? 16 : 0) : 4 * g + ((lane >> 2) & 3);
    const uint32_t vread = vrow * S::RB + (((E4 ? 0 : (lane >> 1) & 1) ^ S::v_swizzle(vrow)) * 16) + 8 * (lane & 1);
    auto v_frag = [&](uint32_t base, int cb) __device__ {
        if constexpr (E4) {
            P8 f;
            e4m3_to8(lds_read_tr8(base ^ (16 * cb)), f);
            return f;
        } else {
            return join4<P8>(lds_read_tr16(base ^ (32 * cb)), lds_read_tr16(base ^ (32 * cb), 16 * S::RB));
        }
    };

    while (at < end) {
        // ---- one segment: query group grp of head h of request b ---------
        const int h = uniform(seg / rq.groups), grp = uniform(seg - h * rq.groups);
        const int u1 = uniform(min(rq.T, u0 + (end - at)));
        const int tok0 = p.whole ? 0 : u0 * p.unit;
        const int tok1 = p.whole ? rq.L : int(min((long long)u1 * p.unit, (long long)rq.L));
        const int nq_all = rq.rows * p.G;  // queries of the request
        // this wave's tiles: tok0 + (wave + NW i) * kTokens
        const int ntile = (max(tok1 - tok0, 0) + kTokens - 1) / kTokens;
        const int tiles = uniform(ntile > wave ? (ntile - wave + NW - 1) / NW : 0);
        const ConstInts table = (ConstInts)(a.page_table + (long long)b * a.max_pages);
        const int pmask = (1 << p.pshift) - 1;

        auto tile_at = [&](int i) __device__ { return tok0 + (wave + i * NW) * kTokens; };
        // the page of token t (the last page of the table for tokens past it: they are masked)
        auto page_of = [&](int t) __device__ { return table[min(t >> p.pshift, a.max_pages - 1)]; };
        auto bad_page = [&](int page) __device__ { return page < 0 || page >= a.n_pages; };
        // row of the cache where tokens t .. t + 15 start; a page outside the cache reads page 0 and is masked
        auto row_of = [&](int page, int t) __device__ {
            return (((long long)(bad_page(page) ? 0 : page) * a.n_kv_heads + h) << p.pshift) + (t & pmask);
        };
        auto issue = [&](const void *cache, auto swizzle, uint32_t off, uint32_t dst, int t, int pa, int pb) __device__ {
            const uint8_t *ba = static_cast<const uint8_t *>(cache) + row_of(pa, t) * S::RB;
            const uint8_t *bb = static_cast<const uint8_t *>(cache) + row_of(pb, t + 16) * S::RB;
#pragma unroll
            for (int j = 0; j < S::NI; ++j) {
                const int row = j * S::RPI;  // first row of the load; a load stays in one half, so in one page
                dma16(uniform(dst + j * 1024), off ^ (swizzle(row) * 16), uniform((row < 16 ? ba : bb) + (row & 15) * S::RB));
            }
        };
        auto issue_k = [&](int i, int pa, int pb) __device__ {
            const int t = tile_at(i);
            issue(a.k_cache, S::k_swizzle, fresh(kload), ring, t, pa, pb);
            if constexpr (E4) {
                // bytes 0-31: K scales of the tokens, 32-63: V scales (lane i brings 4 bytes; lanes past 15 repeat)
                const uint8_t *sc = (lane & 8) ? a.v_scale : a.k_scale;
                dma4(uniform(ring + 2 * S::BYTES), sc + ((lane & 4) ? row_of(pb, t + 16) : row_of(pa, t)) + 4 * (lane & 3));
            }
        };
        auto issue_v = [&](int i, int pa, int pb) __device__ {
            issue(a.v_cache, S::v_swizzle, fresh(vload), ring + S::BYTES, tile_at(i), pa, pb);
        };

        // ---- queries into LDS (the workgroup's waves share them), first tiles
        constexpr int QCH = D / 8;  // 16-byte chunks of a query row
        for (int j = wave; j < SH::QBYTES / 1024; j += NW) {
            const int slot = j * 64 + lane, row = slot / QCH;
            const int qi = min(grp * QB + row, nq_all - 1);
            const int i = qi / p.G;
            const long long src = (rq.row0 + i) * a.q_stride + (long long)(h * p.G + (qi - i * p.G)) * D +
                                  (((slot % QCH) ^ QS::k_swizzle(row & 15)) * 8);
            dma16(uniform(qlds + j * 1024), static_cast<const uint8_t *>(a.q) + 2 * src);
        }
        int pa = 0, pb = 0, na = 0, nb = 0;  // pages of the tile at hand and of the next one
        auto issue_first = [&]() __device__ {
            if (tiles > 0) {
                pa = page_of(tile_at(0));
                pb = page_of(tile_at(0) + 16);
                issue_k(0, pa, pb);
                issue_v(0, pa, pb);
            }
            if (tiles > 1) {
                na = page_of(tile_at(1));
                nb = page_of(tile_at(1) + 16);
            }
        };
        issue_first();
        if (tiles > 0)
            vm_wait<SH::KL + SH::VL>();
        else
            vm_wait<0>();
        wg_barrier();
        V8 qf[NQ][KS];
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                // the 8 channels lane group g takes at step k (an 8-bit K chunk holds two steps')
                const int ch = E4 ? 2 * (4 * (k / 2) + g) + (k & 1) : 4 * k + g;
                qf[q][k] = __builtin_bit_cast(
                    V8, lds_read<u32x4v_t>(qlds + (16 * q + n) * D * 2 + ((ch ^ QS::k_swizzle(n)) * 16)));
            }
        int lim[NQ];  // tokens visible to the lane's query
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int qi = grp * QB + 16 * q + n;
            lim[q] = qi >= nq_all ? 0 : (a.causal ? min(rq.L, rq.past + qi / p.G + 1) : rq.L);
        }
        const int lim_min = uniform(a.causal ? min(rq.L, rq.past + (grp * QB) / p.G + 1) : rq.L);

        float m[NQ], l[NQ];
        bool far[NQ];  // the maximum of one of the 16 queries is far from zero
        f32x4_t o[NQ][CB];
        auto reference = [&](int q) __device__ { return far[q] || m[q] == kNegInf ? 0.f : m[q]; };
        auto clear = [&]() __device__ {
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                m[q] = kNegInf;
                l[q] = 0.f;
                far[q] = false;
#pragma unroll
                for (int c = 0; c < CB; ++c) o[q][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            }
        };
        clear();

        // This wave's tiles, whose first is on its way (CAREFUL: with every one looked over).
        auto walk = [&](auto careful_tag) __device__ __attribute__((always_inline)) {
            constexpr bool CAREFUL = decltype(careful_tag)::value;
            for (int i = 0; i < tiles; ++i) {
                const int t = tile_at(i);
                const int bad_now = int(bad_page(pa)) | int(bad_page(pb)) << 1;  // the tile's halves on pages outside the cache
                const bool more = i + 1 < tiles;
                int fa = 0, fb = 0;  // pages of the tile after next, on their way
                if (i + 2 < tiles) {
                    fa = page_of(tile_at(i + 2));
                    fb = page_of(tile_at(i + 2) + 16);
                }
                // ---- scores: s[q][half][r] is token 16 half + 4 g + r, query n
                vm_wait<SH::VL>();
                const uint32_t kbase = fresh(ring + kread);
                f32x4_t s[NQ][2];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q) s[q][hf] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < KSTEP; ++k) {
                        const u32x4v_t x = lds_read<u32x4v_t>(kbase ^ (64 * k), 16 * hf * S::RB);
                        if constexpr (E4) {
                            V8 lo, hi;
                            e4m3_to8(u32x2_t{x[0], x[1]}, lo);
                            e4m3_to8(u32x2_t{x[2], x[3]}, hi);
#pragma unroll
                            for (int q = 0; q < NQ; ++q) s[q][hf] = mma16(lo, qf[q][2 * k], s[q][hf]);
#pragma unroll
                            for (int q = 0; q < NQ; ++q) s[q][hf] = mma16(hi, qf[q][2 * k + 1], s[q][hf]);
                        } else {
#pragma unroll
                            for (int q = 0; q < NQ; ++q)
                                s[q][hf] = mma16(__builtin_bit_cast(V8, x), qf[q][k], s[q][hf]);
                        }
                    }
                }
                float vs[2][4];
                if constexpr (E4) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint32_t kw = lds_read<uint32_t>(ring + 2 * S::BYTES + 16 * hf + 4 * g);
                        const uint32_t vw = lds_read<uint32_t>(ring + 2 * S::BYTES + 32 + 16 * hf + 4 * g);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float ks = scale_of((kw >> (8 * r)) & 255);
                            vs[hf][r] = scale_of((vw >> (8 * r)) & 255);
#pragma unroll
                            for (int q = 0; q < NQ; ++q) s[q][hf][r] *= ks;
                        }
                    }
                }
                lds_drain();
                if (more) issue_k(i + 1, na, nb);

                // ---- running maximum, probabilities
                const bool masked = t + kTokens > lim_min || bad_now != 0;
                P8 pf[NQ], pr_rest[kTwoTerms<T, E4> ? NQ : 1];
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    if (masked) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (t + 16 * hf + 4 * g + r >= lim[q] || ((bad_now >> hf) & 1)) s[q][hf][r] = kNegInf;
                    }
                    float mx = fmaxf(fmaxf(fmaxf(s[q][0][0], s[q][0][1]), fmaxf(s[q][0][2], s[q][0][3])),
                                     fmaxf(fmaxf(s[q][1][0], s[q][1][1]), fmaxf(s[q][1][2], s[q][1][3])));
                    mx = lowered<PT>(max_x16(max_x32(mx)) * p.c, kLift);
                    const float mn = fmaxf(m[q], mx);
                    if (__any(mn > m[q])) {
                        const float al = fast_exp2(m[q] - (mn == kNegInf ? 0.f : mn));
                        l[q] *= al;
#pragma unroll
                        for (int c = 0; c < CB; ++c) o[q][c] *= al;
                        m[q] = mn;
                        far[q] = __any(is_far(mn));
                    }
                    if (far[q]) {  // scores far from zero become exponents at once
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                            for (int r = 0; r < 4; ++r) s[q][hf][r] = far_exponent(s[q][hf][r], p.c, mn);
                    }
                    const float ms = reference(q), cs = far[q] ? 1.f : p.c;
                    float pr[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) pr[e] = fast_exp2(__builtin_fmaf(s[q][e >> 2][e & 3], cs, -ms));
                    l[q] += ((pr[0] + pr[1]) + (pr[2] + pr[3])) + ((pr[4] + pr[5]) + (pr[6] + pr[7]));
                    if constexpr (E4) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            // a masked token's scale may be anything: its product stays zero
                            const float x = pr[e] * vs[e >> 2][e & 3];
                            pr[e] = masked && s[q][e >> 2][e & 3] == kNegInf ? 0.f : x;
                        }
                    }
                    using E = typename PT::E;
                    pf[q] = P8{E(pr[0]), E(pr[1]), E(pr[2]), E(pr[3]), E(pr[4]), E(pr[5]), E(pr[6]), E(pr[7])};
                    if constexpr (kTwoTerms<T, E4>) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) pr_rest[q][e] = E(pr[e] - float(pf[q][e]));
                    }
                }

                // ---- products with V
                if (more)
                    vm_wait<SH::KL>();
                else
                    vm_wait<0>();
                const uint32_t vbuf = ring + S::BYTES;
                const uint32_t vbase = fresh(vbuf + vread);
                if (CAREFUL || masked) {
                    // rows that no query sees (past the request's end, pages outside the cache) may hold anything
#pragma unroll 1
                    for (int slot = lane; slot < kTokens * S::CPR; slot += 64) {
                        const int row = slot / S::CPR;
                        if (t + row >= rq.L || ((bad_now >> (row >> 4)) & 1)) lds_write(vbuf + slot * 16, u32x4v_t{0, 0, 0, 0});
                    }
                    lds_drain();
                    // A row that some queries see and others must not is harmless where it is finite, as the others'
                    // probabilities are zero; 0 * v tells.  What is not finite is taken out of the tile: the queries
                    // that see it get their share of it here.  (The share's probability is taken anew in 32 bits: rounded
                    // to float16 it may be zero, and 0 * inf is NaN.  8-bit values that are not finite are NaN anyway.)
                    if (CAREFUL || (t + kTokens > lim_min && lim_min < rq.L)) {
                        bool odd = false;
                        if (CAREFUL && !masked) {  // NaN that all see need no care
#pragma unroll 1
                            for (int slot = lane; slot < kTokens * S::CPR; slot += 64) {
                                const u32x4v_t w = lds_read<u32x4v_t>(vbuf + slot * 16);
#pragma unroll
                                for (int x = 0; x < 4; ++x) odd |= has_infinity<T>(w[x]);
                            }
                        } else {
                            const P8 zero = {};
                            f32x4_t z = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int c = 0; c < CB; ++c) z = mma16(v_frag(vbase, c), zero, z);
                            odd = !(z[0] == 0.f && z[1] == 0.f && z[2] == 0.f && z[3] == 0.f);
                        }
                        if (__any(odd)) {
#pragma unroll 1
                            for (int k = 0; k < kTokens; ++k) {
                                // token k is element e of lane group (k / 4) % 4; the lane holds channels 16 c + 4 g ..
                                const int e = (k & 3) + 4 * (k >> 4), from = ((k >> 2) & 3) * 16 + n;
                                const uint32_t row = vbuf + k * S::RB + (E4 ? 4 * g : 8 * (g & 1));
                                const int sw = S::v_swizzle(k);
#pragma unroll
                                for (int q = 0; q < NQ; ++q) {
                                    float pk = 1.f;
                                    if constexpr (!E4) {
                                        float score = 0.f;
#pragma unroll
                                        for (int x = 0; x < 8; ++x) score = x == e ? s[q][x >> 2][x & 3] : score;
                                        pk = __shfl(fast_exp2(__builtin_fmaf(score, far[q] ? 1.f : p.c, -reference(q))), from);
                                    }
                                    const bool sees = t + k < lim[q];
#pragma unroll
                                    for (int c = 0; c < CB; ++c) {
                                        asm volatile("" : : : "memory");  // read four values at a time: registers are short
                                        float v[4];
                                        if constexpr (E4)
                                            e4m3_to4(lds_read<uint32_t>(row + ((c ^ sw) * 16)), v);
                                        else
                                            widen4<T>(lds_read<u32x2_t>(row + (((2 * c + (g >> 1)) ^ sw) * 16)), v);
                                        if (__any(sees && !(is_finite(v[0]) && is_finite(v[1]) && is_finite(v[2]) && is_finite(v[3])))) {
#pragma unroll
                                            for (int r = 0; r < 4; ++r)
                                                o[q][c][r] += sees && !is_finite(v[r]) ? pk * v[r] : 0.f;
                                        }
                                    }
                                }
                            }
                            lds_drain();
#pragma unroll 1
                            for (int slot = lane; slot < kTokens * S::CPR; slot += 64) {
                                u32x4v_t w = lds_read<u32x4v_t>(vbuf + slot * 16);
#pragma unroll
                                for (int x = 0; x < 4; ++x) w[x] = E4 ? finite_e4m3(w[x]) : finite_pair<T>(w[x]);
                                lds_write(vbuf + slot * 16, w);
                            }
                            lds_drain();
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < CB; ++c) {
                    const P8 vf = v_frag(vbase, c);
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        o[q][c] = mma16(vf, pf[q], o[q][c]);
                        if constexpr (kTwoTerms<T, E4>) o[q][c] = mma16(vf, pr_rest[q], o[q][c]);
                    }
                }
                lds_drain();
                if (more) issue_v(i + 1, na, nb);
                pa = na;
                pb = nb;
                na = fa;
                nb = fb;
            }
        };
        walk(std::false_type{});
        // A small enough float16 probability is zero, and 0 * inf is NaN where the
        // row should be infinite.  A wave that finds NaN beside good sums walks its
        // tiles again, all of them looked over.  (bfloat16 has the range of the sums.)
        if constexpr (!E4 && std::is_same<T, TypeF16>::value) {
            bool nan = false;
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int c = 0; c < CB; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r) nan |= lim[q] > 0 && o[q][c][r] != o[q][c][r] && is_finite(l[q]);
            if (__any(nan)) {
                issue_first();
                clear();
                walk(std::true_type{});
            }
        }

        // ---- the waves' results through LDS ------------------------------
        wg_barrier();
        const uint32_t jml = lds0 + NW * QB * SH::OROW * 4;  // [wave][QB][2]: maximum, sum
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            l[q] = sum_x16(sum_x32(l[q]));
            const int row = wave * QB + 16 * q + n;
            if (g == 0) lds_write(jml + row * 8, u32x2_t{__float_as_uint(m[q]), __float_as_uint(l[q])});
#pragma unroll
            for (int c = 0; c < CB; ++c) lds_write(lds0 + (row * SH::OROW + 16 * c + 4 * g) * 4, o[q][c]);
        }
        wg_barrier();
        const bool starts = u0 == 0, ends = u1 == rq.T;
        const long long slot = 2LL * blockIdx.x + (starts ? 1 : 0);
        for (int e = tid; e < QB * (D / 4); e += NT) {
            const int q = e / (D / 4), c4 = e % (D / 4);
            const int qi = grp * QB + q;
            float mw[NW], lw[NW], mm = kNegInf, ll = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const u32x2_t x = lds_read<u32x2_t>(jml + (w * QB + q) * 8);
                mw[w] = __uint_as_float(x[0]);
                lw[w] = __uint_as_float(x[1]);
                mm = fmaxf(mm, mw[w]);
            }
            f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
            const float ms = mm == kNegInf ? 0.f : mm;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = fast_exp2(mw[w] - ms);
                ll += lw[w] * f;
                acc += lds_read<f32x4_t>(lds0 + ((w * QB + q) * SH::OROW + 4 * c4) * 4) * f;
            }
            if (starts && ends) {
                if (qi < nq_all) store_row<T>(a.out, a.lse, (long long)(rq.row0 + qi / p.G) * a.n_heads + h * p.G + qi % p.G, c4, D, acc, mm, ll);
            } else {
                *reinterpret_cast<f32x4_t *>(p.w.o + (slot * QB + q) * D + 4 * c4) = acc;
                if (c4 == 0) {
                    p.w.ml[slot * 2 * QB + q] = mm;
                    p.w.ml[slot * 2 * QB + QB + q] = ll;
                }
            }
        }
        if (starts && !ends && tid == 0)
            p.w.meta[blockIdx.x] = make_int4((rq.T - u1 + per - 1) / per, b, h, grp);
        wg_barrier();

        at += u1 - u0;
        u0 = 0;
        if (++seg >= rq.groups * a.n_kv_heads && at < end) {
            seg = 0;
            do {
                if (++b >= a.B) return;  // (not with offsets that do not decrease)
                rq = request_of<QB>(p, b);
            } while (rq.groups == 0);
        }
    }
}

// The segments that workgroups left unfinished: workgroup (i, y) merges KQ
// queries of the segment that workgroup i started and its successors went on
// with, in an order that the split alone fixes.  256 / KQ threads a query take
// the partials in turn, D / 4 threads each, four loads in flight.
template <typename T, int D, int QB, int KQ>
__global__ __launch_bounds__(256) void paged_join_kernel(PagedParams p) {
    constexpr int TPQ = 256 / KQ, TPP = D / 4, LANES = TPQ / TPP;  // threads a query, a partial; partials in turn
    __shared__ float red[KQ == 1 ? 4 : 1][D + 2];
    const int4 seg = p.w.meta[blockIdx.x];
    if (seg.x == 0) return;
    const Request rq = request_of<QB>(p, seg.y);
    const int lane = threadIdx.x % TPQ, q = blockIdx.y * KQ + threadIdx.x / TPQ;
    const int qi = seg.w * QB + q;
    if (qi >= rq.rows * p.G) return;  // (uniform where the waves of a query meet below)
    const int grp = lane / TPP, c4 = lane % TPP;
    const int parts = seg.x + 1;
    float m = kNegInf, l = 0.f;
    f32x4_t o = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int j0 = grp; j0 < parts; j0 += 4 * LANES) {
        float pm[4], pl[4];
        f32x4_t po[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = min(j0 + i * LANES, parts - 1);
            // partial j lies in slot 2 i + 1 (the start) or 2 (i + j)
            const long long slot = 2LL * (blockIdx.x + j) + (j == 0 ? 1 : 0);
            pm[i] = p.w.ml[slot * 2 * QB + q];
            pl[i] = p.w.ml[slot * 2 * QB + QB + q];
            po[i] = *reinterpret_cast<const f32x4_t *>(p.w.o + (slot * QB + q) * D + 4 * c4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j0 + i * LANES < parts) merge_partial(m, l, o, pm[i], pl[i], po[i]);
    }
#pragma unroll
    for (int s = TPP; s < 64; s <<= 1) {
        const float m2 = __shfl_xor(m, s), l2 = __shfl_xor(l, s);
        const f32x4_t o2 = f32x4_t{__shfl_xor(o[0], s), __shfl_xor(o[1], s), __shfl_xor(o[2], s), __shfl_xor(o[3], s)};
        merge_partial(m, l, o, m2, l2, o2);
    }
    if constexpr (KQ == 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) < TPP) {
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][4 * c4 + i] = o[i];
            if (c4 == 0) {
                red[wave][D] = m;
                red[wave][D + 1] = l;
            }
        }
        __syncthreads();
        if (threadIdx.x >= TPP) return;
        for (int w = 1; w < 4; ++w)
            merge_partial(m, l, o, red[w][D], red[w][D + 1],
                          f32x4_t{red[w][4 * c4], red[w][4 * c4 + 1], red[w][4 * c4 + 2], red[w][4 * c4 + 3]});
    }
    if (grp == 0)
        store_row<T>(p.a.out, p.a.lse, (long long)(rq.row0 + qi / p.G) * p.a.n_heads + seg.z * p.G + qi % p.G, c4, D, o, m, l);
}

template <typename T, bool E4, int D, int NQ>
hipError_t launch_paged_typed(const PagedParams &pp, const PagedPlan &plan, hipStream_t s) {
    const dim3 grid(plan.grid);
    bool done = false;
    if constexpr (paged_per_cu(E4, D, NQ, 8) >= 1)
        if (plan.waves == 8) {
            launch_kernel("paged_attention", paged_kernel<T, E4, D, NQ, 8>, grid, dim3(512), s, pp);
            done = true;
        }
    if (!done) launch_kernel("paged_attention", paged_kernel<T, E4, D, NQ, 4>, grid, dim3(256), s, pp);
    if (!plan.whole && plan.grid > 1) {
        // long runs of partials (few segments): a workgroup a query; else four
        if (plan.long_runs)
            launch_kernel("paged_join", paged_join_kernel<T, D, 16 * NQ, 1>, dim3(plan.grid - 1, 16 * NQ), dim3(256), s, pp);
        else
            launch_kernel("paged_join", paged_join_kernel<T, D, 16 * NQ, 4>, dim3(plan.grid - 1, 4 * NQ), dim3(256), s, pp);
    }
    return hipGetLastError();
}

template <typename T, bool E4, int D>
hipError_t launch_paged_queries(const PagedParams &pp, const PagedPlan &plan, hipStream_t s) {
    switch (plan.qblocks) {
        case 1: return launch_paged_typed<T, E4, D, 1>(pp, plan, s);
        case 2: return launch_paged_typed<T, E4, D, 2>(pp, plan, s);
        default:
            if constexpr (D < (E4 ? 128 : 256))
                return launch_paged_typed<T, E4, D, 4>(pp, plan, s);
            else
                return hipErrorInvalidValue;
    }
}

template <typename T, bool E4>
hipError_t launch_paged_dim(const PagedParams &pp, const PagedPlan &plan, hipStream_t s) {
    switch (pp.a.head_dim) {
        case 64: return launch_paged_queries<T, E4, 64>(pp, plan, s);
        case 128: return launch_paged_queries<T, E4, 128>(pp, plan, s);
        default: return launch_paged_queries<T, E4, 256>(pp, plan, s);
    }
}

}  // namespace

// The query blocks cover a request's rows times its group where they fit
// (16 to 64 queries; 32 at D = 256, whose accumulators are twice as long);
// more rows take several groups, which read the cache again.
PagedPlan paged_plan(const PagedSizes &z) {
    PagedPlan p{};
    const long long queries = (long long)z.max_rows * (z.n_heads / z.n_kv_heads);
    // Every block of queries walks the keys again, so the fewest blocks win until
    // the registers of 64 queries leave too few waves.  Us a call in blocks of
    // 16 / 32 / 64 queries (64 requests behind 2000 tokens, 8 key heads, D = 128):
    // 24 queries 200 / 121 / 124, 40 281 / 214 / 127, 68 448 / 304 / 228; from an
    // 8-bit cache 24 105 / 75 / 135, 40 143 / 125 / 138, 68 232 / 168 / 249, and
    // with D = 64 48 queries 84 / 87 / 75.
    const int most = z.head_dim >= (z.e4 ? 128 : 256) ? 2 : 4;
    p.qblocks = queries <= 16 ? 1 : (queries <= 32 || most == 2 ? 2 : 4);
    p.waves = 4;
    p.grid = 256 * paged_per_cu(z.e4, z.head_dim, p.qblocks, 4);
    p.whole = z.table_tokens <= kWholeTokens;
    if (p.whole && z.table_tokens > kUnit && z.requests * z.n_kv_heads <= kFewSegments &&
        paged_per_cu(z.e4, z.head_dim, p.qblocks, 8) >= 1)
        p.waves = 8;
    // no more workgroups than there can be work for
    const long long segments = z.n_rows * z.n_heads / (16 * p.qblocks) + z.requests * z.n_kv_heads;
    const long long units = p.whole ? segments : segments * ((z.table_tokens + kUnit - 1) / kUnit);
    p.grid = int(std::min<long long>(p.grid, p.whole ? units : (units + kMinUnits - 1) / kMinUnits));
    // Eight or more partials a segment: a workgroup a query, which reads them side
    // by side (one request of 32,000 tokens: join 9.2 -> 4.1 us); else four
    // queries share one (64 requests of 1 to 6 rows: 4.7 against 8.2 us).
    p.long_runs = segments * 8 <= p.grid;
    return p;
}

PagedWork paged_carve(void *ws, const PagedPlan &p, int head_dim, size_t *bytes) {
    Carve c(ws);
    PagedWork w{};
    w.meta = c.take<int4>(p.grid);
    w.ml = c.take<float>(size_t(2) * p.grid * 2 * 16 * p.qblocks);
    w.o = c.take<float>(size_t(2) * p.grid * 16 * p.qblocks * head_dim);
    if (bytes) *bytes = (c.off + 255) & ~size_t(255);
    return w;
}

hipError_t launch_paged(const PagedArgs &a, const PagedPlan &plan, const PagedWork &w, hipStream_t s) {
    PagedParams p{};
    p.a = a;
    p.w = w;
    p.G = a.n_heads / a.n_kv_heads;
    p.pshift = log2_of(a.page_size);
    p.whole = plan.whole;
    p.unit = kUnit;
    const long long segments = (long long)a.n_rows * a.n_heads / (16 * plan.qblocks) + (long long)a.B * a.n_kv_heads;  // at most
    const long long tokens = (long long)a.max_pages * a.page_size;
    while (segments * (tokens / p.unit + 1) > INT32_MAX) p.unit *= 2;
    p.c = a.scale * kLog2e;
    const bool e4 = a.cache_dtype == DSPARK_E4M3;
    if (a.dtype == DSPARK_BF16)
        return e4 ? launch_paged_dim<TypeBf16, true>(p, plan, s) : launch_paged_dim<TypeBf16, false>(p, plan, s);
    return e4 ? launch_paged_dim<TypeF16, true>(p, plan, s) : launch_paged_dim<TypeF16, false>(p, plan, s);
}

}  // namespace dspark
