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
#include "paged.hpp"

namespace dspark {

namespace {

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
constexpr int kWindowWhole = 4096;  // tokens that a window and the sinks leave

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
    // Walks behind a window end at its length, so that whole segments may load the
    // chip evenly once there are enough; but texts may be shorter, and a batch lasts
    // as long as its longest segment then.  Us a call, split / whole, 8 key heads, of
    // texts past the window; of 0 to 2 windows; one past it, the others up to 400:
    //   one row, bfloat16, D = 128, window 1500
    //     128 segments 27.3 / 17.6; 23.5 / 17.1; 15.0 / 15.7    512 65 / 64; 61 / 50; 24 / 25
    //   3000    128 36.8 / 30.0; 30.3 / 25.5; 16.3 / 23.2       512 120 / 118; 116 / 97; 25 / 39
    //   8000    128 85 / 79; 66 / 72; 23 / 49                   512 319 / 314; 260 / 249; 31 / 84
    //   30,000  128 307 / 334; 275 / 326; 39 / 166              512 1251 / 1246; 969 / 989; 48 / 293
    //   up to 6 rows over 8 bits, window 1500
    //     128 segments 29.7 / 25.1; 24.2 / 24.0; 20.2 / 20.1    512 48 / 45; 69 / 43; 31 / 28
    //   3000    128 31.6 / 40.8; 31.0 / 39.6; 20.1 / 38.6       512 78 / 74; 89 / 69; 28 / 47
    //   8000    128 63 / 88; 53 / 85; 25 / 65                   512 191 / 180; 150 / 164; 38 / 136
    //   the same, D = 256, window 1500
    //     128 segments 47.1 / 53.2; 42.5 / 52.3; 29.2 / 39.7    512 109 / 106; 134 / 104; 61 / 78
    if (z.window && z.table_tokens <= kWindowWhole)
        p.whole |= z.requests * z.n_kv_heads >= (z.e4 && (z.table_tokens > 2048 || z.head_dim == 256) ? 512 : 128);
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
    return launch_paged_any<false>(a, plan, w, s);
}

}  // namespace dspark
