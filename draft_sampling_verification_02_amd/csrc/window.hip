// window.hip -- attention over a paged key-value cache through a sliding window,
// with a few first tokens (sinks) that stay visible.
//
// For row i of request b (position p = start_b + i) and head h:
//   s_t = scale q . k_t over t <= p with p - t < window or t < sinks,
//   out = sum_t exp(s_t - lse) v_t,  lse = log sum_t exp(s_t).
// What no row sees is not read, and its pages may be gone.
//
// Few rows a request (decoding, verification) go through the kernel of paged
// attention (paged.hpp, window_rows.hip): bound by memory; its walk leaves out the tokens between the
// sinks and the first row's window.  Chunks of rows go through the kernel of prompt
// attention (prompt.hpp): bound by the matrix units; each block of 128 queries
// walks the sinks and its own window, the tiles that all its queries see whole in
// the pipelined loop, and those where windows begin or end beside it; keys and
// values come out of their pages by scalar loads of the page ids, one tile ahead.
//
// Measured (MI355X, 32/8 heads, D = 128): rows: 256 requests, window 1024, bfloat16
// 193-202 us (1.07 GB, 5.3 to 5.5 TB/s); up to 6 rows of 128 requests, window 2048, 8 bits
// 112-126 us (510 MB, 4.1 to 4.5 TB/s).  Chunks: eight of 300 to 2048 rows, window 4096
// and 64 sinks, 548-612 us, 845 to 940 TFLOP/s of what rows see, over 8 bits 678-724;
// matrix units busy 46% of 1.8 GHz, a compute unit 90% of the call.  float16 rows of the
// same sizes: rows 200 us, over 8 bits 115 (one row, 256 requests) and 123 (up to 6,
// 128); chunks 609, over 8 bits, where the rows' kernel takes them, 2152.
//
// Probabilities are rounded to 16 bits for the product with V (the operand of the matrix
// instructions), sums and maxima are not.  Errors against 64 bits, relative and root mean
// square: bfloat16 rows 0.0020, chunks 0.0024 (whose largest share need not be 1, so that
// it is rounded too), where the outputs' own rounding alone makes 0.0017; float16 0.00026
// and 0.00029 of 0.00021, over 8 bits, in two bfloat16 terms, no more than that.
#include "prompt.hpp"

namespace dspark {

// As prompt_plan, with kv_tokens walked by every block.  No more than kWindowParts
// parts are written, so that a workspace of one size does for all batches.
PromptPlan window_chunk_plan(int B, int n_rows, long long kv_tokens, int n_heads, int n_kv_heads, int head_dim) {
    PromptPlan p{};
    p.slots = int((long long)n_rows * (n_heads / n_kv_heads) / kPromptQueries + B);
    p.nsplit = 1;
    const double units = (p.slots - 0.5 * B) * n_kv_heads;
    const double tiles = double(kv_tokens) / kKeys, wide = head_dim / 128.0;
    double best = 1e30;
    for (const int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
        if (s > 1 && (tiles < s * kMinTiles || (long long)p.slots * n_kv_heads * s > kWindowParts)) break;
        const double cost = (0.4 + 0.8 * wide) * tiles / s * std::max(1.0, units * s / 512) + (s > 1 ? 5 + 0.033 * wide * units * s : 0.0);
        if (cost < best) {
            best = cost;
            p.nsplit = s;
        }
    }
    return p;
}

hipError_t launch_window_chunks(const PromptArgs &a, const PromptPlan &plan, const PromptWork &w, hipStream_t s) {
    return launch_prompt_any<true>(a, plan, w, s);
}

}  // namespace dspark
