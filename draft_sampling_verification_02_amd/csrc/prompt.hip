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
#include "prompt.hpp"

namespace dspark {

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
    return launch_prompt_any<false>(a, plan, w, s);
}

}  // namespace dspark
