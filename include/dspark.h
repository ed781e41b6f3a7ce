/*
 * dspark.h -- C ABI of the MI355X (gfx950) library for one DSpark
 * draft-and-verify round over vocabulary-sized logits.
 *
 * Sources (page title -- section):
 *  [MG] "DSpark：DeepSeek 线上跑的投机解码，半自回归 + 置信度调度怎么做到的"
 *       (marsggbo.github.io): 3.2 Sequential Stage -- Markov head
 *       B_k = W2(W1[x_{k-1}]), the RNN head, and the left-to-right sampling
 *       loop;
 *       4.1 Confidence Head -- c_k from [h_k, W1[x_{k-1}]], acceptance
 *       probability 1 - TV; 4.2 -- survival products;
 *       4.3 Hardware-Aware Prefix Scheduler -- a_{r,j}, B, tau, Theta, greedy
 *       extension in descending a with early stop.
 *  [CE] "DeepSeek DSpark explained" (share.concentrate1.com): section 02 --
 *       the first rejection truncates the suffix, a bonus token follows when
 *       every draft passes; section 03 -- q_k = softmax(U_k + B_k); section
 *       04 -- a_j, tau, Theta = tau * SPS(B); section 05 -- accept with
 *       min(1, p/q), resample from max(p - q, 0) normalised.
 *
 * Conventions shared by every entry point:
 *  - Arrays are row-major and densely packed.  "device" pointers are HIP
 *    device memory (or memory the device can read at full speed); "host"
 *    pointers are ordinary CPU memory.
 *  - The caller owns every buffer.  The library never allocates or frees
 *    device memory: scratch space is the caller's `workspace`, sized by the
 *    matching *_workspace_size query.  Workspace contents need no
 *    initialisation and are not meaningful between calls, except that
 *    dspark_verify_check reads the status the last dspark_verify left there.
 *    The one exception is dspark_draft_sample_noalloc, which takes no
 *    workspace and uses a fixed array the library holds on each device.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Device entry
 *    points only enqueue work on it and return; results are ready when the
 *    stream is.  Two calls that share a workspace must be ordered on one
 *    stream.  dspark_schedule is synchronous host code.
 *  - Every entry point returns a dspark_status.  Arguments are validated on
 *    the host before anything is enqueued; on an error nothing is enqueued
 *    and no output is written.
 *  - Random numbers come from Philox4x32-10 (Salmon et al., SC'11), keyed by
 *    `seed` and addressed by the counter (stream << 24 | position, i >> 2 or
 *    0, request index, low 32 bits of round_id), output word i & 3, where i
 *    is a vocabulary entry (streams 0 and 2) or a 32-entry vocabulary tile
 *    (streams 3 and 4).  Streams: 0 = draft entry noise, 1 = accept uniforms
 *    (word 0 of counter word1 = 0), 2 = resample / bonus entry noise, 3 =
 *    draft tile noise, 4 = resample / bonus tile noise.  Uniforms are
 *    ((w >> 8) + 0.5) * 2^-24, Gumbel noise -ln(-ln u).  Every sampled draw is
 *    a two-level Gumbel-max: tile t = v / 32 wins the race of
 *    logsumexp_{v in t} log-mass + tile noise, then entry v of that tile wins
 *    log-mass(v) + entry noise -- an exact draw from the normalised mass.
 *    Outputs are a pure function of the inputs, seed and round_id: two
 *    identical calls give identical bits.
 *  - Logits may be -inf (probability 0).  NaN inputs give undefined values
 *    but never out-of-bounds accesses or hangs.
 */
#ifndef DSPARK_H_
#define DSPARK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dspark_status {
    DSPARK_OK = 0,
    DSPARK_ERR_ARG = -1,          /* null required pointer or size out of range */
    DSPARK_ERR_UNSUPPORTED = -2,  /* valid arguments this build has no kernel for */
    DSPARK_ERR_WORKSPACE = -3,    /* workspace missing or smaller than queried */
    DSPARK_ERR_HIP = -4,          /* a HIP runtime call or kernel launch failed */
    DSPARK_ERR_DEVICE_INPUT = -5, /* device-resident input failed its check */
    DSPARK_ERR_SCRATCH = -6       /* sizes need more than the allocation-free entry point's fixed scratch */
} dspark_status;

/* Element types.  The Markov factors W1 and W2 are DSPARK_BF16 or DSPARK_F32;
 * attention rows and caches DSPARK_BF16 or DSPARK_F16, caches also
 * DSPARK_E4M3. */
typedef enum dspark_dtype {
    DSPARK_BF16 = 0, /* bfloat16 bit patterns (uint16_t) */
    DSPARK_F32 = 1,  /* IEEE float32 */
    DSPARK_F16 = 2,  /* IEEE float16 bit patterns (uint16_t) */
    DSPARK_E4M3 = 3  /* OCP FP8 E4M3 bit patterns (uint8_t), scaled by powers of two */
} dspark_dtype;

/* Size limits checked by every entry point. */
#define DSPARK_MAX_GAMMA 32
#define DSPARK_MAX_BATCH 65536
#define DSPARK_MAX_VOCAB 16777215
#define DSPARK_MAX_HIDDEN 65536 /* d of the confidence head */
#define DSPARK_MAX_STS_SAMPLES (1 << 28) /* samples of one calibration fit */
#define DSPARK_MAX_STS_CELLS 4096        /* grid values x bins of one fit */
#define DSPARK_MAX_STS_GRID 1024         /* grid values of one fit */
#define DSPARK_MAX_ROWS (1 << 24)        /* packed rows of one attention or cache call */
#define DSPARK_MAX_HEADS 1024            /* query heads */
#define DSPARK_MAX_CACHE_TOKENS (1 << 30) /* max_pages * page_size */
#define DSPARK_MAX_ROW_STRIDE (1 << 24)  /* elements from one packed row to the next */

/* Library version, major * 10000 + minor * 100 + patch. */
int dspark_version(void);

/* Static text for a dspark_status value (never NULL). */
const char *dspark_status_string(int status);

/* ------------------------------------------------------------------ */
/* Draft half ([MG] 3.2; [CE] 03)                                      */
/* ------------------------------------------------------------------ */

/* Bytes of device workspace dspark_draft_sample needs for these sizes;
 * 0 when the sizes are invalid. */
size_t dspark_draft_workspace_size(int B, int gamma, int V, int r);

/* Markov-head draft sampling for B requests over block positions k = 1..gamma.
 * For every request b and k, with x_0 = anchor[b]:
 *   z_k = (U[b, k-1, :] + W1[x_{k-1}, :] . W2^T) / T_b
 *   T_b > 0: x_k = the two-level Gumbel-max draw from q_k = softmax(z_k)
 *            (tile noise stream 3, entry noise stream 0, position k);
 *   T_b = 0: x_k = argmax_v z_k(v), lowest index first among equal values.
 * The [B, V] bias W1[x_{k-1}] W2^T is never written to memory.
 *
 *   U           device [B, gamma, V] float32   base logits U_k of the parallel stage
 *   W1, W2      device [V, r] of `wdtype`      Markov factors (W1: embedding rows,
 *                                              W2: output projection rows)
 *   anchor      device [B] int32 in [0, V)     x_0 of each request
 *   temperature device [B] float32 >= 0        T_b (0 = greedy)
 *   B in [1, DSPARK_MAX_BATCH], gamma in [1, DSPARK_MAX_GAMMA],
 *   V in [1, DSPARK_MAX_VOCAB], r in {16, 32, 64, 128, 256} (bf16) or
 *   {16, 32, 64, 128} (f32), otherwise DSPARK_ERR_UNSUPPORTED.
 *   seed, round_id                             Philox key and round counter
 *   x_out       device [B, gamma] int32        sampled drafts x_1..x_gamma
 *   lse_out     device [B, gamma] float32      logsumexp(z_k), so q_k = exp(z_k - lse);
 *                                              for T_b = 0 the largest logit
 *   qx_out      device [B, gamma] float32      q_k(x_k) (1 for T_b = 0)
 *   margin_out  device [B, gamma] float32 or NULL   the smaller of the draw's two
 *                                              top-two score gaps (tile race and
 *                                              entry race; logits for T_b = 0)
 *   workspace   device, >= dspark_draft_workspace_size bytes
 * Anchors outside [0, V) are clamped into range on the device. */
int dspark_draft_sample(const float *U, const void *W1, const void *W2, int wdtype,
                        const int32_t *anchor, const float *temperature,
                        int B, int gamma, int V, int r,
                        uint64_t seed, uint64_t round_id,
                        int32_t *x_out, float *lse_out, float *qx_out, float *margin_out,
                        void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of the fixed device array dspark_draft_sample_noalloc draws its
 * scratch from (one array on each device the library runs on, held until the
 * process ends). */
#define DSPARK_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)

/* dspark_draft_sample for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  It takes no workspace: its scratch is a fixed array of
 * DSPARK_NOALLOC_SCRATCH_BYTES in the library, one per device, whose address
 * is resolved once per device on the first call made with that device
 * current.  The call itself allocates nothing (no hipMalloc, hipFree or
 * allocating library routine; with per-kernel profiling off, no host
 * allocation either).  Outputs are the bits dspark_draft_sample writes for the
 * same inputs.
 *
 *   every argument: as for dspark_draft_sample, without the workspace; the
 *   device current at the call must be the one that holds the buffers and
 *   owns `stream`.
 * Returns DSPARK_ERR_SCRATCH when dspark_draft_workspace_size(B, gamma, V, r)
 * exceeds DSPARK_NOALLOC_SCRATCH_BYTES (B above 13,696 at V = 129,280,
 * r = 256), DSPARK_ERR_HIP when the array's address cannot be resolved, and
 * otherwise the errors of dspark_draft_sample.
 * Every call on one device shares that device's array and leaves it in an
 * arbitrary state; nothing in it needs clearing before a call.  Calls that
 * overlap on one device (on different streams, or from threads that do not
 * order their streams) race on the array and give undefined outputs. */
int dspark_draft_sample_noalloc(const float *U, const void *W1, const void *W2, int wdtype,
                                const int32_t *anchor, const float *temperature, int B, int gamma, int V,
                                int r, uint64_t seed, uint64_t round_id, int32_t *x_out, float *lse_out,
                                float *qx_out, float *margin_out, void *stream);

/* dspark_draft_sample plus the confidence head of every position ([MG] 4.1
 * Confidence Head; [MG] 4.2 and [CE] 04 for the survival products): with
 * x_0 = anchor and the drafts this call samples,
 *   c_k = 1 / (1 + exp(-(w[0..d) . h_k + w[d..d+r) . W1[x_{k-1}]) / tau_k))
 * -- a bias-free linear layer over the concatenation [h_k, W1[x_{k-1}]] and
 * a sigmoid -- and a_k = c_1 * ... * c_k, the estimated probability that
 * drafts 1..k all survive verification.  The sampling outputs are the same
 * bits dspark_draft_sample writes for the same inputs.
 *
 *   hidden        device [B, gamma, d] float32: h_k of request b at row
 *                 b * gamma + k - 1 (may be NULL when d = 0)
 *   conf_w        device [d + r] float32: the head's weights, the h_k part
 *                 first
 *   d             0 .. DSPARK_MAX_HIDDEN
 *   conf_tau      device [gamma] float32 or NULL: the head's per-position
 *                 temperatures tau_k (those dspark_sts_fit chooses; NULL = 1)
 *   conf_out      device [B, gamma] float32: c_k
 *   survival_out  device [B, gamma] float32: a_k
 *   every other argument: as for dspark_draft_sample (same workspace size).
 * Rows of hidden and conf_w that are 16-byte aligned with d a multiple of 4
 * are read as float4. */
int dspark_draft_sample_confidence(const float *U, const void *W1, const void *W2, int wdtype,
                                   const int32_t *anchor, const float *temperature,
                                   int B, int gamma, int V, int r,
                                   uint64_t seed, uint64_t round_id,
                                   const float *hidden, const float *conf_w, int d, const float *conf_tau,
                                   int32_t *x_out, float *lse_out, float *qx_out, float *margin_out,
                                   float *conf_out, float *survival_out,
                                   void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace dspark_draft_sample_rnn needs; 0 for invalid
 * sizes.  Besides the draft step's partials and the two states it holds,
 * when d >= 4r and gamma >= 2, the h part of every position's gate product,
 * Wgco[:, 2r:] h_k, computed for the whole block before position 1 (float32
 * split-K partials, at most 512 MiB; otherwise the per-position product
 * covers h itself and the space is not taken). */
size_t dspark_draft_rnn_workspace_size(int B, int gamma, int V, int r, int d);

/* Draft sampling with the RNN head ([MG] 3.2, RNN Head) in place of the
 * Markov head: a recurrent state s_k over the block, s_0 = 0.  For every
 * request b and k = 1..gamma, with x_0 = anchor[b]:
 *   z   = [s_{k-1}, W1[x_{k-1}], h_k]                       (2r + d entries)
 *   g   = sigmoid(Wgco[0:r] z),  c = tanh(Wgco[r:2r] z),  o = Wgco[2r:3r] z
 *   s_k = g * s_{k-1} + (1 - g) * c,   e_k = tanh(o)
 *   z_k = (U[b, k-1, :] + e_k . W2^T) / T_b, and x_k drawn from it exactly as
 *   dspark_draft_sample draws (same streams, same outputs).
 * The head's products take bfloat16 operands: s_{k-1} and h_k are rounded to
 * bfloat16 (nearest, ties to even) where they enter the gate product, and e_k
 * is rounded to bfloat16 before the W2 product; s_k is kept in float32.
 *
 *   Wgco        device [3r, 2r + d] bfloat16 (nn.Linear weight layout: row j
 *               holds the weights of gate output j; rows 0..r-1 gate,
 *               r..2r-1 candidate, 2r..3r-1 output; columns in z's order)
 *   hidden      device [B, gamma, d] float32: h_k of request b at row
 *               b * gamma + k - 1 (may be NULL when d = 0); 16-byte aligned
 *   d           0 .. DSPARK_MAX_HIDDEN, a multiple of 32
 *   e_out       device [B, gamma, r] bfloat16, 16-byte aligned: the rows e_k
 *               the W2 product used -- what dspark_verify_rnn and
 *               dspark_acceptance_rnn need to rebuild q_k
 *   state_out   device [B, r] float32 or NULL: s_gamma
 *   workspace   device, >= dspark_draft_rnn_workspace_size bytes
 *   every other argument: as for dspark_draft_sample; wdtype must be
 *   DSPARK_BF16 (DSPARK_F32 returns DSPARK_ERR_UNSUPPORTED). */
int dspark_draft_sample_rnn(const float *U, const void *W1, const void *W2, const void *Wgco, int wdtype,
                            const int32_t *anchor, const float *temperature, const float *hidden, int d,
                            int B, int gamma, int V, int r, uint64_t seed, uint64_t round_id,
                            int32_t *x_out, float *lse_out, float *qx_out, float *margin_out,
                            void *e_out, float *state_out,
                            void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------ */
/* Sequential temperature scaling of the confidences ([MG] 4.2)        */
/* ------------------------------------------------------------------ */

/* Bytes of device workspace dspark_sts_fit needs; 0 for invalid sizes. */
size_t dspark_sts_workspace_size(int N, int gamma, int G, int n_bins);

/* Calibrates the confidence head from N observed rounds, left to right: for
 * k = 1..gamma, with the temperatures of positions < k fixed, tau_k is the
 * first grid value that minimises
 *   ECE_k(tau) = sum over n_bins equal-width bins of |sum y - sum a'| / N_k,
 *   a'_k = c'_1 ... c'_k,  c'_i = 1 / (1 + exp(-logit(c_i) / tau_i)),
 *   y_k = 1 if sample n accepted drafts 1..k (n_accept >= k), else 0,
 * over the N_k samples that verified position k (ell >= k); a' falls in bin
 * min(floor(a' n_bins), n_bins - 1).  Temperature scaling keeps the drafts'
 * order (tau > 0).  A position that no sample verified keeps tau_k = 1 and
 * gets ECE NaN; grid values <= 0 are never chosen.  The sums over samples
 * are exact integer sums (a' in 2^-32 fixed point), so results do not depend
 * on the order the GPU adds them in.
 *
 *   c            device [N, gamma] float32: the head's confidences (raw, tau = 1)
 *   n_accept     device [N] int32: accepted drafts of the sample's round
 *   ell          device [N] int32 or NULL (= gamma): verified positions
 *   grid         device [G] float32: candidate temperatures
 *   N            1 .. DSPARK_MAX_STS_SAMPLES
 *   G, n_bins    >= 1, G <= DSPARK_MAX_STS_GRID, G * n_bins <= DSPARK_MAX_STS_CELLS
 *   tau_out      device [gamma] float32 (feed it to the head's conf_tau)
 *   ece_out      device [gamma] float32: the ECE at the chosen tau_k
 *   ece_grid_out device [gamma, G] float32 or NULL: every grid value's ECE
 *                (+inf for grid values <= 0)
 *   workspace    device, >= dspark_sts_workspace_size bytes */
int dspark_sts_fit(const float *c, const int32_t *n_accept, const int32_t *ell, int N, int gamma,
                   const float *grid, int G, int n_bins, float *tau_out, float *ece_out,
                   float *ece_grid_out, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------ */
/* Verify half ([CE] 02, 05; [MG] 1, 4.1)                              */
/* ------------------------------------------------------------------ */

/* Bytes of device workspace dspark_verify needs; 0 for invalid sizes. */
size_t dspark_verify_workspace_size(int B, int gamma, int V, int r);

/* Exact rejection-sampling verification with per-request verify lengths.
 * Request b verifies its first ell[b] drafts against packed target rows
 * off_b .. off_b + ell[b] (row off_b + k - 1 = target logits for position
 * k; the last one feeds the bonus token).  With p_k = softmax(t_k / T_b)
 * and q_k the draft distribution recomputed from U, W1, W2 and lse_q:
 *   k = 1..ell[b]: accept x_k iff u_k * q_k(x_k) < p_k(x_k), u_k a Philox
 *                  uniform (T_b = 0: iff x_k = argmax t_k);
 *   first rejection j: y drawn from r = max(p_j - q_j, 0) / S, S = sum of
 *                  the residual (T_b = 0: y = argmax t_j); S = 0 falls back
 *                  to p_j;
 *   every draft accepted: y drawn from p_{ell+1} (the bonus token).
 * The draws are two-level Gumbel-max draws at position j (tile noise stream
 * 4, entry noise stream 2); entries of zero mass never win.
 * Request b emits n_b + 1 tokens: x_1..x_{n_b}, y.
 *
 *   target        device [n_target_rows, V] float32   packed target logits
 *   n_target_rows rows in `target`; a request whose rows fall outside it is
 *                 not verified (outputs -1, device status set)
 *   ell           device [B] int32 in [0, gamma]
 *   row_offsets   device [B + 1] int32 or NULL: off_b, the exclusive scan of
 *                 (1 + ell); NULL = computed on the device
 *   U, W1, W2, wdtype, temperature, B, gamma, V, r: as for dspark_draft_sample
 *   anchor, x     device [B] and [B, gamma] int32: x_0 and the drafts
 *   lse_q, qx     device [B, gamma] float32: lse_out and qx_out of the draft
 *   seed, round_id  same values as the draft call of this round
 *   n_accept_out  device [B] int32: n_b (-1 for a request that failed its check)
 *   tokens_out    device [B, gamma + 1] int32: x_1..x_n, y, then -1
 *   out_offsets   device [B + 1] int32 or NULL: exclusive scan of (n_b + 1)
 *   diag_out      device [B, gamma + 1, 2] float32 or NULL: for tested
 *                 positions (p_k(x_k), min(1, p_k(x_k) / q_k(x_k))), NaN elsewhere
 *   resid_out     device [B] float32 or NULL: residual mass S at a sampled
 *                 rejection, -1 otherwise
 *   workspace     device, >= dspark_verify_workspace_size bytes
 * Invalid ell / row_offsets values are device-resident, so they are found on
 * the device: the affected request outputs -1 and dspark_verify_check
 * reports DSPARK_ERR_DEVICE_INPUT. */
int dspark_verify(const float *target, int n_target_rows, const int32_t *ell,
                  const int32_t *row_offsets,
                  const float *U, const void *W1, const void *W2, int wdtype,
                  const int32_t *anchor, const int32_t *x, const float *lse_q, const float *qx,
                  const float *temperature, int B, int gamma, int V, int r,
                  uint64_t seed, uint64_t round_id,
                  int32_t *n_accept_out, int32_t *tokens_out, int32_t *out_offsets,
                  float *diag_out, float *resid_out,
                  void *workspace, size_t workspace_bytes, void *stream);

/* Waits for `stream`, then returns DSPARK_OK or DSPARK_ERR_DEVICE_INPUT for
 * the device-side input checks of the last dspark_verify that used
 * `workspace` (DSPARK_ERR_HIP if the copy fails). */
int dspark_verify_check(const void *workspace, void *stream);

/* dspark_verify for drafts of the RNN head: q_k is rebuilt from the head's
 * rows e_k (head_rows, the e_out of dspark_draft_sample_rnn, [B, gamma, r]
 * of `wdtype`, 16-byte aligned) instead of W1[x_{k-1}].  Arguments, outputs,
 * workspace and device checks as for dspark_verify. */
int dspark_verify_rnn(const float *target, int n_target_rows, const int32_t *ell,
                      const int32_t *row_offsets,
                      const float *U, const void *head_rows, const void *W2, int wdtype,
                      const int32_t *anchor, const int32_t *x, const float *lse_q, const float *qx,
                      const float *temperature, int B, int gamma, int V, int r,
                      uint64_t seed, uint64_t round_id,
                      int32_t *n_accept_out, int32_t *tokens_out, int32_t *out_offsets,
                      float *diag_out, float *resid_out,
                      void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------ */
/* Per-position acceptance probability ([MG] 4.1; [CE] 05)             */
/* ------------------------------------------------------------------ */

/* Bytes of device workspace dspark_acceptance needs; 0 for invalid sizes. */
size_t dspark_acceptance_workspace_size(int B, int gamma, int V, int r);

/* The probability that draft k of request b passes the rejection test, taken
 * before x_k is drawn -- the confidence head's training label:
 *   alpha_k = sum_v min(p_k(v), q_k(v)) = 1 - TV(p_k, q_k),
 * with p_k = softmax(t_k / T_b) and q_k = softmax((U_k + W1[x_{k-1}] W2^T) / T_b)
 * recomputed from U, W1, W2 and lse_q on the drafted prefix (x_0 = anchor).
 * T_b = 0: alpha_k = 1 if x_k is the lowest-index argmax of t_k, else 0.
 * Every verified position k = 1..ell[b] is evaluated, also past the first
 * rejection (the target rows exist for the whole verified block).
 *
 *   target, n_target_rows, ell, row_offsets, U, W1, W2, wdtype, anchor, x,
 *   lse_q, temperature, B, gamma, V, r: as for dspark_verify (packed target
 *                 rows; row off_b + k - 1 holds position k)
 *   alpha_out     device [B, gamma] float32: alpha_k for k <= ell[b], NaN for
 *                 k > ell[b] and for every position of a request whose ell /
 *                 row_offsets fail the checks dspark_verify makes
 *   workspace     device, >= dspark_acceptance_workspace_size bytes
 * Cost: every verified row is read twice (its logsumexp, then the accepted
 * mass beside its U_k row and the W2 tiles), so this is a labelling pass, not
 * a step of the serving round. */
int dspark_acceptance(const float *target, int n_target_rows, const int32_t *ell,
                      const int32_t *row_offsets,
                      const float *U, const void *W1, const void *W2, int wdtype,
                      const int32_t *anchor, const int32_t *x, const float *lse_q,
                      const float *temperature, int B, int gamma, int V, int r,
                      float *alpha_out, void *workspace, size_t workspace_bytes, void *stream);

/* dspark_acceptance for drafts of the RNN head: q_k from head_rows as in
 * dspark_verify_rnn. */
int dspark_acceptance_rnn(const float *target, int n_target_rows, const int32_t *ell,
                          const int32_t *row_offsets,
                          const float *U, const void *head_rows, const void *W2, int wdtype,
                          const int32_t *anchor, const int32_t *x, const float *lse_q,
                          const float *temperature, int B, int gamma, int V, int r,
                          float *alpha_out, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------ */
/* Rules on logits (in front of dspark_verify: what is drawn has to     */
/* keep to them)                                                        */
/* ------------------------------------------------------------------ */

/* Penalties for repeated tokens, biases and grammar masks on the target rows of a
 * round: logits of any float type in, the float32 rows dspark_verify takes out.
 * Row j (from 0) of request b, token v:
 *   z = logits[v]
 *   v in the request's text (its prompt included), or among the drafts x_1 .. x_j
 *     in front of the row:  z = z > 0 ? z / repetition[b] : z * repetition[b]
 *   c > 0 times in the generated part of the text and those drafts:
 *     z = z - (frequency[b] * c + presence[b])
 *   z = z + the biases of v
 *   z = -inf where the row's mask forbids v (whatever the logit, NaN included)
 * in float32.
 *   logits      device [n_rows, V] of `dtype` (DSPARK_BF16, DSPARK_F16 or
 *               DSPARK_F32), row stride `stride` elements (>= V)
 *   row_offsets device [B + 1] int32, as for the cache entry points (NULL: one row a
 *               request, n_rows = B); rows of no request are not written
 *   history     device [B, max_history] int32: the tokens of each request so far, the
 *               anchor last; the first prompt_len[b] (NULL: 0) are the prompt's, those
 *               up to history_len[b] are generated.  NULL: no text.
 *   drafts      device [B, gamma] int32 or NULL: dspark_draft_sample's x
 *   repetition, frequency, presence   device [B] float32, each may be NULL (1, 0, 0);
 *               repetition > 0
 *   bias_offsets, bias_ids, bias_values   device [B + 1] int32, [n_biases] int32 and
 *               float32: request b owns entries bias_offsets[b] ..
 *               bias_offsets[b + 1] - 1; a token that stands there twice gets the sum.
 *               bias_offsets NULL: none
 *   masks       device [n_masks, mask_stride] int32, mask_stride >= ceil(V / 32): token
 *               v is allowed where bit v % 32 of word v / 32 is set.  NULL: none
 *   mask_index  device [n_rows] int32: each row's mask; an index outside [0, n_masks)
 *               stands for no mask
 *   out         device [n_rows, V] float32, row stride out_stride (>= V): the logits
 *               themselves (float32, same stride), or rows that do not overlap them
 * Token ids outside [0, V) are passed over.  max_history and n_biases are at most
 * DSPARK_MAX_CACHE_TOKENS, B * ceil(V / 4096) is below 2^23.
 * Counts are whole numbers and biases are added in their order: outputs are a pure
 * function of the inputs.  Lengths, offsets and indexes are read on the device, so
 * a captured call follows them as they change. */
int dspark_logit_rules(const void *logits, int64_t stride, int dtype, const int32_t *row_offsets, int n_rows, int B,
                       int V, const int32_t *history, int max_history, const int32_t *history_len,
                       const int32_t *prompt_len, const int32_t *drafts, int gamma, const float *repetition,
                       const float *frequency, const float *presence, const int32_t *bias_offsets,
                       const int32_t *bias_ids, const float *bias_values, int n_biases, const int32_t *masks,
                       int n_masks, int64_t mask_stride, const int32_t *mask_index, float *out, int64_t out_stride,
                       void *stream);

/* ------------------------------------------------------------------ */
/* Paged key-value cache ([CE] 02: the target forward of a round)      */
/* ------------------------------------------------------------------ */

/* Conventions of the cache, rotation and attention entry points.
 *
 * Packed rows.  A call works on n_rows rows of B requests; request b owns rows
 * row_offsets[b] .. row_offsets[b + 1] - 1 (device [B + 1] int32, non-decreasing;
 * NULL = one row a request, n_rows = B).  For a verify step these are the
 * 1 + ell[b] target rows of dspark_verify, with the same offsets.  Rows of no
 * request (before row_offsets[0], from row_offsets[B] on) are neither read into
 * a result nor written.  Offsets are clamped into [0, n_rows] on the device.
 * A row is [heads, head_dim]; q, k and v may be slices of wider rows: their
 * *_stride is the distance of two rows in elements, a multiple of 8, at least
 * heads * head_dim and at most DSPARK_MAX_ROW_STRIDE; rows are 16-byte aligned.
 *
 * Cache.  k_cache and v_cache are [n_pages, n_kv_heads, page_size, head_dim] of
 * cache_dtype; page_size is a power of two from 16 to 1024.  Token t of request
 * b lies in page page_table[b, t / page_size] (device [B, max_pages] int32) at
 * slot t % page_size.  Several requests may share pages; a page id outside
 * [0, n_pages) stands for no page, and so do tokens past the table: writes to
 * them are dropped, reads give zeros, attention leaves them out.
 * max_pages * page_size is at most DSPARK_MAX_CACHE_TOKENS; caches may be larger
 * than 4 GiB.
 *
 * 8-bit caches (DSPARK_E4M3) hold, for each (token, head), head_dim e4m3 values
 * and one scale byte e + 127 in k_scale / v_scale [n_pages, n_kv_heads,
 * page_size] uint8: the element stands for value * 2^e.  dspark_kv_write takes
 * the smallest e >= -126 with max|x| <= 448 * 2^e over the row's finite values
 * and rounds x * 2^-e to the nearest e4m3 value, ties to even; infinities and
 * NaN become NaN.  For other caches the scales are NULL.
 *
 * cache_len (device [B] int32) is the number of a request's tokens already in
 * the cache: its row i of this call stands at position cache_len[b] + i.  After
 * a verify step cache_len grows by n_accept + 1 (the anchor and the accepted
 * drafts); the rows past them are simply written again.  A negative cache_len
 * takes the request out of the call (a padded batch): nothing of it is written,
 * attention gives it zeros.
 *
 * head_dim is 64, 128 or 256, otherwise DSPARK_ERR_UNSUPPORTED.  Row types are
 * DSPARK_BF16 or DSPARK_F16; a cache has the rows' type or DSPARK_E4M3
 * (otherwise DSPARK_ERR_UNSUPPORTED).  n_rows = 0 is valid and does nothing.
 * One launch takes all of a call: n_rows * n_heads is below 2^31, the K and V
 * of a write or read are below 256 GiB, the rows of a rotation or an append
 * too, and n_rows * n_heads / 128 + (B + 1) * n_kv_heads of a prompt
 * call is below 2^24 (otherwise DSPARK_ERR_ARG).  Calls
 * that may overlap in time, on two streams or in two captured graphs, need a
 * workspace each.
 * The device current at the call must be the one that holds the buffers and
 * owns `stream`. */

/* Writes rows k, v [n_rows, n_kv_heads, head_dim] into the cache at positions
 * cache_len[b] + i.  No two rows of one call may name the same slot (the result
 * would be either's values).
 *   k, v        device rows of `dtype`, row strides k_stride and v_stride
 *   k_cache, v_cache, k_scale, v_scale   device, written at the rows' slots only */
int dspark_kv_write(const void *k, const void *v, int64_t k_stride, int64_t v_stride, int dtype,
                    const int32_t *row_offsets, int n_rows, const int32_t *cache_len, const int32_t *page_table, int B,
                    int max_pages, int n_kv_heads, int head_dim, void *k_cache, void *v_cache, uint8_t *k_scale,
                    uint8_t *v_scale, int cache_dtype, int n_pages, int page_size, void *stream);

/* Reads rows back: row i of request b is the token at position first[b] + i
 * (first NULL = 0; a negative first[b] gives zeros), as values of `dtype`.
 * 8-bit values come back as value * 2^e rounded to `dtype` (exact in its normal
 * range; what passes the type's largest value becomes that value).
 *   k_out, v_out   device [n_rows, n_kv_heads, head_dim] of `dtype`, dense */
int dspark_kv_read(const void *k_cache, const void *v_cache, const uint8_t *k_scale, const uint8_t *v_scale,
                   int cache_dtype, int n_pages, int page_size, const int32_t *row_offsets, int n_rows,
                   const int32_t *first, const int32_t *page_table, int B, int max_pages, int n_kv_heads, int head_dim,
                   void *k_out, void *v_out, int dtype, void *stream);

/* Heads normed and turned by their positions, on their way from the projections
 * to the attention.  For each head x of a row at position p:
 *   y = x, or with norm weights w:  y = x w / sqrt(mean(x^2) + eps),
 *   (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a),  a = p inv_freq[m]
 * for m < rotary_dim / 2 over the pairs (i, j) = (m, m + rotary_dim / 2), or the
 * neighbours (2 m, 2 m + 1) where `neighbours` is not 0; channels from rotary_dim
 * on keep y.  Row i of request b stands at position first[b] + i (first NULL = 0; a
 * negative first[b] takes the request out: its rows are not written, nor are rows
 * of no request).  Computed in float32, angles to 2^-51 of their size, and rounded
 * once (a head whose squares sum past float32's range is normed to zeros).
 *   q, k        device rows of `dtype` (DSPARK_BF16 or DSPARK_F16), row strides
 *               q_stride and k_stride; one of the two may be absent (NULL, 0 heads)
 *   inv_freq    device [rotary_dim / 2] float32 (may be NULL where rotary_dim is 0)
 *   rotary_dim  0 (no rotation) to head_dim, a multiple of 16
 *   q_norm, k_norm   device [head_dim] of norm_dtype (`dtype` or DSPARK_F32), one or
 *               both NULL: no norm
 *   eps         >= 0, finite
 *   q_out, k_out     device rows of `dtype`, row strides q_out_stride and
 *               k_out_stride: q and k themselves (same strides), or rows that
 *               overlap neither */
int dspark_rotary(const void *q, const void *k, int64_t q_stride, int64_t k_stride, int dtype,
                  const int32_t *row_offsets, int n_rows, const int32_t *first, int B, int n_heads, int n_kv_heads,
                  int head_dim, const float *inv_freq, int rotary_dim, int neighbours, const void *q_norm,
                  const void *k_norm, int norm_dtype, float eps, void *q_out, void *k_out, int64_t q_out_stride,
                  int64_t k_out_stride, void *stream);

/* dspark_rotary and dspark_kv_write in one: queries are normed, turned and written
 * to q_out; keys are normed, turned and written into the cache at positions
 * cache_len[b] + i, and values beside them as they are.  An 8-bit cache takes the
 * keys straight from their float32 values, in the format of dspark_kv_write.
 *   q           may be NULL with n_heads 0 (keys and values alone); otherwise as for
 *               dspark_rotary.  The query rows of a request with a negative
 *               cache_len are not written.
 *   k, v, the cache, cache_len, page_table   as for dspark_kv_write */
int dspark_kv_append(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                     int64_t v_stride, int dtype, const int32_t *row_offsets, int n_rows, const int32_t *cache_len,
                     const int32_t *page_table, int B, int max_pages, int n_heads, int n_kv_heads, int head_dim,
                     const float *inv_freq, int rotary_dim, int neighbours, const void *q_norm, const void *k_norm,
                     int norm_dtype, float eps, void *q_out, int64_t q_out_stride, void *k_cache, void *v_cache,
                     uint8_t *k_scale, uint8_t *v_scale, int cache_dtype, int n_pages, int page_size, void *stream);

/* ------------------------------------------------------------------ */
/* Attention ([CE] 02: one causal forward over the block's positions)  */
/* ------------------------------------------------------------------ */

/* Bytes of device workspace dspark_paged_attention needs; 0 for invalid sizes. */
size_t dspark_paged_attention_workspace_size(int max_rows, int n_heads, int n_kv_heads, int head_dim);

/* Attention of each request's rows over its cached tokens: row i of request b
 * (position cache_len[b] + i), head h, with key-value head h / (n_heads /
 * n_kv_heads):
 *   s_t = scale * q . k_t,  out = sum_t softmax(s)_t v_t,  lse = log sum_t exp(s_t)
 * over the tokens t <= cache_len[b] + i (causal != 0: decoding, verification)
 * or t < cache_len[b] + rows of b (causal = 0: the rows see each other, as in a
 * parallel draft stage).  The rows' own keys and values must be in the cache
 * (dspark_kv_write of the same rows, before this call on the stream).  A row
 * that sees no token (or none with a score above -inf) gives zeros and lse =
 * -inf.  Infinities and NaN in tokens a row does not see, or in unused slots, do
 * not reach it; infinities of V that it sees make their channel infinite (NaN
 * where both signs meet, or where the probability is below float32's range).
 * Scores, softmax sums and products are kept in float32; probabilities enter the
 * V product in the rows' type (over 8-bit caches in bfloat16, for float16 rows in
 * two bfloat16 terms).
 *   q           device [n_rows, n_heads, head_dim] of `dtype`, row stride q_stride
 *   n_heads     a multiple of n_kv_heads, at most DSPARK_MAX_HEADS
 *   max_rows    >= 1: how many rows a request usually has at most (1 for
 *               decoding, gamma + 1 for verification).  It only picks the
 *               kernel: requests may have more or fewer.
 *   scale       > 0, at most 2.3e38 (usually head_dim^-1/2)
 *   out         device [n_rows, n_heads, head_dim] of `dtype`, dense, 16-byte aligned
 *   lse_out     device [n_rows, n_heads] float32 or NULL
 *   workspace   device, >= dspark_paged_attention_workspace_size bytes
 * The work is split over a request's length and joined in a fixed order:
 * outputs are a pure function of the inputs.  Lengths, offsets and pages are
 * read on the device, so a captured call follows them as they change. */
int dspark_paged_attention(const void *q, int64_t q_stride, int dtype, const int32_t *row_offsets, int n_rows,
                           int max_rows, const int32_t *cache_len, const int32_t *page_table, int B, int max_pages,
                           int n_heads, int n_kv_heads, int head_dim, const void *k_cache, const void *v_cache,
                           const uint8_t *k_scale, const uint8_t *v_scale, int cache_dtype, int n_pages, int page_size,
                           float scale, int causal, void *out, float *lse_out, void *workspace, size_t workspace_bytes,
                           void *stream);

/* Bytes of device workspace dspark_window_attention needs; 0 for invalid sizes. */
size_t dspark_window_attention_workspace_size(int max_rows, int n_heads, int n_kv_heads, int head_dim);

/* dspark_paged_attention (causal) through a sliding window: the row at position
 * p = cache_len[b] + i sees the tokens t <= p with p - t < window, and the first
 * `sinks` tokens of its request (t <= p and t < sinks).  Any number of rows a
 * request, from one (decoding) to chunks of a prompt of thousands.  Tokens that no
 * row of a request sees are not read: their pages may be gone from page_table.
 *   window      >= 1
 *   sinks       >= 0
 *   max_rows    >= 1: how many rows a request usually has at most (where chunks stand
 *               beside single rows: the chunks'); picks the kernel
 *   everything else as for dspark_paged_attention, the rounding of the probabilities
 *   too (calls of many rows take the values of an 8-bit cache in bfloat16: those past
 *   its largest, 3.39e38, are infinite) */
int dspark_window_attention(const void *q, int64_t q_stride, int dtype, const int32_t *row_offsets, int n_rows,
                            int max_rows, const int32_t *cache_len, const int32_t *page_table, int B, int max_pages,
                            int n_heads, int n_kv_heads, int head_dim, const void *k_cache, const void *v_cache,
                            const uint8_t *k_scale, const uint8_t *v_scale, int cache_dtype, int n_pages,
                            int page_size, int window, int sinks, float scale, void *out, float *lse_out,
                            void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace dspark_prompt_attention needs; 0 for invalid sizes. */
size_t dspark_prompt_attention_workspace_size(int B, int n_rows, int n_kv_rows, int n_heads, int n_kv_heads,
                                              int head_dim);

/* Attention over whole prompts, packed: sequence b has query rows
 * row_offsets[b] .. row_offsets[b + 1] - 1 of q and key rows kv_offsets[b] ..
 * kv_offsets[b + 1] - 1 of k and v (kv_offsets NULL: the same rows, n_kv_rows =
 * n_rows).  With R query rows and L keys, query row i stands at position
 * L - R + i: causal != 0 lets it see keys t <= L - R + i (behind a prefix read
 * back by dspark_kv_read L > R; rows with L - R + i < 0 see nothing), causal = 0
 * every key of its sequence.  Outputs, empty rows, masked infinities and
 * precision as for dspark_paged_attention.
 *   q           device [n_rows, n_heads, head_dim] of `dtype`, row stride q_stride
 *   k, v        device [n_kv_rows, n_kv_heads, head_dim], row strides k_stride, v_stride
 *   out, lse_out   as for dspark_paged_attention; rows of no sequence are left alone
 *   workspace   device, >= dspark_prompt_attention_workspace_size bytes */
int dspark_prompt_attention(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, int dtype, const int32_t *row_offsets, int n_rows,
                            const int32_t *kv_offsets, int n_kv_rows, int B, int n_heads, int n_kv_heads, int head_dim,
                            float scale, int causal, void *out, float *lse_out, void *workspace,
                            size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------ */
/* Host scheduler ([MG] 4.3; [CE] 04)                                  */
/* ------------------------------------------------------------------ */

/* Confidence-scheduled prefix lengths.  Synchronous, host memory only.
 *   c         host [R, gamma] double in [0, 1]: calibrated confidences c_{r,j}
 *   sps       host [sps_len] double: SPS(B) for B = 0..sps_len-1; B beyond the
 *             table counts as 0.  sps_len must exceed R.
 *   ell_out   host [R] int32: chosen verify lengths
 *   theta_out, tau_out, B_out  (each may be NULL): Theta, tau and B of the choice
 * a_{r,j} = prod_{i<=j} c_{r,i}; starting from ell = 0 (B = tau = R), the
 * candidates with a > 0 are taken in descending a (ties: lower r, then lower
 * j); each extends its request by one (B += 1, tau += a) and is kept while
 * Theta = tau * SPS(B) strictly improves; the first step that does not
 * improve ends the search.  R = 0 is valid and returns Theta = 0. */
int dspark_schedule(const double *c, int R, int gamma, const double *sps, int sps_len,
                    int32_t *ell_out, double *theta_out, double *tau_out, int32_t *B_out);

/* Production-style scheduling ([CE] 04, the strict implementation: in an
 * asynchronous pipeline the step's capacity comes from the previous two
 * steps' predictions and the current candidates are only sorted into it).
 *
 * dspark_history_capacity: the capacity of the current step, R requests,
 *   round(R * mean_i B_hist[i] / R_hist[i]) over the first min(n_hist, 2)
 *   entries with R_hist[i] > 0 (the synchronous scheduler's B and R of the
 *   previous steps), rounding half up, clamped to [R, R (1 + gamma)];
 *   R (1 + gamma) (verify everything) when no entry is usable.  Host.
 * dspark_schedule_capacity: with c, R, gamma as for dspark_schedule, extends
 *   the requests in the same candidate order (-a, r, j) under the same
 *   prefix rule until B = capacity (or the candidates with a > 0 run out),
 *   without the early stop; ell_out [R], tau_out and B_out as for
 *   dspark_schedule.  With the capacity the synchronous scheduler chose it
 *   returns that scheduler's lengths; for any capacity its tau is the largest
 *   a prefix-valid choice of that B reaches.  Host, synchronous. */
int dspark_history_capacity(const int32_t *B_hist, const int32_t *R_hist, int n_hist, int R, int gamma,
                            int64_t *capacity_out);
int dspark_schedule_capacity(const double *c, int R, int gamma, int64_t capacity,
                             int32_t *ell_out, double *tau_out, int32_t *B_out);

/* ------------------------------------------------------------------ */
/* Diagnostics                                                         */
/* ------------------------------------------------------------------ */

/* Writes the library's 32-bit Philox words for indices v0 .. v0 + n - 1
 * (entries for streams 0 and 2, tiles for 3 and 4; ignored for stream 1) of
 * random stream `stream_id` in [0, 4] at position k of request `req` to
 * device [n] uint32 `out`. */
int dspark_debug_random_words(uint64_t seed, uint64_t round_id, int stream_id, int k, int req,
                              int v0, int n, uint32_t *out, void *stream);

/* Applies the library's device Gumbel transform to n device words:
 * out[i] = -log2(-log2(u_i)), u_i = ((w_i >> 8) + 0.5) * 2^-24. */
int dspark_debug_gumbel(const uint32_t *words, int n, float *out, void *stream);

/* The Markov-bias product alone, to measure the matrix-unit tiling of the
 * draft step ([MG] 3.2; [CE] 03: B_k = W1[x_{k-1}] W2^T) without the rest of
 * the step: rowmax_out[b] = max_v sum_i W1[idx[b]][i] * W2[v][i], computed
 * with the draft step's workgroups, LDS-staged W2 tiles and MFMA tiles, with
 * no U_k read and no sampling.
 *   W1, W2, wdtype, V, r  as for dspark_draft_sample
 *   idx         device [B] int32: the W1 rows (clamped into [0, V))
 *   rowmax_out  device [B] float32
 *   workspace   device, >= dspark_draft_workspace_size(B, 1, V, r) bytes
 * Same argument checks and error codes as dspark_draft_sample. */
int dspark_debug_bias_gemm(const void *W1, const void *W2, int wdtype, const int32_t *idx, int B, int V, int r,
                           float *rowmax_out, void *workspace, size_t workspace_bytes, void *stream);

/* Per-kernel timing with HIP events.  While enabled, every kernel the
 * library enqueues is launched with a start / stop event pair that the
 * dispatch itself stamps (hipExtLaunchKernel), so a duration is the kernel's
 * own execution time, without the launch gap; dspark_profile_collect waits
 * for the events and adds their durations to per-kernel totals.  Not for
 * concurrent use from several threads. */
int dspark_profile_enable(int enable);
int dspark_profile_collect(void);
/* Number of kernel names with totals, and the totals of entry i. */
int dspark_profile_count(void);
int dspark_profile_get(int i, const char **name, int64_t *launches, double *total_ms);
int dspark_profile_reset(void);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_H_ */
