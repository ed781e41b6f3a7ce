// api.cpp -- the extern "C" entry points of libdspark.so: argument
// validation, workspace layout, kernel sequencing and per-kernel profiling.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "dspark.h"
#include "internal.hpp"

namespace dspark {

// ------------------------------------------------------------------ profiling

namespace {

struct ProfEntry {
    std::string name;
    int64_t launches = 0;
    double total_ms = 0.0;
};

struct Pending {
    int entry;
    hipEvent_t start, stop;
};

struct Profiler {
    std::mutex mu;
    bool enabled = false;
    // read without the lock on every launch: with profiling off a launch
    // takes no lock
    std::atomic<bool> on{false};
    std::vector<ProfEntry> entries;
    std::vector<Pending> pending;
    std::vector<hipEvent_t> pool;

    int entry_for(const char *name) {
        for (size_t i = 0; i < entries.size(); ++i)
            if (entries[i].name == name) return int(i);
        entries.push_back(ProfEntry{name});
        return int(entries.size() - 1);
    }
    hipEvent_t take_event() {
        if (!pool.empty()) {
            hipEvent_t e = pool.back();
            pool.pop_back();
            return e;
        }
        hipEvent_t e = nullptr;
        if (hipEventCreate(&e) != hipSuccess) return nullptr;
        return e;
    }
};

Profiler &prof() {
    static Profiler p;
    return p;
}

}  // namespace

ProfEvents prof_events(const char *name) {
    Profiler &p = prof();
    if (!p.on.load(std::memory_order_acquire)) return {};
    std::lock_guard<std::mutex> g(p.mu);
    if (!p.enabled) return {};
    Pending pd{p.entry_for(name), p.take_event(), p.take_event()};
    if (!pd.start || !pd.stop) return {};
    p.pending.push_back(pd);
    return {pd.start, pd.stop};
}

}  // namespace dspark

using namespace dspark;

namespace {

bool rank_supported(int wdtype, int r) {
    if (wdtype == DSPARK_BF16) return r == 16 || r == 32 || r == 64 || r == 128 || r == 256;
    if (wdtype == DSPARK_F32) return r == 16 || r == 32 || r == 64 || r == 128;
    return false;
}

bool sizes_ok(int B, int gamma, int V, int r) {
    return B >= 1 && B <= DSPARK_MAX_BATCH && gamma >= 1 && gamma <= DSPARK_MAX_GAMMA && V >= 1 &&
           V <= DSPARK_MAX_VOCAB && r >= 1;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t draft_bytes(int B, int V) {
    const DraftPlan p = draft_plan(B, V);
    size_t bytes = 0;
    draft_carve(nullptr, B, p, &bytes);
    return bytes;
}

size_t accept_bytes(int B, int gamma, int V) {
    const AcceptPlan p = accept_plan(B, gamma, V);
    size_t bytes = 0;
    accept_carve(nullptr, B, gamma, p, &bytes);
    return bytes;
}

size_t verify_bytes(int B, int gamma, int V) {
    const VerifyPlan p = verify_plan(B, gamma, V);
    size_t bytes = 0;
    verify_carve(nullptr, B, gamma, V, p, &bytes);
    return bytes;
}

}  // namespace

extern "C" {

int dspark_version(void) { return 10000; }

const char *dspark_status_string(int status) {
    switch (status) {
        case DSPARK_OK: return "ok";
        case DSPARK_ERR_ARG: return "invalid argument";
        case DSPARK_ERR_UNSUPPORTED: return "unsupported size or type";
        case DSPARK_ERR_WORKSPACE: return "workspace missing or too small";
        case DSPARK_ERR_HIP: return "HIP runtime error";
        case DSPARK_ERR_DEVICE_INPUT: return "device-side input check failed";
        case DSPARK_ERR_SCRATCH: return "sizes exceed the allocation-free entry point's fixed scratch";
        default: return "unknown status";
    }
}

size_t dspark_draft_workspace_size(int B, int gamma, int V, int r) {
    if (!sizes_ok(B, gamma, V, r)) return 0;
    return draft_bytes(B, V);
}

}  // extern "C"

namespace {

// The host-side argument checks of the draft entry points.
int draft_args(const float *U, const void *W1, const void *W2, int wdtype, const int32_t *anchor,
               const float *temperature, int B, int gamma, int V, int r, const int32_t *x_out, const float *lse_out,
               const float *qx_out) {
    if (!U || !W1 || !W2 || !anchor || !temperature || !x_out || !lse_out || !qx_out) return DSPARK_ERR_ARG;
    if (!sizes_ok(B, gamma, V, r)) return DSPARK_ERR_ARG;
    if (wdtype != DSPARK_BF16 && wdtype != DSPARK_F32) return DSPARK_ERR_ARG;
    if (!rank_supported(wdtype, r)) return DSPARK_ERR_UNSUPPORTED;
    if (!aligned16(W1) || !aligned16(W2)) return DSPARK_ERR_ARG;
    return DSPARK_OK;
}

int draft_common(const float *U, const void *W1, const void *W2, int wdtype, const int32_t *anchor,
                 const float *temperature, int B, int gamma, int V, int r, uint64_t seed, uint64_t round_id,
                 const float *hidden, const float *conf_w, int d, const float *conf_tau, int32_t *x_out,
                 float *lse_out, float *qx_out, float *margin_out, float *conf_out, float *survival_out,
                 void *workspace, size_t workspace_bytes, void *stream) {
    const int st = draft_args(U, W1, W2, wdtype, anchor, temperature, B, gamma, V, r, x_out, lse_out, qx_out);
    if (st != DSPARK_OK) return st;
    const DraftPlan plan = draft_plan(B, V);
    size_t need = 0;
    draft_carve(nullptr, B, plan, &need);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DSPARK_ERR_WORKSPACE;
    const DraftWork w = draft_carve(workspace, B, plan, nullptr);
    DraftArgs a{};
    a.U = U;
    a.W1 = W1;
    a.W2 = W2;
    a.wdtype = wdtype;
    a.anchor = anchor;
    a.temperature = temperature;
    a.B = B;
    a.gamma = gamma;
    a.V = V;
    a.r = r;
    a.key0 = uint32_t(seed);
    a.key1 = uint32_t(seed >> 32);
    a.round32 = uint32_t(round_id);
    a.x_out = x_out;
    a.lse_out = lse_out;
    a.qx_out = qx_out;
    a.margin_out = margin_out;
    a.hidden = hidden;
    a.conf_w = conf_w;
    a.d = d;
    a.conf_tau = conf_tau;
    a.conf_out = conf_out;
    a.surv_out = survival_out;
    const hipError_t e = launch_draft(a, plan, w, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

}  // namespace

extern "C" {

int dspark_draft_sample(const float *U, const void *W1, const void *W2, int wdtype, const int32_t *anchor,
                        const float *temperature, int B, int gamma, int V, int r, uint64_t seed,
                        uint64_t round_id, int32_t *x_out, float *lse_out, float *qx_out, float *margin_out,
                        void *workspace, size_t workspace_bytes, void *stream) {
    return draft_common(U, W1, W2, wdtype, anchor, temperature, B, gamma, V, r, seed, round_id, nullptr, nullptr, 0,
                        nullptr, x_out, lse_out, qx_out, margin_out, nullptr, nullptr, workspace, workspace_bytes,
                        stream);
}

}  // extern "C"

namespace {

// The allocation-free entry point's scratch: a fixed array in the library's
// device code, so each device the library runs on holds its own copy from
// module load until the process ends.  Host code never uses the array's name
// as an address (it is a host-side stand-in); the device address comes from
// hipGetSymbolAddress, once per device with that device current, and is kept
// here.  The fast path is one atomic load; the first call on a device
// resolves the address under a lock.
static __device__ __align__(256) uint8_t scratch[DSPARK_NOALLOC_SCRATCH_BYTES];
constexpr int kScratchDevices = 256;
std::atomic<void *> scratch_addr[kScratchDevices];
std::mutex scratch_mu;

int scratch_for_current_device(void **out) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kScratchDevices) return DSPARK_ERR_HIP;
    void *p = scratch_addr[dev].load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> g(scratch_mu);
        p = scratch_addr[dev].load(std::memory_order_relaxed);
        if (!p) {
            if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return DSPARK_ERR_HIP;
            scratch_addr[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return DSPARK_OK;
}

}  // namespace

extern "C" {

int dspark_draft_sample_noalloc(const float *U, const void *W1, const void *W2, int wdtype, const int32_t *anchor,
                                const float *temperature, int B, int gamma, int V, int r, uint64_t seed,
                                uint64_t round_id, int32_t *x_out, float *lse_out, float *qx_out, float *margin_out,
                                void *stream) {
    const int st = draft_args(U, W1, W2, wdtype, anchor, temperature, B, gamma, V, r, x_out, lse_out, qx_out);
    if (st != DSPARK_OK) return st;
    if (draft_bytes(B, V) > DSPARK_NOALLOC_SCRATCH_BYTES) return DSPARK_ERR_SCRATCH;
    void *ws = nullptr;
    const int sc = scratch_for_current_device(&ws);
    if (sc != DSPARK_OK) return sc;
    // the draft's scratch needs no clearing: every partial is written before it is read
    return draft_common(U, W1, W2, wdtype, anchor, temperature, B, gamma, V, r, seed, round_id, nullptr, nullptr, 0,
                        nullptr, x_out, lse_out, qx_out, margin_out, nullptr, nullptr, ws,
                        DSPARK_NOALLOC_SCRATCH_BYTES, stream);
}

int dspark_draft_sample_confidence(const float *U, const void *W1, const void *W2, int wdtype,
                                   const int32_t *anchor, const float *temperature, int B, int gamma, int V, int r,
                                   uint64_t seed, uint64_t round_id, const float *hidden, const float *conf_w, int d,
                                   const float *conf_tau, int32_t *x_out, float *lse_out, float *qx_out,
                                   float *margin_out,
                                   float *conf_out, float *survival_out, void *workspace, size_t workspace_bytes,
                                   void *stream) {
    if (d < 0 || d > DSPARK_MAX_HIDDEN || (d > 0 && !hidden) || !conf_w || !conf_out || !survival_out)
        return DSPARK_ERR_ARG;
    return draft_common(U, W1, W2, wdtype, anchor, temperature, B, gamma, V, r, seed, round_id, hidden, conf_w, d,
                        conf_tau, x_out, lse_out, qx_out, margin_out, conf_out, survival_out, workspace,
                        workspace_bytes, stream);
}

size_t dspark_draft_rnn_workspace_size(int B, int gamma, int V, int r, int d) {
    if (!sizes_ok(B, gamma, V, r) || d < 0 || d > DSPARK_MAX_HIDDEN) return 0;
    const DraftPlan p = draft_plan(B, V);
    size_t bytes = 0;
    draft_carve(nullptr, B, p, &bytes, r, gamma, d);
    return bytes;
}

int dspark_draft_sample_rnn(const float *U, const void *W1, const void *W2, const void *Wgco, int wdtype,
                            const int32_t *anchor, const float *temperature, const float *hidden, int d, int B,
                            int gamma, int V, int r, uint64_t seed, uint64_t round_id, int32_t *x_out, float *lse_out,
                            float *qx_out, float *margin_out, void *e_out, float *state_out, void *workspace,
                            size_t workspace_bytes, void *stream) {
    if (!U || !W1 || !W2 || !Wgco || !anchor || !temperature || !x_out || !lse_out || !qx_out || !e_out)
        return DSPARK_ERR_ARG;
    if (!sizes_ok(B, gamma, V, r)) return DSPARK_ERR_ARG;
    if (wdtype != DSPARK_BF16 && wdtype != DSPARK_F32) return DSPARK_ERR_ARG;
    if (wdtype != DSPARK_BF16 || !rank_supported(wdtype, r)) return DSPARK_ERR_UNSUPPORTED;
    if (d < 0 || d > DSPARK_MAX_HIDDEN || (d > 0 && !hidden)) return DSPARK_ERR_ARG;
    if (d % 32 != 0) return DSPARK_ERR_UNSUPPORTED;
    if (!aligned16(W1) || !aligned16(W2) || !aligned16(Wgco) || !aligned16(e_out) || (d > 0 && !aligned16(hidden)))
        return DSPARK_ERR_ARG;
    const DraftPlan plan = draft_plan(B, V);
    size_t need = 0;
    draft_carve(nullptr, B, plan, &need, r, gamma, d);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DSPARK_ERR_WORKSPACE;
    const DraftWork w = draft_carve(workspace, B, plan, nullptr, r, gamma, d);
    DraftArgs a{};
    a.U = U;
    a.W1 = W1;
    a.W2 = W2;
    a.wdtype = wdtype;
    a.anchor = anchor;
    a.temperature = temperature;
    a.B = B;
    a.gamma = gamma;
    a.V = V;
    a.r = r;
    a.key0 = uint32_t(seed);
    a.key1 = uint32_t(seed >> 32);
    a.round32 = uint32_t(round_id);
    a.x_out = x_out;
    a.lse_out = lse_out;
    a.qx_out = qx_out;
    a.margin_out = margin_out;
    a.Wgco = Wgco;
    a.rnn_h = hidden;
    a.rnn_d = d;
    a.e_out = static_cast<uint16_t *>(e_out);
    a.state_out = state_out;
    const hipError_t e = launch_draft(a, plan, w, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

size_t dspark_sts_workspace_size(int N, int gamma, int G, int n_bins) {
    if (N < 1 || gamma < 1 || gamma > DSPARK_MAX_GAMMA || G < 1 || n_bins < 1 || G > DSPARK_MAX_STS_GRID ||
        G * n_bins > DSPARK_MAX_STS_CELLS)
        return 0;
    size_t bytes = 0;
    sts_carve(nullptr, N, gamma, G, n_bins, &bytes);
    return bytes;
}

int dspark_sts_fit(const float *c, const int32_t *n_accept, const int32_t *ell, int N, int gamma, const float *grid,
                   int G, int n_bins, float *tau_out, float *ece_out, float *ece_grid_out, void *workspace,
                   size_t workspace_bytes, void *stream) {
    if (!c || !n_accept || !grid || !tau_out || !ece_out) return DSPARK_ERR_ARG;
    if (N < 1 || N > DSPARK_MAX_STS_SAMPLES || gamma < 1 || gamma > DSPARK_MAX_GAMMA || G < 1 || n_bins < 1 ||
        G > DSPARK_MAX_STS_GRID || G * n_bins > DSPARK_MAX_STS_CELLS)
        return DSPARK_ERR_ARG;
    size_t need = 0;
    sts_carve(nullptr, N, gamma, G, n_bins, &need);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DSPARK_ERR_WORKSPACE;
    const StsWork w = sts_carve(workspace, N, gamma, G, n_bins, nullptr);
    StsArgs a{};
    a.c = c;
    a.n = n_accept;
    a.ell = ell;
    a.N = N;
    a.gamma = gamma;
    a.grid = grid;
    a.G = G;
    a.M = n_bins;
    a.tau_out = tau_out;
    a.ece_out = ece_out;
    a.ece_grid = ece_grid_out;
    const hipError_t e = launch_sts(a, sts_plan(N, gamma, G, n_bins), w, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

size_t dspark_verify_workspace_size(int B, int gamma, int V, int r) {
    if (!sizes_ok(B, gamma, V, r)) return 0;
    return verify_bytes(B, gamma, V);
}

static int verify_common(const float *target, int n_target_rows, const int32_t *ell, const int32_t *row_offsets,
                         const float *U, const void *W1, const void *W2, int wdtype, const int32_t *anchor,
                         const int32_t *x, const float *lse_q, const float *qx, const float *temperature, int B,
                         int gamma, int V, int r, uint64_t seed, uint64_t round_id, int32_t *n_accept_out,
                         int32_t *tokens_out, int32_t *out_offsets, float *diag_out, float *resid_out,
                         void *workspace, size_t workspace_bytes, void *stream, int erow_mode) {
    if (!target || !ell || !U || !W1 || !W2 || !anchor || !x || !lse_q || !qx || !temperature ||
        !n_accept_out || !tokens_out)
        return DSPARK_ERR_ARG;
    if (!sizes_ok(B, gamma, V, r) || n_target_rows < 1) return DSPARK_ERR_ARG;
    if (wdtype != DSPARK_BF16 && wdtype != DSPARK_F32) return DSPARK_ERR_ARG;
    if (!rank_supported(wdtype, r)) return DSPARK_ERR_UNSUPPORTED;
    if (!aligned16(W1) || !aligned16(W2)) return DSPARK_ERR_ARG;
    const VerifyPlan plan = verify_plan(B, gamma, V);
    size_t need = 0;
    verify_carve(nullptr, B, gamma, V, plan, &need);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DSPARK_ERR_WORKSPACE;
    const VerifyWork w = verify_carve(workspace, B, gamma, V, plan, nullptr);
    VerifyArgs a{};
    a.target = target;
    a.n_target_rows = n_target_rows;
    a.ell = ell;
    a.row_offsets = row_offsets;
    a.U = U;
    a.W1 = W1;
    a.W2 = W2;
    a.wdtype = wdtype;
    a.anchor = anchor;
    a.x = x;
    a.lse_q = lse_q;
    a.qx = qx;
    a.temperature = temperature;
    a.B = B;
    a.gamma = gamma;
    a.V = V;
    a.r = r;
    a.key0 = uint32_t(seed);
    a.key1 = uint32_t(seed >> 32);
    a.round32 = uint32_t(round_id);
    a.n_accept_out = n_accept_out;
    a.tokens_out = tokens_out;
    a.out_offsets = out_offsets;
    a.diag_out = diag_out;
    a.resid_out = resid_out;
    a.erow_mode = erow_mode;
    const hipError_t e = launch_verify(a, plan, w, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

int dspark_verify(const float *target, int n_target_rows, const int32_t *ell, const int32_t *row_offsets,
                  const float *U, const void *W1, const void *W2, int wdtype, const int32_t *anchor,
                  const int32_t *x, const float *lse_q, const float *qx, const float *temperature, int B,
                  int gamma, int V, int r, uint64_t seed, uint64_t round_id, int32_t *n_accept_out,
                  int32_t *tokens_out, int32_t *out_offsets, float *diag_out, float *resid_out,
                  void *workspace, size_t workspace_bytes, void *stream) {
    return verify_common(target, n_target_rows, ell, row_offsets, U, W1, W2, wdtype, anchor, x, lse_q, qx,
                         temperature, B, gamma, V, r, seed, round_id, n_accept_out, tokens_out, out_offsets, diag_out,
                         resid_out, workspace, workspace_bytes, stream, 0);
}

int dspark_verify_rnn(const float *target, int n_target_rows, const int32_t *ell, const int32_t *row_offsets,
                      const float *U, const void *head_rows, const void *W2, int wdtype, const int32_t *anchor,
                      const int32_t *x, const float *lse_q, const float *qx, const float *temperature, int B,
                      int gamma, int V, int r, uint64_t seed, uint64_t round_id, int32_t *n_accept_out,
                      int32_t *tokens_out, int32_t *out_offsets, float *diag_out, float *resid_out,
                      void *workspace, size_t workspace_bytes, void *stream) {
    return verify_common(target, n_target_rows, ell, row_offsets, U, head_rows, W2, wdtype, anchor, x, lse_q, qx,
                         temperature, B, gamma, V, r, seed, round_id, n_accept_out, tokens_out, out_offsets, diag_out,
                         resid_out, workspace, workspace_bytes, stream, 1);
}

size_t dspark_acceptance_workspace_size(int B, int gamma, int V, int r) {
    if (!sizes_ok(B, gamma, V, r)) return 0;
    return accept_bytes(B, gamma, V);
}

static int acceptance_common(const float *target, int n_target_rows, const int32_t *ell, const int32_t *row_offsets,
                             const float *U, const void *W1, const void *W2, int wdtype, const int32_t *anchor,
                             const int32_t *x, const float *lse_q, const float *temperature, int B, int gamma,
                             int V, int r, float *alpha_out, void *workspace, size_t workspace_bytes, void *stream,
                             int erow_mode) {
    if (!target || !ell || !U || !W1 || !W2 || !anchor || !x || !lse_q || !temperature || !alpha_out)
        return DSPARK_ERR_ARG;
    if (!sizes_ok(B, gamma, V, r) || n_target_rows < 1) return DSPARK_ERR_ARG;
    if (wdtype != DSPARK_BF16 && wdtype != DSPARK_F32) return DSPARK_ERR_ARG;
    if (!rank_supported(wdtype, r)) return DSPARK_ERR_UNSUPPORTED;
    if (!aligned16(W1) || !aligned16(W2)) return DSPARK_ERR_ARG;
    const AcceptPlan plan = accept_plan(B, gamma, V);
    size_t need = 0;
    accept_carve(nullptr, B, gamma, plan, &need);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DSPARK_ERR_WORKSPACE;
    const AcceptWork w = accept_carve(workspace, B, gamma, plan, nullptr);
    AcceptArgs a{};
    a.target = target;
    a.n_target_rows = n_target_rows;
    a.ell = ell;
    a.row_offsets = row_offsets;
    a.U = U;
    a.W1 = W1;
    a.W2 = W2;
    a.wdtype = wdtype;
    a.anchor = anchor;
    a.x = x;
    a.lse_q = lse_q;
    a.temperature = temperature;
    a.B = B;
    a.gamma = gamma;
    a.V = V;
    a.r = r;
    a.alpha_out = alpha_out;
    a.erow_mode = erow_mode;
    const hipError_t e = launch_accept(a, plan, w, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

int dspark_acceptance(const float *target, int n_target_rows, const int32_t *ell, const int32_t *row_offsets,
                      const float *U, const void *W1, const void *W2, int wdtype, const int32_t *anchor,
                      const int32_t *x, const float *lse_q, const float *temperature, int B, int gamma, int V,
                      int r, float *alpha_out, void *workspace, size_t workspace_bytes, void *stream) {
    return acceptance_common(target, n_target_rows, ell, row_offsets, U, W1, W2, wdtype, anchor, x, lse_q,
                             temperature, B, gamma, V, r, alpha_out, workspace, workspace_bytes, stream, 0);
}

int dspark_acceptance_rnn(const float *target, int n_target_rows, const int32_t *ell, const int32_t *row_offsets,
                          const float *U, const void *head_rows, const void *W2, int wdtype, const int32_t *anchor,
                          const int32_t *x, const float *lse_q, const float *temperature, int B, int gamma, int V,
                          int r, float *alpha_out, void *workspace, size_t workspace_bytes, void *stream) {
    return acceptance_common(target, n_target_rows, ell, row_offsets, U, head_rows, W2, wdtype, anchor, x, lse_q,
                             temperature, B, gamma, V, r, alpha_out, workspace, workspace_bytes, stream, 1);
}

int dspark_verify_check(const void *workspace, void *stream) {
    if (!workspace) return DSPARK_ERR_ARG;
    if (hipStreamSynchronize(static_cast<hipStream_t>(stream)) != hipSuccess) return DSPARK_ERR_HIP;
    int32_t st = 0;
    // the status word is the first region of the verify workspace
    if (hipMemcpy(&st, workspace, sizeof(st), hipMemcpyDeviceToHost) != hipSuccess) return DSPARK_ERR_HIP;
    return st == 0 ? DSPARK_OK : DSPARK_ERR_DEVICE_INPUT;
}

int dspark_debug_random_words(uint64_t seed, uint64_t round_id, int stream_id, int k, int req, int v0, int n,
                              uint32_t *out, void *stream) {
    if (!out || n < 0 || stream_id < 0 || stream_id > 4 || k < 0 || k >= (1 << 24) || v0 < 0) return DSPARK_ERR_ARG;
    const hipError_t e = launch_debug_words(uint32_t(seed), uint32_t(seed >> 32), uint32_t(round_id), stream_id,
                                            k, req, v0, n, out, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

int dspark_debug_bias_gemm(const void *W1, const void *W2, int wdtype, const int32_t *idx, int B, int V, int r,
                           float *rowmax_out, void *workspace, size_t workspace_bytes, void *stream) {
    if (!W1 || !W2 || !idx || !rowmax_out) return DSPARK_ERR_ARG;
    if (!sizes_ok(B, 1, V, r)) return DSPARK_ERR_ARG;
    if (wdtype != DSPARK_BF16 && wdtype != DSPARK_F32) return DSPARK_ERR_ARG;
    if (!rank_supported(wdtype, r)) return DSPARK_ERR_UNSUPPORTED;
    if (!aligned16(W1) || !aligned16(W2)) return DSPARK_ERR_ARG;
    const DraftPlan plan = draft_plan(B, V);
    size_t need = 0;
    draft_carve(nullptr, B, plan, &need);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DSPARK_ERR_WORKSPACE;
    const DraftWork w = draft_carve(workspace, B, plan, nullptr);
    const hipError_t e =
        launch_bias_gemm(W1, W2, wdtype, idx, B, V, r, plan, w, rowmax_out, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

int dspark_debug_gumbel(const uint32_t *words, int n, float *out, void *stream) {
    if (!words || !out || n < 0) return DSPARK_ERR_ARG;
    const hipError_t e = launch_debug_gumbel(words, n, out, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

int dspark_profile_enable(int enable) {
    Profiler &p = prof();
    std::lock_guard<std::mutex> g(p.mu);
    p.enabled = enable != 0;
    p.on.store(p.enabled, std::memory_order_release);
    return DSPARK_OK;
}

int dspark_profile_collect(void) {
    Profiler &p = prof();
    std::lock_guard<std::mutex> g(p.mu);
    int status = DSPARK_OK;
    for (const Pending &pd : p.pending) {
        float ms = 0.f;
        if (hipEventSynchronize(pd.stop) != hipSuccess || hipEventElapsedTime(&ms, pd.start, pd.stop) != hipSuccess) {
            status = DSPARK_ERR_HIP;
        } else {
            p.entries[size_t(pd.entry)].launches += 1;
            p.entries[size_t(pd.entry)].total_ms += ms;
        }
        p.pool.push_back(pd.start);
        p.pool.push_back(pd.stop);
    }
    p.pending.clear();
    return status;
}

int dspark_profile_count(void) {
    Profiler &p = prof();
    std::lock_guard<std::mutex> g(p.mu);
    return int(p.entries.size());
}

int dspark_profile_get(int i, const char **name, int64_t *launches, double *total_ms) {
    Profiler &p = prof();
    std::lock_guard<std::mutex> g(p.mu);
    if (i < 0 || i >= int(p.entries.size())) return DSPARK_ERR_ARG;
    if (name) *name = p.entries[size_t(i)].name.c_str();
    if (launches) *launches = p.entries[size_t(i)].launches;
    if (total_ms) *total_ms = p.entries[size_t(i)].total_ms;
    return DSPARK_OK;
}

int dspark_profile_reset(void) {
    Profiler &p = prof();
    std::lock_guard<std::mutex> g(p.mu);
    for (ProfEntry &e : p.entries) {
        e.launches = 0;
        e.total_ms = 0.0;
    }
    return DSPARK_OK;
}

}  // extern "C"

// ---------------------------------------------------------------- attention

namespace {

bool head_dim_supported(int d) { return d == 64 || d == 128 || d == 256; }

bool row_stride_ok(int64_t stride, int heads, int head_dim) {
    return stride >= int64_t(heads) * head_dim && stride <= DSPARK_MAX_ROW_STRIDE && stride % 8 == 0;
}

// Sizes and types of a cache call, in the order their errors are reported.
int cache_geometry(int dtype, const int32_t *row_offsets, int n_rows, int B, int max_pages, int n_kv_heads, int head_dim,
                   int cache_dtype, int n_pages, int page_size) {
    if (B < 1 || B > DSPARK_MAX_BATCH || n_rows < 0 || n_rows > DSPARK_MAX_ROWS || (!row_offsets && n_rows != B))
        return DSPARK_ERR_ARG;
    if (n_kv_heads < 1 || n_kv_heads > DSPARK_MAX_HEADS || head_dim < 1 || n_pages < 1 || max_pages < 1 || page_size < 1)
        return DSPARK_ERR_ARG;
    if (int64_t(max_pages) * page_size > DSPARK_MAX_CACHE_TOKENS) return DSPARK_ERR_ARG;
    if ((dtype != DSPARK_BF16 && dtype != DSPARK_F16 && dtype != DSPARK_F32 && dtype != DSPARK_E4M3) ||
        (cache_dtype != DSPARK_BF16 && cache_dtype != DSPARK_F16 && cache_dtype != DSPARK_F32 &&
         cache_dtype != DSPARK_E4M3))
        return DSPARK_ERR_ARG;
    if (dtype != DSPARK_BF16 && dtype != DSPARK_F16) return DSPARK_ERR_UNSUPPORTED;
    if (cache_dtype != dtype && cache_dtype != DSPARK_E4M3) return DSPARK_ERR_UNSUPPORTED;
    if (!head_dim_supported(head_dim)) return DSPARK_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return DSPARK_ERR_UNSUPPORTED;
    return DSPARK_OK;
}

// K and V of a write or read in pieces of 16 bytes: a launch holds fewer than
// 2^32 threads, each with four of them.
bool cache_launchable(int n_rows, int n_kv_heads, int head_dim) {
    return int64_t(n_rows) * 2 * n_kv_heads * (head_dim / 8) < (int64_t(1) << 34) - 1024;
}

int cache_buffers(const void *k_cache, const void *v_cache, const uint8_t *k_scale, const uint8_t *v_scale,
                  int cache_dtype) {
    if (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache)) return DSPARK_ERR_ARG;
    if (cache_dtype == DSPARK_E4M3 && (!k_scale || !v_scale || !aligned16(k_scale) || !aligned16(v_scale)))
        return DSPARK_ERR_ARG;
    return DSPARK_OK;
}

// Query heads against key-value heads, and the rows they make.
int head_geometry(int n_rows, int n_heads, int n_kv_heads) {
    if (n_heads < 1 || n_heads > DSPARK_MAX_HEADS || n_kv_heads < 1 || n_heads % n_kv_heads != 0) return DSPARK_ERR_ARG;
    if (int64_t(n_rows) * n_heads > INT32_MAX) return DSPARK_ERR_ARG;
    return DSPARK_OK;
}

// Query blocks of a prompt call, all sequences' last ones counted whole: a
// launch holds fewer than 2^32 threads, 256 a block.
bool prompt_launchable(int B, int n_rows, int n_heads, int n_kv_heads) {
    return int64_t(n_rows) * n_heads / 128 + (int64_t(B) + 1) * n_kv_heads < (1 << 24);
}

// Sizes and types of a rotation; v_heads: heads of values that are moved beside.
int rotary_geometry(int dtype, int n_rows, int n_heads, int n_kv_heads, int v_heads, int head_dim, int rotary_dim,
                    int norm_dtype, float eps) {
    if (n_heads < 0 || n_heads > DSPARK_MAX_HEADS || n_kv_heads < 0 || n_kv_heads > DSPARK_MAX_HEADS || head_dim < 1 ||
        rotary_dim < 0 || rotary_dim > head_dim || !(eps >= 0.f && eps <= 3.4e38f))
        return DSPARK_ERR_ARG;
    if (dtype != DSPARK_BF16 && dtype != DSPARK_F16 && dtype != DSPARK_F32 && dtype != DSPARK_E4M3) return DSPARK_ERR_ARG;
    if ((dtype != DSPARK_BF16 && dtype != DSPARK_F16) || (norm_dtype != dtype && norm_dtype != DSPARK_F32) ||
        !head_dim_supported(head_dim) || rotary_dim % 16 != 0)
        return DSPARK_ERR_UNSUPPORTED;
    // a launch holds fewer than 2^32 threads, 256 a workgroup
    if (n_heads + n_kv_heads > 0 && rotary_plan(n_rows, n_heads + n_kv_heads + v_heads, head_dim, false).blocks >= (1 << 24))
        return DSPARK_ERR_ARG;
    return DSPARK_OK;
}

// Rows that are turned into rows: both there, or no heads at all.
bool rotary_rows_ok(const void *in, const void *out, int64_t stride, int64_t out_stride, int heads, int head_dim) {
    if (heads == 0) return true;
    return in && out && aligned16(in) && aligned16(out) && row_stride_ok(stride, heads, head_dim) &&
           row_stride_ok(out_stride, heads, head_dim) && (in != out || stride == out_stride);
}

// Whether a windowed call goes by query blocks (prompt.hpp), or row by row as paged
// attention does (float16 rows over 8 bits always: their range there needs the
// rows' kernel, though a chunk's blocks all walk from its first window to its last
// row: 2000 rows behind 1024 tokens 363 us, 67 for bfloat16 rows).  Us a call, rows / blocks (window 1000, four query heads a key
// head; 255 single rows beside a chunk of 2000, window 1024, 715 / 270; 64 requests of 8 key heads, D = 128: 16 rows 88 / 96, 20 138 / 85, 32 167 /
// 117, 64 333 / 135; over 8 bits 16 rows 76 / 120, 32 141 / 142, 64 278 / 163; D = 64:
// 32 rows 66 / 98, 48 98 / 103, 64 130 / 106, over 8 bits 32 83 / 114, 64 168 / 129;
// 16 requests, D = 256: 16 rows 56 / 77, 20 86 / 78, 48 148 / 85, over 8 bits 32 88 /
// 98, 64 179 / 159; one request, D = 128: 4 rows 15.2 / 15.0, 8 18.6 / 15.2, 16
// 27 / 16).
bool window_in_chunks(long long segments, int max_rows, int group, int head_dim, int dtype, int cache_dtype) {
    const bool e4 = cache_dtype == DSPARK_E4M3;
    if (e4 && dtype != DSPARK_BF16) return false;
    const int64_t queries = int64_t(max_rows) * group;
    return queries > (head_dim == 64 ? 192 : e4 ? 128 : 64) || (!e4 && queries > 16 && segments <= 16);
}

// the kernels multiply by scale * log2(e), which has to be finite
bool scale_ok(float scale) { return scale > 0.f && scale <= 2.3e38f; }

}  // namespace

extern "C" {

int dspark_kv_write(const void *k, const void *v, int64_t k_stride, int64_t v_stride, int dtype,
                    const int32_t *row_offsets, int n_rows, const int32_t *cache_len, const int32_t *page_table, int B,
                    int max_pages, int n_kv_heads, int head_dim, void *k_cache, void *v_cache, uint8_t *k_scale,
                    uint8_t *v_scale, int cache_dtype, int n_pages, int page_size, void *stream) {
    int st = cache_geometry(dtype, row_offsets, n_rows, B, max_pages, n_kv_heads, head_dim, cache_dtype, n_pages,
                            page_size);
    if (st != DSPARK_OK) return st;
    if (!cache_launchable(n_rows, n_kv_heads, head_dim)) return DSPARK_ERR_ARG;
    if (n_rows == 0) return DSPARK_OK;
    if (!k || !v || !cache_len || !page_table || !aligned16(k) || !aligned16(v)) return DSPARK_ERR_ARG;
    if (!row_stride_ok(k_stride, n_kv_heads, head_dim) || !row_stride_ok(v_stride, n_kv_heads, head_dim))
        return DSPARK_ERR_ARG;
    st = cache_buffers(k_cache, v_cache, k_scale, v_scale, cache_dtype);
    if (st != DSPARK_OK) return st;
    CacheArgs a{};
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.dtype = dtype;
    a.row_offsets = row_offsets;
    a.start = cache_len;
    a.page_table = page_table;
    a.B = B;
    a.n_rows = n_rows;
    a.max_pages = max_pages;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.cache_dtype = cache_dtype;
    a.n_pages = n_pages;
    a.page_size = page_size;
    return launch_cache(a, true, static_cast<hipStream_t>(stream)) == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

int dspark_kv_read(const void *k_cache, const void *v_cache, const uint8_t *k_scale, const uint8_t *v_scale,
                   int cache_dtype, int n_pages, int page_size, const int32_t *row_offsets, int n_rows,
                   const int32_t *first, const int32_t *page_table, int B, int max_pages, int n_kv_heads, int head_dim,
                   void *k_out, void *v_out, int dtype, void *stream) {
    int st = cache_geometry(dtype, row_offsets, n_rows, B, max_pages, n_kv_heads, head_dim, cache_dtype, n_pages,
                            page_size);
    if (st != DSPARK_OK) return st;
    if (!cache_launchable(n_rows, n_kv_heads, head_dim)) return DSPARK_ERR_ARG;
    if (n_rows == 0) return DSPARK_OK;
    if (!k_out || !v_out || !page_table || !aligned16(k_out) || !aligned16(v_out)) return DSPARK_ERR_ARG;
    st = cache_buffers(k_cache, v_cache, k_scale, v_scale, cache_dtype);
    if (st != DSPARK_OK) return st;
    CacheArgs a{};
    a.k_out = k_out;
    a.v_out = v_out;
    a.dtype = dtype;
    a.row_offsets = row_offsets;
    a.start = first;
    a.page_table = page_table;
    a.B = B;
    a.n_rows = n_rows;
    a.max_pages = max_pages;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.k_cache = const_cast<void *>(k_cache);
    a.v_cache = const_cast<void *>(v_cache);
    a.k_scale = const_cast<uint8_t *>(k_scale);
    a.v_scale = const_cast<uint8_t *>(v_scale);
    a.cache_dtype = cache_dtype;
    a.n_pages = n_pages;
    a.page_size = page_size;
    return launch_cache(a, false, static_cast<hipStream_t>(stream)) == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

int dspark_rotary(const void *q, const void *k, int64_t q_stride, int64_t k_stride, int dtype,
                  const int32_t *row_offsets, int n_rows, const int32_t *first, int B, int n_heads, int n_kv_heads,
                  int head_dim, const float *inv_freq, int rotary_dim, int neighbours, const void *q_norm,
                  const void *k_norm, int norm_dtype, float eps, void *q_out, void *k_out, int64_t q_out_stride,
                  int64_t k_out_stride, void *stream) {
    if (B < 1 || B > DSPARK_MAX_BATCH || n_rows < 0 || n_rows > DSPARK_MAX_ROWS || (!row_offsets && n_rows != B))
        return DSPARK_ERR_ARG;
    int st = rotary_geometry(dtype, n_rows, n_heads, n_kv_heads, 0, head_dim, rotary_dim, norm_dtype, eps);
    if (st != DSPARK_OK) return st;
    if (n_heads + n_kv_heads < 1) return DSPARK_ERR_ARG;
    if (n_rows == 0) return DSPARK_OK;
    if ((!inv_freq && rotary_dim > 0) || !rotary_rows_ok(q, q_out, q_stride, q_out_stride, n_heads, head_dim) ||
        !rotary_rows_ok(k, k_out, k_stride, k_out_stride, n_kv_heads, head_dim))
        return DSPARK_ERR_ARG;
    RotaryArgs a{};
    a.c.k = k;
    a.c.k_stride = k_stride;
    a.c.k_out = k_out;
    a.c.dtype = dtype;
    a.c.row_offsets = row_offsets;
    a.c.start = first;
    a.c.B = B;
    a.c.n_rows = n_rows;
    a.c.n_kv_heads = n_kv_heads;
    a.c.head_dim = head_dim;
    a.q = q;
    a.q_out = q_out;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.k_out_stride = k_out_stride;
    a.n_heads = n_heads;
    a.inv_freq = inv_freq;
    a.rot = rotary_dim;
    a.neighbours = neighbours != 0;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.norm_dtype = norm_dtype;
    a.eps = eps;
    const RotaryPlan plan = rotary_plan(n_rows, n_heads + n_kv_heads, head_dim, false);
    return launch_rotary(a, plan, static_cast<hipStream_t>(stream)) == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

int dspark_kv_append(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                     int64_t v_stride, int dtype, const int32_t *row_offsets, int n_rows, const int32_t *cache_len,
                     const int32_t *page_table, int B, int max_pages, int n_heads, int n_kv_heads, int head_dim,
                     const float *inv_freq, int rotary_dim, int neighbours, const void *q_norm, const void *k_norm,
                     int norm_dtype, float eps, void *q_out, int64_t q_out_stride, void *k_cache, void *v_cache,
                     uint8_t *k_scale, uint8_t *v_scale, int cache_dtype, int n_pages, int page_size, void *stream) {
    int st = cache_geometry(dtype, row_offsets, n_rows, B, max_pages, n_kv_heads, head_dim, cache_dtype, n_pages,
                            page_size);
    if (st != DSPARK_OK) return st;
    st = rotary_geometry(dtype, n_rows, n_heads, n_kv_heads, n_kv_heads, head_dim, rotary_dim, norm_dtype, eps);
    if (st != DSPARK_OK) return st;
    if (n_rows == 0) return DSPARK_OK;
    if ((!inv_freq && rotary_dim > 0) || !rotary_rows_ok(q, q_out, q_stride, q_out_stride, n_heads, head_dim))
        return DSPARK_ERR_ARG;
    if (!k || !v || !cache_len || !page_table || !aligned16(k) || !aligned16(v)) return DSPARK_ERR_ARG;
    if (!row_stride_ok(k_stride, n_kv_heads, head_dim) || !row_stride_ok(v_stride, n_kv_heads, head_dim))
        return DSPARK_ERR_ARG;
    st = cache_buffers(k_cache, v_cache, k_scale, v_scale, cache_dtype);
    if (st != DSPARK_OK) return st;
    RotaryArgs a{};
    a.c.k = k;
    a.c.v = v;
    a.c.k_stride = k_stride;
    a.c.v_stride = v_stride;
    a.c.dtype = dtype;
    a.c.row_offsets = row_offsets;
    a.c.start = cache_len;
    a.c.page_table = page_table;
    a.c.B = B;
    a.c.n_rows = n_rows;
    a.c.max_pages = max_pages;
    a.c.n_kv_heads = n_kv_heads;
    a.c.head_dim = head_dim;
    a.c.k_cache = k_cache;
    a.c.v_cache = v_cache;
    a.c.k_scale = k_scale;
    a.c.v_scale = v_scale;
    a.c.cache_dtype = cache_dtype;
    a.c.n_pages = n_pages;
    a.c.page_size = page_size;
    a.q = q;
    a.q_out = q_out;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.n_heads = n_heads;
    a.inv_freq = inv_freq;
    a.rot = rotary_dim;
    a.neighbours = neighbours != 0;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.norm_dtype = norm_dtype;
    a.eps = eps;
    const RotaryPlan plan = rotary_plan(n_rows, n_heads + 2 * n_kv_heads, head_dim, true);
    return launch_rotary(a, plan, static_cast<hipStream_t>(stream)) == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

size_t dspark_paged_attention_workspace_size(int max_rows, int n_heads, int n_kv_heads, int head_dim) {
    if (max_rows < 1 || head_geometry(0, n_heads, n_kv_heads) != DSPARK_OK || !head_dim_supported(head_dim)) return 0;
    size_t bytes = 0;
    for (const bool e4 : {false, true}) {
        size_t need = 0;
        // the largest grid, whatever the batch
        const PagedSizes z{DSPARK_MAX_ROWS, DSPARK_MAX_BATCH, DSPARK_MAX_CACHE_TOKENS, max_rows, n_heads, n_kv_heads,
                           head_dim, e4};
        paged_carve(nullptr, paged_plan(z), head_dim, &need);
        bytes = need > bytes ? need : bytes;
    }
    return bytes;
}

int dspark_paged_attention(const void *q, int64_t q_stride, int dtype, const int32_t *row_offsets, int n_rows,
                           int max_rows, const int32_t *cache_len, const int32_t *page_table, int B, int max_pages,
                           int n_heads, int n_kv_heads, int head_dim, const void *k_cache, const void *v_cache,
                           const uint8_t *k_scale, const uint8_t *v_scale, int cache_dtype, int n_pages, int page_size,
                           float scale, int causal, void *out, float *lse_out, void *workspace, size_t workspace_bytes,
                           void *stream) {
    int st = cache_geometry(dtype, row_offsets, n_rows, B, max_pages, n_kv_heads, head_dim, cache_dtype, n_pages,
                            page_size);
    if (st != DSPARK_OK) return st;
    st = head_geometry(n_rows, n_heads, n_kv_heads);
    if (st != DSPARK_OK) return st;
    if (max_rows < 1 || !scale_ok(scale)) return DSPARK_ERR_ARG;
    if (n_rows == 0) return DSPARK_OK;
    if (!q || !cache_len || !page_table || !out || !aligned16(q) || !aligned16(out)) return DSPARK_ERR_ARG;
    if (!row_stride_ok(q_stride, n_heads, head_dim)) return DSPARK_ERR_ARG;
    st = cache_buffers(k_cache, v_cache, k_scale, v_scale, cache_dtype);
    if (st != DSPARK_OK) return st;
    const PagedSizes z{n_rows, B, (long long)max_pages * page_size, max_rows, n_heads, n_kv_heads, head_dim,
                       cache_dtype == DSPARK_E4M3};
    const PagedPlan plan = paged_plan(z);
    size_t need = 0;
    paged_carve(nullptr, plan, head_dim, &need);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DSPARK_ERR_WORKSPACE;
    const PagedWork w = paged_carve(workspace, plan, head_dim, nullptr);
    PagedArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.dtype = dtype;
    a.row_offsets = row_offsets;
    a.start = cache_len;
    a.page_table = page_table;
    a.B = B;
    a.n_rows = n_rows;
    a.max_pages = max_pages;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.cache_dtype = cache_dtype;
    a.n_pages = n_pages;
    a.page_size = page_size;
    a.scale = scale;
    a.causal = causal != 0;
    a.out = out;
    a.lse = lse_out;
    return launch_paged(a, plan, w, static_cast<hipStream_t>(stream)) == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

size_t dspark_window_attention_workspace_size(int max_rows, int n_heads, int n_kv_heads, int head_dim) {
    const size_t rows = dspark_paged_attention_workspace_size(max_rows, n_heads, n_kv_heads, head_dim);
    if (rows == 0) return 0;
    size_t chunks = 0;
    PromptPlan plan{};  // the most parts there are
    plan.slots = kWindowParts / 2;
    plan.nsplit = 2;
    prompt_carve(nullptr, plan, 1, head_dim, &chunks);
    return rows > chunks ? rows : chunks;
}

int dspark_window_attention(const void *q, int64_t q_stride, int dtype, const int32_t *row_offsets, int n_rows,
                            int max_rows, const int32_t *cache_len, const int32_t *page_table, int B, int max_pages,
                            int n_heads, int n_kv_heads, int head_dim, const void *k_cache, const void *v_cache,
                            const uint8_t *k_scale, const uint8_t *v_scale, int cache_dtype, int n_pages,
                            int page_size, int window, int sinks, float scale, void *out, float *lse_out,
                            void *workspace, size_t workspace_bytes, void *stream) {
    int st = cache_geometry(dtype, row_offsets, n_rows, B, max_pages, n_kv_heads, head_dim, cache_dtype, n_pages,
                            page_size);
    if (st != DSPARK_OK) return st;
    st = head_geometry(n_rows, n_heads, n_kv_heads);
    if (st != DSPARK_OK) return st;
    if (max_rows < 1 || !scale_ok(scale) || window < 1 || sinks < 0) return DSPARK_ERR_ARG;
    if (n_rows == 0) return DSPARK_OK;
    if (!q || !cache_len || !page_table || !out || !aligned16(q) || !aligned16(out)) return DSPARK_ERR_ARG;
    if (!row_stride_ok(q_stride, n_heads, head_dim)) return DSPARK_ERR_ARG;
    st = cache_buffers(k_cache, v_cache, k_scale, v_scale, cache_dtype);
    if (st != DSPARK_OK) return st;
    // no request has more tokens than these
    window = window < DSPARK_MAX_CACHE_TOKENS ? window : DSPARK_MAX_CACHE_TOKENS;
    sinks = sinks < DSPARK_MAX_CACHE_TOKENS ? sinks : DSPARK_MAX_CACHE_TOKENS;
    // what a request of the usual number of rows walks at most: sinks and windows in whole tiles
    const long long table = (long long)max_pages * page_size, walked = (long long)window + sinks + max_rows + 64;
    size_t need = 0;
    if (window_in_chunks((long long)B * n_kv_heads, max_rows, n_heads / n_kv_heads, head_dim, dtype, cache_dtype) &&
        prompt_launchable(B, n_rows, n_heads, n_kv_heads)) {
        const PromptPlan plan = window_chunk_plan(B, n_rows, walked < table ? walked : table, n_heads, n_kv_heads, head_dim);
        prompt_carve(nullptr, plan, n_kv_heads, head_dim, &need);
        if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DSPARK_ERR_WORKSPACE;
        const PromptWork w = prompt_carve(workspace, plan, n_kv_heads, head_dim, nullptr);
        PromptArgs a{};
        a.q = q;
        a.k = k_cache;
        a.v = v_cache;
        a.q_stride = q_stride;
        a.dtype = dtype;
        a.q_offsets = row_offsets;
        a.start = cache_len;
        a.k_scale = cache_dtype == DSPARK_E4M3 ? k_scale : nullptr;  // which tells the kernel the cache's type
        a.v_scale = cache_dtype == DSPARK_E4M3 ? v_scale : nullptr;
        a.page_table = page_table;
        a.B = B;
        a.n_rows = n_rows;
        a.max_pages = max_pages;
        a.n_heads = n_heads;
        a.n_kv_heads = n_kv_heads;
        a.head_dim = head_dim;
        a.n_pages = n_pages;
        a.page_size = page_size;
        a.scale = scale;
        a.causal = 1;
        a.window = window;
        a.sinks = sinks;
        a.out = out;
        a.lse = lse_out;
        return launch_window_chunks(a, plan, w, static_cast<hipStream_t>(stream)) == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
    }
    const PagedSizes z{n_rows, B, walked < table ? walked : table, max_rows, n_heads, n_kv_heads, head_dim,
                       cache_dtype == DSPARK_E4M3, walked < table};
    const PagedPlan plan = paged_plan(z);
    paged_carve(nullptr, plan, head_dim, &need);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DSPARK_ERR_WORKSPACE;
    const PagedWork w = paged_carve(workspace, plan, head_dim, nullptr);
    PagedArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.dtype = dtype;
    a.row_offsets = row_offsets;
    a.start = cache_len;
    a.page_table = page_table;
    a.B = B;
    a.n_rows = n_rows;
    a.max_pages = max_pages;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.cache_dtype = cache_dtype;
    a.n_pages = n_pages;
    a.page_size = page_size;
    a.scale = scale;
    a.causal = 1;
    a.window = window;
    a.sinks = sinks;
    a.out = out;
    a.lse = lse_out;
    return launch_window_rows(a, plan, w, static_cast<hipStream_t>(stream)) == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

size_t dspark_prompt_attention_workspace_size(int B, int n_rows, int n_kv_rows, int n_heads, int n_kv_heads,
                                              int head_dim) {
    if (B < 1 || B > DSPARK_MAX_BATCH || n_rows < 0 || n_rows > DSPARK_MAX_ROWS || n_kv_rows < 0 ||
        n_kv_rows > DSPARK_MAX_ROWS || head_geometry(n_rows, n_heads, n_kv_heads) != DSPARK_OK ||
        !prompt_launchable(B, n_rows, n_heads, n_kv_heads) || !head_dim_supported(head_dim))
        return 0;
    size_t bytes = 0;
    prompt_carve(nullptr, prompt_plan(B, n_rows, n_kv_rows, n_heads, n_kv_heads, head_dim), n_kv_heads, head_dim, &bytes);
    return bytes;
}

int dspark_prompt_attention(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, int dtype, const int32_t *row_offsets, int n_rows,
                            const int32_t *kv_offsets, int n_kv_rows, int B, int n_heads, int n_kv_heads, int head_dim,
                            float scale, int causal, void *out, float *lse_out, void *workspace,
                            size_t workspace_bytes, void *stream) {
    if (B < 1 || B > DSPARK_MAX_BATCH || n_rows < 0 || n_rows > DSPARK_MAX_ROWS || n_kv_rows < 0 ||
        n_kv_rows > DSPARK_MAX_ROWS || !row_offsets || (!kv_offsets && n_kv_rows != n_rows) || head_dim < 1)
        return DSPARK_ERR_ARG;
    const int st = head_geometry(n_rows, n_heads, n_kv_heads);
    if (st != DSPARK_OK) return st;
    if (!prompt_launchable(B, n_rows, n_heads, n_kv_heads)) return DSPARK_ERR_ARG;
    if (dtype != DSPARK_BF16 && dtype != DSPARK_F16 && dtype != DSPARK_F32 && dtype != DSPARK_E4M3)
        return DSPARK_ERR_ARG;
    if ((dtype != DSPARK_BF16 && dtype != DSPARK_F16) || !head_dim_supported(head_dim)) return DSPARK_ERR_UNSUPPORTED;
    if (!scale_ok(scale)) return DSPARK_ERR_ARG;
    if (n_rows == 0) return DSPARK_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out) || !row_stride_ok(q_stride, n_heads, head_dim))
        return DSPARK_ERR_ARG;
    if (n_kv_rows > 0 && (!k || !v || !aligned16(k) || !aligned16(v) || !row_stride_ok(k_stride, n_kv_heads, head_dim) ||
                          !row_stride_ok(v_stride, n_kv_heads, head_dim)))
        return DSPARK_ERR_ARG;
    const PromptPlan plan = prompt_plan(B, n_rows, n_kv_rows, n_heads, n_kv_heads, head_dim);
    size_t need = 0;
    prompt_carve(nullptr, plan, n_kv_heads, head_dim, &need);
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DSPARK_ERR_WORKSPACE;
    const PromptWork w = prompt_carve(workspace, plan, n_kv_heads, head_dim, nullptr);
    PromptArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.dtype = dtype;
    a.q_offsets = row_offsets;
    a.kv_offsets = kv_offsets;
    a.B = B;
    a.n_rows = n_rows;
    a.n_kv_rows = n_kv_rows;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.scale = scale;
    a.causal = causal != 0;
    a.out = out;
    a.lse = lse_out;
    return launch_prompt(a, plan, w, static_cast<hipStream_t>(stream)) == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

// ---------------------------------------------------------------- rules on logits

int dspark_logit_rules(const void *logits, int64_t stride, int dtype, const int32_t *row_offsets, int n_rows, int B,
                       int V, const int32_t *history, int max_history, const int32_t *history_len,
                       const int32_t *prompt_len, const int32_t *drafts, int gamma, const float *repetition,
                       const float *frequency, const float *presence, const int32_t *bias_offsets,
                       const int32_t *bias_ids, const float *bias_values, int n_biases, const int32_t *masks,
                       int n_masks, int64_t mask_stride, const int32_t *mask_index, float *out, int64_t out_stride,
                       void *stream) {
    if (B < 1 || B > DSPARK_MAX_BATCH || n_rows < 0 || n_rows > DSPARK_MAX_ROWS || (!row_offsets && n_rows != B) ||
        V < 1 || V > DSPARK_MAX_VOCAB || stride < V || stride > DSPARK_MAX_ROW_STRIDE || out_stride < V ||
        out_stride > DSPARK_MAX_ROW_STRIDE)
        return DSPARK_ERR_ARG;
    if (int64_t(B) * ((V + 4095) / 4096) >= (1 << 23)) return DSPARK_ERR_ARG;  // a launch holds fewer than 2^32 threads
    if (dtype != DSPARK_BF16 && dtype != DSPARK_F16 && dtype != DSPARK_F32 && dtype != DSPARK_E4M3) return DSPARK_ERR_ARG;
    if (dtype == DSPARK_E4M3) return DSPARK_ERR_UNSUPPORTED;
    // (the kernel steps past the end of a text or a list by less than 2^14)
    if (history && (max_history < 0 || max_history > DSPARK_MAX_CACHE_TOKENS || !history_len)) return DSPARK_ERR_ARG;
    if (drafts && (gamma < 0 || gamma > DSPARK_MAX_GAMMA)) return DSPARK_ERR_ARG;
    if (n_biases < 0 || n_biases > DSPARK_MAX_CACHE_TOKENS || (bias_offsets && n_biases > 0 && (!bias_ids || !bias_values))) return DSPARK_ERR_ARG;
    if (masks && (n_masks < 0 || mask_stride < (V + 31) / 32 || mask_stride > DSPARK_MAX_ROW_STRIDE || !mask_index))
        return DSPARK_ERR_ARG;
    if (n_rows == 0) return DSPARK_OK;
    const uintptr_t at = reinterpret_cast<uintptr_t>(logits), to = reinterpret_cast<uintptr_t>(out);
    if (!logits || !out || at % (dtype == DSPARK_F32 ? 4 : 2) != 0 || to % 4 != 0) return DSPARK_ERR_ARG;
    if (at == to && (dtype != DSPARK_F32 || stride != out_stride)) return DSPARK_ERR_ARG;
    RulesArgs a{};
    a.logits = logits;
    a.stride = stride;
    a.dtype = dtype;
    a.row_offsets = row_offsets;
    a.n_rows = n_rows;
    a.B = B;
    a.V = V;
    a.history = history;
    a.history_len = history_len;
    a.prompt_len = prompt_len;
    a.max_history = max_history;
    a.drafts = drafts;
    a.gamma = gamma;
    a.repetition = repetition;
    a.frequency = frequency;
    a.presence = presence;
    a.bias_offsets = bias_offsets;
    a.bias_ids = bias_ids;
    a.bias_values = bias_values;
    a.n_biases = n_biases;
    a.masks = masks;
    a.mask_index = masks ? mask_index : nullptr;
    a.n_masks = n_masks;
    a.mask_stride = mask_stride;
    a.out = out;
    a.out_stride = out_stride;
    return launch_rules(a, static_cast<hipStream_t>(stream)) == hipSuccess ? DSPARK_OK : DSPARK_ERR_HIP;
}

}  // extern "C"
