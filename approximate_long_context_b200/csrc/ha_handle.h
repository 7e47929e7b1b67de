// ha_handle.h -- the handle behind hyper_attn_t and the helpers every C entry point uses: error text, device
// guard, profiling brackets. Host code only.
#pragma once

#include <cstdarg>
#include <cstdio>
#include <string>
#include <vector>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "../../include/hyper_attn.h"
#include "ha_internal.h"

struct hyper_attn_s {
    int device = 0;
    ha_options opt{};
    std::string err;
    // device workspace (grow-only)
    unsigned char *ws = nullptr;
    size_t ws_bytes = 0;
    // page-locked staging of the draws, and the event that guards its reuse
    unsigned char *pin = nullptr;
    size_t pin_bytes = 0;
    cudaEvent_t pin_free = nullptr;
    // device copies for hyper_attn_forward_host (grow-only), and its copy streams and chunk events
    unsigned char *io = nullptr;
    size_t io_bytes = 0;
    cudaStream_t cs_in = nullptr, cs_out = nullptr;
    std::vector<cudaEvent_t> pipe_ev;
    // test hook: the number of upcoming allocations to fail (hyper_attn_test_fail_alloc)
    int fail_alloc = 0;
    // draws currently resident in the workspace, and a host copy of their projection matrix ([d][r]), which the
    // hash kernel takes as launch parameters
    bool draws_valid = false;
    std::vector<float> hostP;
    uint64_t dk_seed = 0;
    int dk_d = 0, dk_r = 0, dk_m = 0, dk_causal = 0;
    int64_t dk_bh = 0, dk_n = 0, dk_base = 0, dk_off = 0;
    // layout of the last forward (for debug copies)
    struct Layout {
        size_t status, P, S, rank, near, lse, perm_tmp, hist, Opart, Lpart, end;
        std::vector<size_t> perm, inv;
        std::vector<size_t> perm_bytes;
        size_t rank_bytes, near_bytes, lse_bytes;
        // row-norm sampling (0 bytes when off): squared norms, chunk sums, cumulative sums, draws, log weights
        size_t rn_nrm, rn_csum, rn_cdf, rn_S, rn_lw, rn_bytes;
    } lay{};
    bool have_last = false;
    // the forward pass runs for a backward pass: fp32 O, per-row log normalisers captured (causal: final ones)
    bool bwd = false;
    int last_launches = 0;
    int last_kernel = 0;
    // profiling: event pairs recorded around kernel-class launches
    bool profiling = false;
    std::vector<cudaEvent_t> ev_pool;
    struct Rec { int cls, launches; size_t e0, e1; };
    std::vector<Rec> recs;
    size_t ev_used = 0;
    // status word of the serving entry points: allocated with the handle and never moved, so that a captured
    // graph may go on writing to it; the word kTakenStatus behind it is what hyper_attn_status took
    static constexpr int kTakenStatus = 32;
    int *serve_status = nullptr;
    int sms = 0;
};

inline int fail(hyper_attn_t h, int code, const char *fmt, ...) __attribute__((format(printf, 3, 4)));
inline int fail(hyper_attn_t h, int code, const char *fmt, ...) {
    if (h) {
        char buf[512];
        va_list ap;
        va_start(ap, fmt);
        vsnprintf(buf, sizeof buf, fmt, ap);
        va_end(ap);
        h->err = buf;
    }
    return code;
}

#define HA_CUDA(h, call)                                                                                \
    do {                                                                                                \
        cudaError_t e_ = (call);                                                                        \
        if (e_ != cudaSuccess) return fail((h), HA_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_));  \
    } while (0)

struct DeviceGuard {
    int prev = -1;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev != dev) cudaSetDevice(dev);
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

// While one lives, the calls of this thread that allocate or free do not end a capture that is under way somewhere else.
class RelaxedCapture {
public:
    RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode_); }
    ~RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode_); }

private:
    cudaStreamCaptureMode mode_ = cudaStreamCaptureModeRelaxed;
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Brackets one kernel class's enqueue: an NVTX range (a no-op unless a tracing tool is attached) and, with
// profiling on, two events from the handle's pool (grown on demand) on the stream. Not under capture: events recorded
// there have no time, and no later read could pass them.
class ProfScope {
public:
    ProfScope(hyper_attn_t h, int cls, const char *name, cudaStream_t st) : h_(h), cls_(cls), st_(st) {
        nvtxRangePushA(name);
        cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
        if (!h->profiling || cudaStreamIsCapturing(st, &capture) != cudaSuccess || capture != cudaStreamCaptureStatusNone) return;
        while (h->ev_pool.size() < h->ev_used + 2) {
            cudaEvent_t e;
            if (cudaEventCreate(&e) != cudaSuccess) return;
            h->ev_pool.push_back(e);
        }
        at_ = static_cast<long>(h->ev_used);
        h->ev_used += 2;
        cudaEventRecord(h->ev_pool[at_], st);
    }
    void end(int launches) {
        nvtxRangePop();
        open_ = false;
        if (at_ < 0) return;
        cudaEventRecord(h_->ev_pool[at_ + 1], st_);
        h_->recs.push_back({cls_, launches > 0 ? launches : 0, static_cast<size_t>(at_), static_cast<size_t>(at_ + 1)});
    }
    ~ProfScope() {
        if (open_) nvtxRangePop();
    }

private:
    hyper_attn_t h_;
    int cls_;
    cudaStream_t st_;
    long at_ = -1;
    bool open_ = true;
};
