// prefill_ws.h -- what the prefill attention (K2) of a quantised cache needs
// beside the cache: a bf16 workspace of one layer's rows, and K2's launches on
// it.  Also what such caches' host sides share: the rotary tables, and scopes.
#pragma once

#include <cuda_runtime.h>

#include "k2_parts.h"
#include "qa.h"
#include "qa_internal.h"

namespace qa {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr size_t align256(size_t bytes) { return (bytes + 255) & ~size_t(255); }

// Makes the cache's device current for one call.
class DeviceScope {
  public:
    explicit DeviceScope(int device) {
        ok_ = cudaGetDevice(&before_) == cudaSuccess &&
              (before_ == device || cudaSetDevice(device) == cudaSuccess);
        back_ = ok_ && before_ != device;
    }
    ~DeviceScope() {
        if (back_) cudaSetDevice(before_);
    }
    bool ok() const { return ok_; }

  private:
    int before_ = 0;
    bool ok_ = false, back_ = false;
};

// Allocations of a call that is not captured itself are no part of a capture
// that is under way on another stream.
class OutsideCapture {
  public:
    OutsideCapture() { cudaThreadExchangeStreamCaptureMode(&mode_); }
    ~OutsideCapture() { cudaThreadExchangeStreamCaptureMode(&mode_); }

  private:
    cudaStreamCaptureMode mode_ = cudaStreamCaptureModeRelaxed;
};

// The body of an entry point whose host side allocates: no exception leaves it.
template <typename F>
qa_status no_throw(F &&body) {
    try {
        return body();
    } catch (...) {
        return QA_ERR_CUDA;
    }
}

// The rotary tables of the quantised caches that are alive.  A table depends on
// theta and head_dim alone and a longer one begins with the shorter ones, so
// caches of one device share it.
// A table of at least `rows` positions on the current device; null on error.
const float2 *rope_table_take(int device, float theta, int D, int rows);
// Gives one back (or null); the caller has synchronised its device.
void rope_table_give(const float2 *tab);

// K2's launches for one group of sequences.
struct K2Job {
    K2ScaledPartParams k2;
    K2JoinParams join;
    bool parts;                     // k2 is of parts, join follows it
    bool scaled;                    // the rows have factors
    int items;
};

// Prefill attention reads one layer's rows in bf16: the sequences of a launch,
// dequantised, laid out [slot][kv head][capacity][head_dim].  Every row that it
// reads is written before it, so nothing is zeroed.
class PrefillWorkspace {
  public:
    // factors: the rows of 64 positions may have some (K2Factors).
    void init(const qa_config &cfg, int num_sms, bool factors = false);
    void release();                 // frees it; the device has been synchronised
    // The workspace and its event, allocated by the first call; false on error.
    bool take();
    int slots() const { return slots_; }
    __nv_bfloat16 *rows(int kv) const { return ws_[kv]; }
    int64_t head_stride() const { return static_cast<int64_t>(cfg_.capacity) * cfg_.head_dim; }
    int64_t seq_stride() const { return head_stride() * cfg_.n_kv_heads; }
    float4 *factors() const { return factors_; }  // [slot][kv head][factor_stride()]
    int factor_stride() const { return (cfg_.capacity + 127) / 128 * 2; }
    cudaEvent_t free_event() const { return free_; }
    size_t bytes() const;           // of all that may come to be allocated
    // K2's launches for n sequences: ntok[i] new tokens at start[i] .., whose rows
    // in qp and out begin at cu[i] (cu[n]: their number, above 0).  scaled: by the factors
    // (no window).  False when a tensor map cannot be made or the sums of parts find no
    // memory.
    bool plan(int window, int n, const int32_t *start, const int32_t *ntok, const int *cu,
              __nv_bfloat16 *qp, uint32_t *err, bool scaled, K2Job &job);
    cudaError_t launch(K2Job &job, cudaStream_t s) const;

  private:
    size_t kv_bytes() const;        // of K or of V
    size_t factor_bytes() const;
    // The parts of a launch have at most two heads' blocks of 128 rows per SM;
    // caches this short are not cut.
    static constexpr int kPartsCapacity = 1024;
    size_t part_rows() const { return static_cast<size_t>(num_sms_) * 256; }
    bool take_sums();

    qa_config cfg_{};
    int num_sms_ = 0, slots_ = 0, G_ = 1;
    bool has_factors_ = false;
    __nv_bfloat16 *ws_[2] = {};     // taken by the first call that needs it
    float4 *factors_ = nullptr;     // behind it, if any
    float *part_o_ = nullptr;       // sums of the parts of a block's keys (k2_parts.h); likewise
    float2 *part_ml_ = nullptr;
    cudaEvent_t free_ = nullptr;    // the last prefill that used the workspace
};

}  // namespace qa
