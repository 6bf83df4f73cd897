// prefill_ws.cu -- the host side that the quantised caches share: their rotary
// tables, and the workspace and launches of prefill attention on one layer.
#include <algorithm>
#include <cmath>
#include <mutex>
#include <vector>

#include "prefill_ws.h"
#include "q4_internal.h"
#include "q4_plan.h"

namespace {

// Angles of the pairs of dims: position * theta^(-2i/D), i below D / 2.
struct RopeFreqs {
    double f[64];
};

// As qa::fill_rope_table: the same product in fp64, its cosine and sine in fp64,
// rounded once (2^20 positions, D 64 and 128, theta 10^4 and 10^6: no bit
// differs from the host's).  Bound by the fp64 units: 16,385 positions of 64
// pairs take 0.06 ms and 2^20 3.5 ms; one host thread takes 18 ms for the former.
__global__ void rope_table_kernel(float2 *tab, int64_t n, int half, const __grid_constant__ RopeFreqs freqs) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
        const int64_t pos = i / half;
        double s, c;
        sincos(static_cast<double>(pos) * freqs.f[i - pos * half], &s, &c);
        tab[i] = make_float2(static_cast<float>(c), static_cast<float>(s));
    }
}

// The rotary tables of the caches that are alive.  A table depends on theta and
// head_dim alone and a longer one begins with the shorter ones, so caches of one
// device share it.
class RopeTables {
  public:
    // A table of at least `rows` positions on the current device; null on error.
    const float2 *take(int device, float theta, int D, int rows) {
        std::lock_guard<std::mutex> lock(mu_);
        for (Table &t : tables_)
            if (t.device == device && t.theta == theta && t.D == D && t.rows >= rows) {
                ++t.users;
                return t.tab;
            }
        tables_.reserve(tables_.size() + 1);
        RopeFreqs freqs{};
        for (int i = 0; i < D / 2; ++i) freqs.f[i] = std::pow(static_cast<double>(theta), -2.0 * i / D);
        const int64_t n = static_cast<int64_t>(rows) * (D / 2);
        float2 *tab = nullptr;
        if (cudaMalloc(reinterpret_cast<void **>(&tab), n * sizeof(float2)) != cudaSuccess) return nullptr;
        rope_table_kernel<<<static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 4096)), 256>>>(tab, n, D / 2, freqs);
        if (cudaGetLastError() != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess) {
            cudaFree(tab);
            return nullptr;
        }
        tables_.push_back({device, theta, D, rows, 1, tab});
        return tab;
    }
    // Gives one back; the caller has synchronised its device.
    void give(const float2 *tab) {
        if (!tab) return;
        std::lock_guard<std::mutex> lock(mu_);
        for (size_t i = 0; i < tables_.size(); ++i)
            if (tables_[i].tab == tab && --tables_[i].users == 0) {
                cudaFree(tables_[i].tab);
                tables_.erase(tables_.begin() + i);
                return;
            }
    }

  private:
    struct Table {
        int device;
        float theta;
        int D, rows, users;
        float2 *tab;
    };
    std::mutex mu_;
    std::vector<Table> tables_;
};
RopeTables g_rope;

}  // namespace

namespace qa {

const float2 *rope_table_take(int device, float theta, int D, int rows) { return g_rope.take(device, theta, D, rows); }
void rope_table_give(const float2 *tab) { g_rope.give(tab); }

void PrefillWorkspace::init(const qa_config &cfg, int num_sms, bool factors) {
    cfg_ = cfg;
    has_factors_ = factors;
    num_sms_ = num_sms;
    slots_ = std::min(cfg.max_batch, kMaxSeqPerLaunch);
    G_ = cfg.n_q_heads / cfg.n_kv_heads;
}

void PrefillWorkspace::release() {
    cudaFree(ws_[0]);
    cudaFree(part_o_);
    if (free_) cudaEventDestroy(free_);
}

size_t PrefillWorkspace::kv_bytes() const { return static_cast<size_t>(slots_) * seq_stride() * 2; }

size_t PrefillWorkspace::factor_bytes() const {
    return has_factors_ ? static_cast<size_t>(slots_) * cfg_.n_kv_heads * factor_stride() * sizeof(float4) : 0;
}

size_t PrefillWorkspace::bytes() const {
    return 2 * kv_bytes() + factor_bytes() +
           (cfg_.capacity < kPartsCapacity ? 0 : part_rows() * (cfg_.head_dim * sizeof(float) + sizeof(float2)));
}

bool PrefillWorkspace::take() {
    if (ws_[0]) return true;
    OutsideCapture scope;
    if (!free_ && cudaEventCreateWithFlags(&free_, cudaEventDisableTiming) != cudaSuccess) {
        free_ = nullptr;
        return false;
    }
    const size_t one = align256(kv_bytes());
    void *p = nullptr;
    if (cudaMalloc(&p, 2 * one + factor_bytes()) != cudaSuccess) return false;
    ws_[0] = static_cast<__nv_bfloat16 *>(p);
    ws_[1] = ws_[0] + one / 2;
    if (has_factors_) factors_ = reinterpret_cast<float4 *>(ws_[0] + one);
    return true;
}

bool PrefillWorkspace::take_sums() {
    if (part_o_) return true;
    OutsideCapture scope;
    const size_t sums = part_rows() * cfg_.head_dim;  // (a multiple of 256 bytes)
    void *p = nullptr;
    if (cudaMalloc(&p, sums * sizeof(float) + part_rows() * sizeof(float2)) != cudaSuccess) return false;
    part_o_ = static_cast<float *>(p);
    part_ml_ = reinterpret_cast<float2 *>(part_o_ + sums);
    return true;
}

bool PrefillWorkspace::plan(int window, int n, const int32_t *start, const int32_t *ntok, const int *cu,
                            __nv_bfloat16 *qp, uint32_t *err, bool scaled, K2Job &job) {
    const int D = cfg_.head_dim, Hq = cfg_.n_q_heads, Hkv = cfg_.n_kv_heads;
    K2ScaledPartParams &k2 = job.k2;
    k2 = K2ScaledPartParams{};
    job.scaled = scaled;
    k2.factors = factors_;
    k2.factor_stride = factor_stride();
    std::vector<QueryRun> runs;
    for (int i = 0; i < n; ++i)
        if (ntok[i] > 0) runs.push_back({i, 0, ntok[i]});
    k2.hpi = std::min(G_, 2);
    std::vector<KeyPart> parts;
    job.parts = cfg_.capacity >= kPartsCapacity &&
               plan_parts(runs, start, window, D, G_, Hkv, num_sms_,
                              kMaxSeqPerLaunch, parts, k2.hpi);
    if (job.parts && !take_sums()) return false;
    k2.npairs = G_ / k2.hpi;
    if (!job.parts) {
        plan_runs(runs, start, window, D, G_, Hkv, num_sms_, kMaxSeqPerLaunch);
        k2.hpi = two_heads(runs, start, window, D, G_, Hkv, num_sms_) ? 2 : 0;
        for (size_t i = 0; i < runs.size(); ++i) parts.push_back({static_cast<int>(i), 0, 1 << 30});
    }
    job.join = K2JoinParams{};
    int nseq = 0, maxqb = 0, part_row = 0;
    const int rows = cu[n];
    job.items = 0;
    for (const KeyPart &part : parts) {
        const QueryRun &r = runs[part.run];
        const int P = start[r.seq] + r.first;
        if (!encode_kv_map(&k2.tm_k[nseq], ws_[0] + r.seq * seq_stride(), D, P + r.len, Hkv, cfg_.capacity, 64) ||
            !encode_kv_map(&k2.tm_v[nseq], ws_[1] + r.seq * seq_stride(), D, P + r.len, Hkv, cfg_.capacity, 128))
            return false;
        k2.len[nseq] = r.len;
        k2.start[nseq] = P;
        k2.slot[nseq] = r.seq;
        k2.cu[nseq] = cu[r.seq] + r.first;
        k2.part_lo[nseq] = part.lo;
        k2.part_hi[nseq] = part.hi;
        k2.part_row[nseq] = part_row;
        if (job.join.parts[part.run]++ == 0) {
            job.join.row0[part.run] = job.join.rows;
            job.join.len[part.run] = r.len;
            job.join.cu[part.run] = k2.cu[nseq];
            job.join.part_row[part.run] = part_row;
            job.join.rows += r.len;
        }
        part_row += r.len;
        maxqb = std::max(maxqb, (r.len + 127) / 128);
        job.items += (r.len + 127) / 128;
        ++nseq;
    }
    if (!encode_q_map(&k2.tm_q, qp, D, Hq, rows)) return false;
    k2.out = qp;
    k2.err = err;
    k2.nseq = nseq;
    k2.Hq = Hq;
    k2.Hkv = Hkv;
    k2.G = G_;
    k2.max_qblocks = maxqb;
    k2.window = window;
    k2.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
    job.items *= Hkv * k2.npairs;
    k2.part_o = part_o_;
    k2.part_ml = part_ml_;
    job.join.part_o = part_o_;
    job.join.part_ml = part_ml_;
    job.join.out = qp;
    job.join.Hq = Hq;
    job.join.nruns = static_cast<int>(runs.size());
    return true;
}

cudaError_t PrefillWorkspace::launch(K2Job &job, cudaStream_t s) const {
    const FaultPlan f = take_fault(QA_KERNEL_PREFILL_ATTN);
    job.k2.fault = f.fault;
    job.k2.wait_ns = f.wait_ns;
    const int D = cfg_.head_dim;
    if (!job.parts) {
        if (!job.scaled) return launch_k2(job.k2, D, job.items, s);
        K2ScaledParams p;
        static_cast<K2Params &>(p) = job.k2;
        static_cast<K2Factors &>(p) = job.k2;
        return launch_k2_scaled(p, D, job.items, s);
    }
    const cudaError_t e = job.scaled ? launch_k2_scaled_parts(job.k2, D, job.items, s) : launch_k2_parts(job.k2, D, job.items, s);
    return e == cudaSuccess ? launch_k2_join(job.join, D, s) : e;
}

}  // namespace qa
