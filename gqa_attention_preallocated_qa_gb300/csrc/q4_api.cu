// q4_api.cu -- the 4-bit cache of include/qa.h (qa_q4_*): its memory, argument
// validation, the split plan of its decode kernel and the order of its
// launches on the caller's stream.  As in qa_api.cu an unsupported shape or an
// invalid argument returns a status before anything is enqueued.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <new>
#include <vector>

#include "prefill_ws.h"
#include "q4_internal.h"
#include "q4_plan.h"
#include "qa.h"

#define QA_API extern "C" __attribute__((visibility("default")))

struct qa_q4_cache {
    qa_config cfg{};
    int device = 0;
    int num_sms = 0;
    int G = 1;
    int rows = 0;              // rows of one (sequence, kv head): the capacity, padded
    int64_t layer_rows = 0;    // rows of one layer
    void *mem = nullptr;       // one allocation: codes, scale bytes, error word, ws_lens
    uint8_t *codes[2] = {}, *scales[2] = {};  // K and V
    uint32_t *err = nullptr;
    int32_t *ws_lens = nullptr;     // written by the transform kernel, not read
    const float2 *rope = nullptr;   // shared (rope_table_take)
    qa::PrefillWorkspace ws;        // what prefill attention needs
    std::vector<int> window;        // per layer: attention window in keys (0: full)
    // Per (layer, sequence): the position after the last one written, -1 when
    // only the device knows it.  A decode step that continues there can tell
    // which rows a launch still running may write.
    std::vector<int32_t> next_pos;
    uint64_t cache_bytes = 0, scratch_bytes = 0;
    std::atomic<uint64_t> launches[QA_Q4_NUM_KERNELS];
};

namespace {

using qa::align256;
using qa::aligned16;
using qa::DeviceScope;
using qa::no_throw;

void free_all(qa_q4_cache *c) {
    qa::rope_table_give(c->rope);
    cudaFree(c->mem);
    c->ws.release();
}

qa_status check_layer(const qa_q4_cache *c, int layer, int batch) {
    if (!c) return QA_ERR_INVALID_ARG;
    if (layer < 0 || layer >= c->cfg.num_layers) return QA_ERR_INVALID_ARG;
    if (batch < 1 || batch > c->cfg.max_batch) return QA_ERR_INVALID_ARG;
    return QA_OK;
}

// Ranges start[b] .. start[b] + ntok[b] - 1 of the call; T: their rows.
qa_status check_ranges(const qa_q4_cache *c, int batch, const int32_t *start, const int32_t *ntok,
                       int64_t *T_out) {
    if (!start || !ntok) return QA_ERR_INVALID_ARG;
    int64_t T = 0;
    for (int b = 0; b < batch; ++b) {
        if (start[b] < 0 || ntok[b] < 0) return QA_ERR_INVALID_ARG;
        if (static_cast<int64_t>(start[b]) + ntok[b] > c->cfg.capacity) return QA_ERR_CAPACITY;
        T += ntok[b];
    }
    if (T > (int64_t(1) << 26)) return QA_ERR_INVALID_ARG;
    *T_out = T;
    return QA_OK;
}

int32_t *next_of(qa_q4_cache *c, int layer) {
    return c->next_pos.data() + static_cast<size_t>(layer) * c->cfg.max_batch;
}

// Row-kernel parameters common to every launch on `layer`.
qa::Q4RowsParams make_rows(const qa_q4_cache *c, int layer) {
    const qa_config &g = c->cfg;
    qa::Q4RowsParams p{};
    for (int i = 0; i < 2; ++i) {
        p.codes[i] = c->codes[i] + layer * c->layer_rows * (g.head_dim / 2);
        p.scales[i] = c->scales[i] + layer * c->layer_rows * (g.head_dim / qa::kQ4Group);
    }
    p.row_head = c->rows;
    p.row_seq = static_cast<int64_t>(c->rows) * g.n_kv_heads;
    p.Hkv = g.n_kv_heads;
    p.kv_first = 0;
    p.kv_count = 2;
    return p;
}

// Packed [T][Hkv][D] rows on either side.
void packed_rows(const qa_config &g, int64_t &tok, int64_t &head) {
    tok = static_cast<int64_t>(g.n_kv_heads) * g.head_dim;
    head = g.head_dim;
}

// Tokens per lane group of a quantising launch of T rows.  Eight make the fewest
// warps and the longest runs (57,000 rows of 8 heads, D 128: 86 us against 91
// with four), but a grid that the device holds at once loads, computes and
// stores in step; there four overlap better (5120 rows: 10.7 us against 12.7).
// The border is about four times what the device holds.
int quantise_unroll(const qa_q4_cache *c, int64_t T) {
    const int64_t warps = T / qa::q4_block_tokens(c->cfg.head_dim, 8) * c->cfg.n_kv_heads * 2;
    return warps > static_cast<int64_t>(c->num_sms) * 128 ? 8 : 4;
}

// The rows of sequences s0 .. s0 + n - 1 of a call on packed tensors, row0 the
// first one's first packed row; false when there is none.
bool fill_ranges(qa::Q4RowsParams &p, const qa_config &g, int s0, int n, const int32_t *start,
                 const int32_t *ntok, int64_t row0, int unroll) {
    const int per = qa::q4_block_tokens(g.head_dim, unroll);
    p.unroll = unroll;
    p.nseq = n;
    p.seq0 = s0;
    p.nblocks = 0;
    for (int i = 0; i < n; ++i) {
        p.start[i] = start[s0 + i];
        p.ntok[i] = ntok[s0 + i];
        p.block0[i] = p.nblocks;
        p.nblocks += (ntok[s0 + i] + per - 1) / per;
        p.src_off[i] = p.dst_off[i] = row0 * g.n_kv_heads * g.head_dim;
        row0 += ntok[s0 + i];
    }
    p.block0[n] = p.nblocks;
    return p.nblocks > 0;
}

struct DecodeCall {
    const void *q, *k, *v, *wq, *wk;
    void *out, *k_held, *v_held;
    const int32_t *start;     // host positions (null: device positions)
    const int32_t *pos_dev;
    const int32_t *ntok;      // null: one token each
};

// Tokens first .. first + 7 of the call's sequences (only of those whose tokens
// come this way), one decode launch per 64 sequences that have any.
qa_status run_decode(qa_q4_cache *c, int layer, int batch, const DecodeCall &a, int first, cudaStream_t s) {
    const qa_config &g = c->cfg;
    const int D = g.head_dim;
    auto tokens = [&](int b) {
        if (!a.ntok) return 1;
        return qa::few_tokens(a.start[b], a.ntok[b], c->window[layer]) ? std::min(a.ntok[b] - first, qa::kQ4MaxTokens) : 0;
    };
    int tmax = 1;
    for (int b = 0; b < batch && a.ntok; ++b) tmax = std::max(tmax, tokens(b));
    const bool multi = tmax > 1;
    int HPC = c->G;
    while (multi && HPC > 1 && qa::kQ4MaxTokens / HPC < tmax) HPC /= 2;
    qa::Q4DecodeParams p{};
    const int64_t row = layer * c->layer_rows;
    p.kc = c->codes[0] + row * (D / 2);
    p.vc = c->codes[1] + row * (D / 2);
    p.ks = c->scales[0] + row * (D / qa::kQ4Group);
    p.vs = c->scales[1] + row * (D / qa::kQ4Group);
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.k = static_cast<const __nv_bfloat16 *>(a.k);
    p.v = static_cast<const __nv_bfloat16 *>(a.v);
    p.wq = static_cast<const __nv_bfloat16 *>(a.wq);
    p.wk = static_cast<const __nv_bfloat16 *>(a.wk);
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.k_held = static_cast<__nv_bfloat16 *>(a.k_held);
    p.v_held = static_cast<__nv_bfloat16 *>(a.v_held);
    p.rope = c->rope;
    p.pos_dev = a.pos_dev;
    p.err = c->err;
    p.row_head = c->rows;
    p.row_seq = static_cast<int64_t>(c->rows) * g.n_kv_heads;
    p.Hq = g.n_q_heads;
    p.Hkv = g.n_kv_heads;
    p.G = c->G;
    p.HG = c->G / HPC;
    p.groups = p.Hkv * p.HG;
    p.cap = g.capacity;
    p.eps = g.rms_eps;
    p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
    p.window = c->window[layer];

    // Which cache rows may be read before the previous kernel has finished: all
    // of them when no launch that may still run writes this layer; when this
    // call continues every sequence where the last one left it, those below the
    // rows such launches append; else none, and the launch signals the next one
    // only after its own wait.
    int32_t *next = next_of(c, layer);
    const int64_t resident = std::max<int64_t>(qa::k3_max_resident_ctas(), 2 * c->num_sms);
    qa::StreamRef at = qa::stream_ref(s, c->device);
    const bool settled = qa::launch_order().layer_settled(at, c, layer, resident);
    bool follows = !a.pos_dev;
    for (int b = 0; b < batch && follows; ++b)
        if (tokens(b) > 0 && next[b] != a.start[b] + first) follows = false;

    const qa::LaunchOrder::Call call(qa::launch_order());
    int b = 0, row0 = 0;
    while (b < batch) {
        int nz = 0, tm = 0;
        const int b0 = b;
        for (; b < batch && nz < qa::kQ4MaxSeqPerLaunch; ++b) {
            const int n = tokens(b);
            if (n > 0) {
                p.seq[nz] = {a.pos_dev ? 0 : a.start[b] + first, b, n, row0 + first, 0, 1, 0, 0};
                tm = std::max(tm, n);
                ++nz;
            }
            row0 += a.ntok ? a.ntok[b] : 1;
        }
        if (nz == 0) break;
        // The longest sequences first: thread blocks start in this order, and the
        // short ones fill in behind them.
        std::stable_sort(p.seq, p.seq + nz, [](const qa::Q4Seq &x, const qa::Q4Seq &y) { return x.pos > y.pos; });
        int keys[qa::kQ4MaxSeqPerLaunch];
        for (int i = 0; i < nz; ++i) {
            keys[i] = a.pos_dev ? g.capacity - 1 : p.seq[i].pos;
            if (p.window > 0) keys[i] = std::min(keys[i], p.window);
        }
        qa::DecodePlan plan;
        qa::plan_decode(D, qa::q4_cluster_capacities(D, HPC, multi), p.groups, nz, keys, plan);
        const int rows = multi ? qa::kQ4MaxTokens : HPC;
        p.ctas = 0;
        int units = 0;
        for (int i = 0; i < nz; ++i) {
            const int S = plan.splits[i];
            p.seq[i].cta0 = p.ctas;
            p.seq[i].S = S;
            p.seq[i].E = ((rows * D + S - 1) / S + 31) & ~31;
            p.seq[i].inv_S = S == 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + S - 1) / S);
            for (int k = 0; k < S; ++k) p.seq_of[units++] = static_cast<uint8_t>(i);
            p.ctas += p.groups * S;
        }
        p.B = nz;
        p.cluster = plan.cluster;
        p.mixed = plan.splits[nz - 1] != plan.cluster ? 1 : 0;
        p.early = !a.pos_dev && (settled || follows) ? 1 : 0;
        const int guard = qa::launch_order().admit(at, c, layer, p.ctas, tm,
                                                   p.early != 0, resident);
        p.guard = settled ? 0 : guard;
        const qa::FaultPlan f = qa::take_fault(QA_KERNEL_DECODE_ATTN);
        p.fault = f.fault;
        p.wait_ns = f.wait_ns;
        if (qa::launch_q4_decode(p, D, HPC, multi, s) != cudaSuccess) {
            cudaGetLastError();
            return QA_ERR_CUDA;
        }
        qa::note_launch(at, s);
        c->launches[QA_Q4_KERNEL_DECODE]++;
        for (int i = b0; i < b; ++i)
            if (tokens(i) > 0) next[i] = a.pos_dev ? -1 : a.start[i] + first + tokens(i);
    }
    return QA_OK;
}

// One launch group of a prefill: up to ws_slots sequences.
struct PrefillGroup {
    qa::Q4PrefillRowsParams rows;
    qa::Q4RowsParams quant, held;
    qa::K2Job k2;
};

// Builds the launches for sequences s0 .. s0 + n - 1; false when a tensor map
// cannot be made or the sums of parts find no memory.
bool plan_prefill(qa_q4_cache *c, int layer, int s0, int n, const int32_t *start, const int32_t *ntok,
                  int64_t row0, const void *q, const void *k, const void *v, const void *wq,
                  const void *wk, void *out, PrefillGroup &pg) {
    const qa_config &g = c->cfg;
    const int D = g.head_dim, Hq = g.n_q_heads, Hkv = g.n_kv_heads;
    const int64_t ws_head = c->ws.head_stride(), ws_seq = c->ws.seq_stride();
    pg.rows = qa::Q4PrefillRowsParams{};
    qa::K1Params &k1 = pg.rows.k1;
    k1.q = static_cast<const __nv_bfloat16 *>(q) + row0 * Hq * D;
    k1.k = static_cast<const __nv_bfloat16 *>(k) + row0 * Hkv * D;
    k1.v = static_cast<const __nv_bfloat16 *>(v) + row0 * Hkv * D;
    k1.wq = static_cast<const __nv_bfloat16 *>(wq);
    k1.wk = static_cast<const __nv_bfloat16 *>(wk);
    k1.qp = static_cast<__nv_bfloat16 *>(out) + row0 * Hq * D;
    k1.kc = c->ws.rows(0);
    k1.vc = c->ws.rows(1);
    k1.lens = c->ws_lens;
    k1.rope = c->rope;
    k1.err = c->err;
    k1.head_stride = ws_head;
    k1.seq_stride = ws_seq;
    k1.Hq = Hq;
    k1.Hkv = Hkv;
    k1.cap = g.capacity;
    k1.eps = g.rms_eps;
    k1.nseq = n;
    // The new rows, for the two-kernel form: quantised in place, so that the
    // workspace holds what the cache holds.
    pg.quant = make_rows(c, layer);
    for (int i = 0; i < 2; ++i) {
        pg.rows.codes[i] = pg.quant.codes[i];
        pg.rows.scales[i] = pg.quant.scales[i];
    }
    pg.rows.row_seq = pg.quant.row_seq;
    pg.rows.row_head = pg.quant.row_head;
    pg.rows.seq0 = s0;
    fill_ranges(pg.quant, g, s0, n, start, ntok, 0, 8);
    // The rows before them that a new token sees, from the first row of the
    // 128-key tile that holds the first one.  Those of the tile that none sees may
    // hold anything, and the attention kernel multiplies them by weights of zero:
    // they are zeros in the workspace.
    pg.held = make_rows(c, layer);
    int32_t from[qa::kMaxSeqPerLaunch], count[qa::kMaxSeqPerLaunch];
    for (int i = 0; i < n; ++i) {
        const int P = start[s0 + i], W = c->window[layer];
        from[i] = W > 0 ? std::max(0, P + 1 - W) / 128 * 128 : 0;
        count[i] = ntok[s0 + i] > 0 ? P - from[i] : 0;
    }
    fill_ranges(pg.held, g, 0, n, from, count, 0, 4);
    for (int i = 0; i < n; ++i) {
        const int W = c->window[layer];
        pg.held.hidden[i] = W > 0 ? std::max(0, start[s0 + i] + 1 - W) : 0;
    }
    pg.held.seq0 = s0;
    for (qa::Q4RowsParams *r : {&pg.quant, &pg.held}) {
        r->src_tok = r->dst_tok = D;
        r->src_head = r->dst_head = ws_head;
        for (int i = 0; i < 2; ++i) {
            r->src[i] = c->ws.rows(i);
            r->dst[i] = c->ws.rows(i);
        }
        for (int i = 0; i < n; ++i)
            r->src_off[i] = r->dst_off[i] = i * ws_seq + static_cast<int64_t>(r->start[i]) * D;
    }
    k1.cu[0] = 0;
    for (int i = 0; i < n; ++i) {
        k1.cu[i + 1] = k1.cu[i] + ntok[s0 + i];
        k1.start[i] = start[s0 + i];
    }
    k1.T = k1.cu[n];
    return k1.T == 0 || c->ws.plan(c->window[layer], n, start + s0, ntok + s0, k1.cu, k1.qp, c->err, false, pg.k2);
}

}  // namespace

QA_API qa_status qa_q4_cache_alloc(const qa_config *cfg, qa_q4_cache **out) {
    if (!cfg || !out) return QA_ERR_INVALID_ARG;
    *out = nullptr;
    const qa_config g = *cfg;
    if (g.num_layers <= 0 || g.max_batch <= 0 || g.capacity <= 0 || g.n_q_heads <= 0 ||
        g.n_kv_heads <= 0 || g.head_dim <= 0 || !(g.rope_theta > 0.f) || !(g.rms_eps >= 0.f))
        return QA_ERR_INVALID_ARG;
    if (!qa::supported_geometry(g.n_q_heads, g.n_kv_heads, g.head_dim)) return QA_ERR_UNSUPPORTED_SHAPE;
    if (g.capacity > (1 << 24) || g.max_batch > 65535 || g.n_q_heads > 65535) return QA_ERR_UNSUPPORTED_SHAPE;
    qa_q4_cache *c = new (std::nothrow) qa_q4_cache();
    if (!c) return QA_ERR_CUDA;
    c->cfg = g;
    for (auto &x : c->launches) x = 0;
    c->G = g.n_q_heads / g.n_kv_heads;
    c->rows = (g.capacity + qa::kQ4RowPad - 1) / qa::kQ4RowPad * qa::kQ4RowPad;
    c->layer_rows = static_cast<int64_t>(g.max_batch) * g.n_kv_heads * c->rows;
    const size_t rows = static_cast<size_t>(c->layer_rows) * g.num_layers;
    const size_t codes = rows * (g.head_dim / 2), scales = rows * (g.head_dim / qa::kQ4Group);
    const size_t total = 2 * (align256(codes) + align256(scales)) + 256;
    bool ok = cudaGetDevice(&c->device) == cudaSuccess &&
              cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, c->device) == cudaSuccess &&
              cudaMalloc(&c->mem, total) == cudaSuccess && cudaMemsetAsync(c->mem, 0, total, nullptr) == cudaSuccess;
    ok = ok && no_throw([&] {
        uint8_t *at = static_cast<uint8_t *>(c->mem);
        for (int i = 0; i < 2; ++i, at += align256(codes)) c->codes[i] = at;
        for (int i = 0; i < 2; ++i, at += align256(scales)) c->scales[i] = at;
        c->err = reinterpret_cast<uint32_t *>(at);
        c->ws_lens = reinterpret_cast<int32_t *>(at + 128);
        static_assert(qa::kMaxSeqPerLaunch * sizeof(int32_t) <= 128, "behind the error word");
        c->window.assign(static_cast<size_t>(g.num_layers), 0);
        c->next_pos.assign(static_cast<size_t>(g.num_layers) * g.max_batch, -1);
        c->rope = qa::rope_table_take(c->device, g.rope_theta, g.head_dim, g.capacity);
        return c->rope && cudaStreamSynchronize(nullptr) == cudaSuccess ? QA_OK : QA_ERR_CUDA;
    }) == QA_OK;
    c->cache_bytes = 2 * (codes + scales);
    c->ws.init(g, c->num_sms);
    c->scratch_bytes = 256 + c->ws.bytes() + static_cast<size_t>(g.capacity) * (g.head_dim / 2) * sizeof(float2);
    if (!ok) {
        free_all(c);
        delete c;
        cudaGetLastError();
        return QA_ERR_CUDA;
    }
    *out = c;
    return QA_OK;
}

QA_API qa_status qa_q4_cache_free(qa_q4_cache *c) {
    if (!c) return QA_OK;
    DeviceScope dev(c->device);
    qa::synchronise_device();
    free_all(c);
    delete c;
    return QA_OK;
}

QA_API qa_status qa_q4_cache_set_window(qa_q4_cache *c, int layer, int window) {
    if (!c || layer < 0 || layer >= c->cfg.num_layers || window < 0) return QA_ERR_INVALID_ARG;
    c->window[layer] = window;
    return QA_OK;
}

QA_API qa_status qa_q4_append(qa_q4_cache *c, int layer, int batch, const int32_t *start,
                              const int32_t *ntok, const void *k, const void *v, void *k_held,
                              void *v_held, void *stream) {
    qa_status st = check_layer(c, layer, batch);
    if (st != QA_OK) return st;
    int64_t T = 0;
    st = check_ranges(c, batch, start, ntok, &T);
    if (st != QA_OK) return st;
    if ((k_held == nullptr) != (v_held == nullptr)) return QA_ERR_INVALID_ARG;
    if (T == 0) return QA_OK;
    if (!k || !v) return QA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_held) || !aligned16(v_held)) return QA_ERR_ALIGNMENT;
    DeviceScope dev(c->device);
    if (!dev.ok()) return QA_ERR_CUDA;
    const qa_config &g = c->cfg;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    qa::Q4RowsParams p = make_rows(c, layer);
    p.src[0] = static_cast<const __nv_bfloat16 *>(k);
    p.src[1] = static_cast<const __nv_bfloat16 *>(v);
    p.dst[0] = static_cast<__nv_bfloat16 *>(k_held);
    p.dst[1] = static_cast<__nv_bfloat16 *>(v_held);
    packed_rows(g, p.src_tok, p.src_head);
    packed_rows(g, p.dst_tok, p.dst_head);
    const int unroll = quantise_unroll(c, T);
    int32_t *next = next_of(c, layer);
    int64_t row0 = 0;
    for (int s0 = 0; s0 < batch; s0 += qa::kQ4MaxSeqPerLaunch) {
        const int n = std::min(qa::kQ4MaxSeqPerLaunch, batch - s0);
        if (fill_ranges(p, g, s0, n, start, ntok, row0, unroll)) {
            if (qa::launch_q4_quantise(p, g.head_dim, s) != cudaSuccess) return QA_ERR_CUDA;
            qa::launch_order().barrier(qa::stream_ref(s, c->device));
            c->launches[QA_Q4_KERNEL_QUANTISE]++;
        }
        for (int i = 0; i < n; ++i) {
            row0 += ntok[s0 + i];
            if (ntok[s0 + i] > 0) next[s0 + i] = start[s0 + i] + ntok[s0 + i];
        }
    }
    return QA_OK;
}

QA_API qa_status qa_q4_read(qa_q4_cache *c, int layer, int batch, const int32_t *start,
                            const int32_t *ntok, void *k_out, void *v_out, void *stream) {
    qa_status st = check_layer(c, layer, batch);
    if (st != QA_OK) return st;
    int64_t T = 0;
    st = check_ranges(c, batch, start, ntok, &T);
    if (st != QA_OK) return st;
    if (T == 0) return QA_OK;
    if (!k_out && !v_out) return QA_ERR_INVALID_ARG;
    if (!aligned16(k_out) || !aligned16(v_out)) return QA_ERR_ALIGNMENT;
    DeviceScope dev(c->device);
    if (!dev.ok()) return QA_ERR_CUDA;
    const qa_config &g = c->cfg;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    qa::Q4RowsParams p = make_rows(c, layer);
    p.dst[0] = static_cast<__nv_bfloat16 *>(k_out);
    p.dst[1] = static_cast<__nv_bfloat16 *>(v_out);
    p.kv_first = k_out ? 0 : 1;
    p.kv_count = k_out && v_out ? 2 : 1;
    packed_rows(g, p.dst_tok, p.dst_head);
    int64_t row0 = 0;
    for (int s0 = 0; s0 < batch; s0 += qa::kQ4MaxSeqPerLaunch) {
        const int n = std::min(qa::kQ4MaxSeqPerLaunch, batch - s0);
        if (fill_ranges(p, g, s0, n, start, ntok, row0, 4)) {
            if (qa::launch_q4_dequantise(p, g.head_dim, s) != cudaSuccess) return QA_ERR_CUDA;
            qa::launch_order().barrier(qa::stream_ref(s, c->device));
            c->launches[QA_Q4_KERNEL_DEQUANTISE]++;
        }
        for (int i = 0; i < n; ++i) row0 += ntok[s0 + i];
    }
    return QA_OK;
}

QA_API qa_status qa_q4_prefill(qa_q4_cache *c, int layer, int batch, const int32_t *start,
                               const int32_t *ntok, const void *q, const void *k, const void *v,
                               const void *q_norm_w, const void *k_norm_w, void *out, void *stream) {
    qa_status st = check_layer(c, layer, batch);
    if (st != QA_OK) return st;
    int64_t T = 0;
    st = check_ranges(c, batch, start, ntok, &T);
    if (st != QA_OK) return st;
    if (T == 0) return QA_OK;
    if (!q || !k || !v || !q_norm_w || !k_norm_w || !out) return QA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_norm_w) ||
        !aligned16(k_norm_w) || !aligned16(out))
        return QA_ERR_ALIGNMENT;
    DeviceScope dev(c->device);
    if (!dev.ok()) return QA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto few_tokens = [&](int b) { return qa::few_tokens(start[b], ntok[b], c->window[layer]); };
    int few = 0;  // the most tokens of a sequence that takes the decode kernel
    bool long_form = false;
    for (int b = 0; b < batch; ++b) {
        if (few_tokens(b))
            few = std::max(few, ntok[b]);
        else
            long_form = true;
    }
    std::vector<PrefillGroup> groups;
    if (long_form) {
        // It goes through the cache's one bf16 workspace: a graph could be replayed
        // beside another call that uses it, so it is not captured, and calls on
        // several streams take turns.
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(s, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone) {
            cudaGetLastError();
            return QA_ERR_STATE;
        }
        if (!c->ws.take()) {
            cudaGetLastError();
            return QA_ERR_CUDA;
        }
        // A group's rows are packed one after the other, so sequences that take
        // the decode kernel stand between groups.
        st = no_throw([&] {
            int64_t row0 = 0;
            for (int s0 = 0; s0 < batch;) {
                int n = 0;
                while (s0 + n < batch && n < c->ws.slots() &&
                       (!few_tokens(s0 + n) || (n > 0 && ntok[s0 + n] == 0)))
                    ++n;
                if (n == 0) {
                    row0 += ntok[s0++];
                    continue;
                }
                groups.emplace_back();
                PrefillGroup &pg = groups.back();
                if (!plan_prefill(c, layer, s0, n, start, ntok, row0, q, k, v, q_norm_w, k_norm_w, out, pg)) {
                    cudaGetLastError();
                    return QA_ERR_CUDA;
                }
                row0 += pg.rows.k1.T;
                s0 += n;
            }
            return QA_OK;
        });
        if (st != QA_OK) return st;
    }
    const DecodeCall a{q, k, v, q_norm_w, k_norm_w, out, nullptr, nullptr, start, nullptr, ntok};
    for (int first = 0; first < few && st == QA_OK; first += qa::kQ4MaxTokens)
        st = no_throw([&] { return run_decode(c, layer, batch, a, first, s); });
    if (st != QA_OK || !long_form) return st;
    if (cudaStreamWaitEvent(s, c->ws.free_event(), 0) != cudaSuccess) return QA_ERR_CUDA;
    int32_t *next = next_of(c, layer);
    for (int b = 0; b < batch; ++b)
        if (!few_tokens(b)) next[b] = start[b] + ntok[b];
    const bool fused = qa::q4_prefill_rows_fits(c->cfg.n_q_heads, c->cfg.n_kv_heads, c->cfg.head_dim);
    const qa::StreamRef at(s, c->device);  // (not being captured)
    auto launch = [&](PrefillGroup &pg) {
        auto older_rows = [&](bool beside) {
            if (pg.held.nblocks == 0) return true;
            pg.held.beside = beside ? 1 : 0;
            if (qa::launch_q4_dequantise(pg.held, c->cfg.head_dim, s) != cudaSuccess) return false;
            qa::launch_order().barrier(at);
            c->launches[QA_Q4_KERNEL_DEQUANTISE]++;
            return true;
        };
        if (fused) {
            pg.rows.k1.signal_early = 1;
            if (qa::launch_q4_prefill_rows(pg.rows, c->cfg.head_dim, s) != cudaSuccess) return QA_ERR_CUDA;
            qa::launch_order().barrier(at);
            c->launches[QA_Q4_KERNEL_QUANTISE]++;
            if (!older_rows(true)) {
                cudaStreamSynchronize(s);  // as below
                return QA_ERR_CUDA;
            }
        } else {
            if (!older_rows(false)) return QA_ERR_CUDA;
            if (qa::launch_k1(pg.rows.k1, c->cfg.head_dim, s) != cudaSuccess) return QA_ERR_CUDA;
            qa::launch_order().barrier(at);
            c->launches[QA_Q4_KERNEL_NORM_ROPE]++;
            if (qa::launch_q4_quantise(pg.quant, c->cfg.head_dim, s) != cudaSuccess) return QA_ERR_CUDA;
            c->launches[QA_Q4_KERNEL_QUANTISE]++;
        }
        if (c->ws.launch(pg.k2, s) != cudaSuccess) {
            // A kernel that signalled early is no longer followed by one that
            // waits for it: let it finish before anything else is enqueued.
            cudaStreamSynchronize(s);
            return QA_ERR_CUDA;
        }
        qa::launch_order().barrier(at);
        c->launches[QA_Q4_KERNEL_PREFILL_ATTN]++;
        return QA_OK;
    };
    for (size_t i = 0; i < groups.size() && st == QA_OK; ++i) st = launch(groups[i]);
    // After a failure too: what was enqueued uses the workspace.
    if (cudaEventRecord(c->ws.free_event(), s) != cudaSuccess) return QA_ERR_CUDA;
    return st;
}

namespace {
qa_status decode_step(qa_q4_cache *c, int layer, int batch, const DecodeCall &a, void *stream) {
    if (!a.q || !a.k || !a.v || !a.wq || !a.wk || !a.out) return QA_ERR_INVALID_ARG;
    if ((a.k_held == nullptr) != (a.v_held == nullptr)) return QA_ERR_INVALID_ARG;
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.wq) ||
        !aligned16(a.wk) || !aligned16(a.out) || !aligned16(a.k_held) || !aligned16(a.v_held))
        return QA_ERR_ALIGNMENT;
    DeviceScope dev(c->device);
    if (!dev.ok()) return QA_ERR_CUDA;
    return no_throw([&] { return run_decode(c, layer, batch, a, 0, static_cast<cudaStream_t>(stream)); });
}
}  // namespace

QA_API qa_status qa_q4_decode_step(qa_q4_cache *c, int layer, int batch, const int32_t *positions,
                                   const void *q, const void *k, const void *v, const void *q_norm_w,
                                   const void *k_norm_w, void *out, void *k_held, void *v_held,
                                   void *stream) {
    qa_status st = check_layer(c, layer, batch);
    if (st != QA_OK) return st;
    if (!positions) return QA_ERR_INVALID_ARG;
    for (int b = 0; b < batch; ++b)
        if (positions[b] < 0) return QA_ERR_INVALID_ARG;
    for (int b = 0; b < batch; ++b)
        if (positions[b] >= c->cfg.capacity) return QA_ERR_CAPACITY;
    return decode_step(c, layer, batch,
                       {q, k, v, q_norm_w, k_norm_w, out, k_held, v_held, positions, nullptr, nullptr}, stream);
}

QA_API qa_status qa_q4_decode_step_device_positions(qa_q4_cache *c, int layer, int batch,
                                                    const int32_t *positions, const void *q,
                                                    const void *k, const void *v, const void *q_norm_w,
                                                    const void *k_norm_w, void *out, void *k_held,
                                                    void *v_held, void *stream) {
    qa_status st = check_layer(c, layer, batch);
    if (st != QA_OK) return st;
    if (!positions) return QA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(positions) & 3u) return QA_ERR_ALIGNMENT;
    return decode_step(c, layer, batch,
                       {q, k, v, q_norm_w, k_norm_w, out, k_held, v_held, nullptr, positions, nullptr}, stream);
}

QA_API qa_status qa_q4_cache_view(qa_q4_cache *c, int layer, void **k_codes, void **k_scales,
                                  void **v_codes, void **v_scales, int64_t strides[3]) {
    if (!c || layer < 0 || layer >= c->cfg.num_layers) return QA_ERR_INVALID_ARG;
    const int64_t row = layer * c->layer_rows;
    const int D = c->cfg.head_dim;
    void **codes[2] = {k_codes, v_codes}, **scales[2] = {k_scales, v_scales};
    for (int i = 0; i < 2; ++i) {
        if (codes[i]) *codes[i] = c->codes[i] + row * (D / 2);
        if (scales[i]) *scales[i] = c->scales[i] + row * (D / qa::kQ4Group);
    }
    if (strides) {
        strides[2] = 1;
        strides[1] = c->rows;
        strides[0] = static_cast<int64_t>(c->rows) * c->cfg.n_kv_heads;
    }
    return QA_OK;
}

QA_API qa_status qa_q4_get_device_error(qa_q4_cache *c, uint32_t *detail) {
    if (!c) return QA_ERR_INVALID_ARG;
    DeviceScope dev(c->device);
    uint32_t word = 0;
    if (!dev.ok() || qa::synchronise_device() != cudaSuccess ||
        cudaMemcpy(&word, c->err, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess ||
        cudaMemset(c->err, 0, sizeof(word)) != cudaSuccess)
        return QA_ERR_CUDA;
    if (detail) *detail = word;
    switch (word & 0xffu) {
        case 0: return QA_OK;
        case qa::kErrTimeout: return QA_ERR_DEVICE_TIMEOUT;
        default: return QA_ERR_DEVICE_BOUNDS;
    }
}

QA_API qa_status qa_q4_stats(qa_q4_cache *c, uint64_t launches[QA_Q4_NUM_KERNELS]) {
    if (!c || !launches) return QA_ERR_INVALID_ARG;
    for (int i = 0; i < QA_Q4_NUM_KERNELS; ++i) launches[i] = c->launches[i].load();
    return QA_OK;
}

QA_API qa_status qa_q4_memory_info(qa_q4_cache *c, uint64_t *cache_bytes, uint64_t *scratch_bytes) {
    if (!c) return QA_ERR_INVALID_ARG;
    if (cache_bytes) *cache_bytes = c->cache_bytes;
    if (scratch_bytes) *scratch_bytes = c->scratch_bytes;
    return QA_OK;
}
