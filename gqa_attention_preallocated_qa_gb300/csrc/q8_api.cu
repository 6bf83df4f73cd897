// q8_api.cu -- the 8-bit cache of include/qa.h (qa_q8_*): its memory, argument
// validation and the order of its launches on the caller's stream.  As in
// qa_api.cu an unsupported shape or an invalid argument returns a status before
// anything is enqueued.
//
// Every kernel of this cache waits for the one before it on the stream before it writes
// anything.  A step signals the next launch at once, reads and computes before that wait
// where the launch record (launch_order.h) says that nothing that may still run writes its
// layer; otherwise it waits first.  The others wait, then signal.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <new>
#include <vector>

#include "prefill_ws.h"
#include "q8_internal.h"
#include "q8_plan.h"
#include "qa.h"

#define QA_API extern "C" __attribute__((visibility("default")))

struct qa_q8_cache {
    qa_config cfg{};
    int device = 0;
    int num_sms = 0;
    int sm_smem = 0, reserved_smem = 0;  // shared memory of an SM, and what it keeps of it for each CTA
    int nblk = 0;              // blocks of one (sequence, kv head)
    void *mem = nullptr;       // one allocation: all of the following
    uint8_t *codes = nullptr;
    float2 *scales = nullptr;
    int8_t *bounds = nullptr;
    __nv_bfloat16 *tail = nullptr;
    qa::Q8Tail *state = nullptr;
    uint32_t *err = nullptr;
    uint32_t *tickets = nullptr;    // of a prefill's rows, [workspace slot][kv head]
    const float2 *rope = nullptr;   // shared (rope_table_take)
    qa::PrefillWorkspace ws;        // what prefill attention needs
    uint64_t cache_bytes = 0, scratch_bytes = 0;
    std::atomic<uint64_t> launches[QA_Q8_NUM_KERNELS];
};

namespace {

using qa::align256;
using qa::aligned16;
using qa::DeviceScope;
using qa::no_throw;

void free_all(qa_q8_cache *c) {
    qa::rope_table_give(c->rope);
    cudaFree(c->mem);
    c->ws.release();
}

qa_status check_layer(const qa_q8_cache *c, int layer, int batch) {
    if (!c) return QA_ERR_INVALID_ARG;
    if (layer < 0 || layer >= c->cfg.num_layers) return QA_ERR_INVALID_ARG;
    if (batch < 1 || batch > c->cfg.max_batch) return QA_ERR_INVALID_ARG;
    return QA_OK;
}

// Ranges start[b] .. start[b] + ntok[b] - 1 of the call; T: their rows.
qa_status check_ranges(const qa_q8_cache *c, int batch, const int32_t *start, const int32_t *ntok, int64_t *T_out) {
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

struct Span {
    const void *p;
    int64_t bytes;
};
bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x && y && x < y + b.bytes && y < x + a.bytes;
}
// What a call writes shares no byte with what it reads, nor with another of its outputs.
template <size_t N, size_t M>
bool apart(const Span (&in)[N], const Span (&out)[M]) {
    for (size_t i = 0; i < M; ++i) {
        for (const Span &x : in)
            if (overlap(x, out[i])) return false;
        for (size_t j = 0; j < i; ++j)
            if (overlap(out[j], out[i])) return false;
    }
    return true;
}

qa::Q8Layer layer_of(const qa_q8_cache *c, int layer) {
    const qa_config &g = c->cfg;
    const int64_t heads = static_cast<int64_t>(layer) * g.max_batch * g.n_kv_heads, blocks = heads * c->nblk;
    qa::Q8Layer l{};
    l.codes = c->codes + blocks * 2 * qa::kQ8Block * g.head_dim;
    l.scales = c->scales + blocks;
    l.bounds = c->bounds + blocks * 2 * g.head_dim;
    l.tail = c->tail + heads * 4 * qa::kQ8Block * g.head_dim;
    l.state = c->state + heads;
    l.nblk = c->nblk;
    l.Hkv = g.n_kv_heads;
    return l;
}

// Row parameters of sequences s0 .. s0 + n - 1 with packed tensors, row0 the first
// one's first packed row; false when there is none.
bool fill_packed(qa::Q8RowsParams &p, const qa_config &g, int s0, int n, const int32_t *start, const int32_t *ntok,
                 int64_t row0, int (*items)(int, int)) {
    p.nseq = n;
    p.seq0 = s0;
    p.tok = static_cast<int64_t>(g.n_kv_heads) * g.head_dim;
    p.head = g.head_dim;
    p.item0[0] = 0;
    for (int i = 0; i < n; ++i) {
        p.start[i] = start[s0 + i];
        p.ntok[i] = ntok[s0 + i];
        p.off[i] = row0 * p.tok;
        p.item0[i + 1] = p.item0[i] + (p.ntok[i] > 0 ? items(p.start[i], p.start[i] + p.ntok[i]) : 0);
        row0 += p.ntok[i];
    }
    return p.item0[n] > 0;
}

int write_items(int start, int end) { return qa::q8_write_items(start, end); }
int read_items(int start, int end) { return qa::q8_read_items(start, end); }

struct StepCall {
    const int32_t *positions;  // host positions (null: device positions)
    const int32_t *pos_dev;
    int n_blocks;
    const void *q, *k, *v, *wq, *wk;
    void *out, *blocks, *k_held, *v_held;
};

qa_status run_step(qa_q8_cache *c, int layer, int batch, const StepCall &a, cudaStream_t s) {
    const qa_config &g = c->cfg;
    qa::Q8StepParams p{};
    p.layer = layer_of(c, layer);
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
    p.blocks = static_cast<int32_t *>(a.blocks);
    p.err = c->err;
    p.n_blocks = a.n_blocks;
    p.Hq = g.n_q_heads;
    p.G = g.n_q_heads / g.n_kv_heads;
    p.cap = g.capacity;
    p.eps = g.rms_eps;
    p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(g.head_dim)));
    qa::StreamRef at = qa::stream_ref(s, c->device);
    const int64_t resident = std::max<int64_t>(qa::k3_max_resident_ctas(), 2 * c->num_sms);
    for (int b0 = 0; b0 < batch; b0 += qa::kQ8MaxSeqPerLaunch) {
        const int n = std::min(qa::kQ8MaxSeqPerLaunch, batch - b0);
        for (int i = 0; i < n; ++i) p.seq[i] = {a.pos_dev ? g.capacity - 1 : a.positions[b0 + i], b0 + i, 0, 0};
        // The longest sequences, which have the most CTAs, first.
        std::sort(p.seq, p.seq + n, [](const qa::Q8Seq &x, const qa::Q8Seq &y) { return x.pos != y.pos ? x.pos > y.pos : x.slot < y.slot; });
        int work[qa::kQ8MaxSeqPerLaunch], splits[qa::kQ8MaxSeqPerLaunch];
        for (int i = 0; i < n; ++i) work[i] = qa::q8_step_work(g.head_dim, p.seq[i].pos / qa::kQ8Block, a.n_blocks);
        const int longest = p.seq[0].pos / qa::kQ8Block;
        p.n_scores = a.blocks && longest > a.n_blocks ? longest : 0;
        const int per_sm = qa::q8_ctas_per_sm(c->sm_smem, c->reserved_smem, qa::q8_step_smem(p, g.head_dim));
        p.cluster = qa::q8_plan_step(c->num_sms, g.n_kv_heads, qa::kQ8MaxSplits, n, work, splits, per_sm);
        p.nseq = n;
        p.ctas = 0;
        p.per_seq = splits[n - 1] == p.cluster ? p.cluster * g.n_kv_heads : 0;
        for (int i = 0; i < n; ++i) {
            p.seq[i].cta0 = p.ctas;
            while (1 << p.seq[i].log_S < splits[i]) ++p.seq[i].log_S;
            p.ctas += splits[i] * g.n_kv_heads;
        }
        p.early = !a.pos_dev && qa::launch_order().layer_settled(at, c, layer, resident) ? 1 : 0;
        const qa::FaultPlan f = qa::take_fault(QA_KERNEL_DECODE_ATTN);
        p.fault = f.fault;
        p.wait_ns = f.wait_ns;
        if (qa::launch_q8_decode(p, g.head_dim, s) != cudaSuccess) {
            cudaGetLastError();
            return QA_ERR_CUDA;
        }
        qa::launch_order().admit(at, c, layer, p.ctas, 1, p.early != 0, resident);
        qa::note_launch(at, s);
        c->launches[a.blocks ? QA_Q8_KERNEL_SPARSE : QA_Q8_KERNEL_DECODE]++;
    }
    return QA_OK;
}

// The checks that the four step calls share.
qa_status step(qa_q8_cache *c, int layer, int batch, const StepCall &a, bool sparse, void *stream) {
    const qa_status st = check_layer(c, layer, batch);
    if (st != QA_OK) return st;
    const qa_config &g = c->cfg;
    if (!a.positions && !a.pos_dev) return QA_ERR_INVALID_ARG;
    if (a.positions) {
        for (int b = 0; b < batch; ++b)
            if (a.positions[b] < 0) return QA_ERR_INVALID_ARG;
        for (int b = 0; b < batch; ++b)
            if (a.positions[b] >= g.capacity) return QA_ERR_CAPACITY;
    }
    if (!a.q || !a.k || !a.v || !a.out) return QA_ERR_INVALID_ARG;
    if ((a.wq == nullptr) != (a.wk == nullptr)) return QA_ERR_INVALID_ARG;
    if ((a.k_held == nullptr) != (a.v_held == nullptr)) return QA_ERR_INVALID_ARG;
    if (sparse && (!a.blocks || a.n_blocks < 1 || a.n_blocks > c->nblk)) return QA_ERR_INVALID_ARG;
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.wq) || !aligned16(a.wk) ||
        !aligned16(a.out) || !aligned16(a.k_held) || !aligned16(a.v_held) ||
        (reinterpret_cast<uintptr_t>(a.pos_dev) & 3u) || (reinterpret_cast<uintptr_t>(a.blocks) & 3u))
        return QA_ERR_ALIGNMENT;
    const int64_t D2 = 2 * g.head_dim, qb = batch * g.n_q_heads * D2, kb = batch * g.n_kv_heads * D2;
    if (!apart({Span{a.q, qb}, Span{a.k, kb}, Span{a.v, kb}, Span{a.wq, D2}, Span{a.wk, D2}, Span{a.pos_dev, 4ll * batch}},
               {Span{a.out, qb}, Span{a.k_held, kb}, Span{a.v_held, kb},
                Span{a.blocks, 4ll * batch * g.n_kv_heads * a.n_blocks}}))
        return QA_ERR_INVALID_ARG;
    DeviceScope dev(c->device);
    if (!dev.ok()) return QA_ERR_CUDA;
    return no_throw([&] { return run_step(c, layer, batch, a, static_cast<cudaStream_t>(stream)); });
}

// One launch group of a prefill: up to ws.slots() sequences.
struct PrefillGroup {
    qa::Q8PrefillRowsParams rows;
    qa::Q8RowsParams older;
    qa::K2Job k2;
};

bool plan_prefill(qa_q8_cache *c, int layer, int s0, int n, const int32_t *start, const int32_t *ntok, int64_t row0,
                  const void *q, const void *k, const void *v, const void *wq, const void *wk, void *out, PrefillGroup &pg) {
    const qa_config &g = c->cfg;
    const int D = g.head_dim, Hq = g.n_q_heads, Hkv = g.n_kv_heads;
    const int64_t ws_seq = c->ws.seq_stride();
    pg.rows = qa::Q8PrefillRowsParams{};
    qa::K1Params &k1 = pg.rows.k1;
    k1.q = static_cast<const __nv_bfloat16 *>(q) + row0 * Hq * D;
    k1.k = static_cast<const __nv_bfloat16 *>(k) + row0 * Hkv * D;
    k1.v = static_cast<const __nv_bfloat16 *>(v) + row0 * Hkv * D;
    k1.wq = static_cast<const __nv_bfloat16 *>(wq);
    k1.wk = static_cast<const __nv_bfloat16 *>(wk);
    k1.qp = static_cast<__nv_bfloat16 *>(out) + row0 * Hq * D;
    k1.kc = c->ws.rows(0);
    k1.vc = c->ws.rows(1);
    k1.rope = c->rope;
    k1.head_stride = c->ws.head_stride();
    k1.seq_stride = ws_seq;
    k1.Hq = Hq;
    k1.Hkv = Hkv;
    k1.eps = g.rms_eps;
    k1.nseq = n;
    pg.rows.layer = layer_of(c, layer);
    pg.rows.tickets = c->tickets;
    pg.rows.seq0 = s0;
    pg.older = qa::Q8RowsParams{};
    pg.older.layer = pg.rows.layer;
    pg.older.rows[0] = c->ws.rows(0);
    pg.older.rows[1] = c->ws.rows(1);
    pg.older.tok = D;
    pg.older.head = c->ws.head_stride();
    pg.older.nseq = n;
    pg.older.seq0 = s0;
    pg.older.factors = c->ws.factors();
    pg.older.factor_stride = c->ws.factor_stride();
    bool scaled = false;  // some chunk sees a complete block
    for (int i = 0; i < n; ++i) {
        const int P = start[s0 + i], N = ntok[s0 + i];
        k1.cu[i + 1] = k1.cu[i] + N;
        k1.start[i] = P;
        pg.rows.item0[i + 1] = pg.rows.item0[i] + (N > 0 ? qa::q8_read_items(P, P + N) : 0);
        // The complete blocks before the new rows, and the factors of all tiles.
        pg.older.ntok[i] = P / qa::kQ8Block * qa::kQ8Block;
        pg.older.off[i] = i * ws_seq;
        pg.older.item0[i + 1] = pg.older.item0[i] + (N > 0 ? qa::q8_tile_items(P + N) : 0);
        scaled = scaled || (N > 0 && P >= qa::kQ8Block);
    }
    if (!scaled) pg.older.item0[n] = 0;  // nothing to read, no factors
    k1.T = k1.cu[n];
    return k1.T == 0 || c->ws.plan(0, n, start + s0, ntok + s0, k1.cu, k1.qp, c->err, scaled, pg.k2);
}

}  // namespace

QA_API qa_status qa_q8_cache_alloc(const qa_config *cfg, qa_q8_cache **out) {
    if (!cfg || !out) return QA_ERR_INVALID_ARG;
    *out = nullptr;
    const qa_config g = *cfg;
    if (g.num_layers <= 0 || g.max_batch <= 0 || g.capacity <= 0 || g.n_q_heads <= 0 ||
        g.n_kv_heads <= 0 || g.head_dim <= 0 || !(g.rope_theta > 0.f) || !(g.rms_eps >= 0.f))
        return QA_ERR_INVALID_ARG;
    if (!qa::supported_geometry(g.n_q_heads, g.n_kv_heads, g.head_dim)) return QA_ERR_UNSUPPORTED_SHAPE;
    if (g.capacity > qa::kQ8MaxBlocks * qa::kQ8Block || g.max_batch > 65535 || g.n_q_heads > 65535)
        return QA_ERR_UNSUPPORTED_SHAPE;
    const int nblk = (g.capacity + qa::kQ8Block - 1) / qa::kQ8Block;
    const size_t heads = static_cast<size_t>(g.num_layers) * g.max_batch * g.n_kv_heads;  // (below 2^63)
    if (heads > (size_t(1) << 40) / nblk) return QA_ERR_UNSUPPORTED_SHAPE;  // the sums of bytes below stay in 64 bits
    qa_q8_cache *c = new (std::nothrow) qa_q8_cache();
    if (!c) return QA_ERR_CUDA;
    c->cfg = g;
    for (auto &x : c->launches) x = 0;
    c->nblk = nblk;
    const size_t blocks = heads * nblk;
    const size_t D = g.head_dim;
    const size_t codes = blocks * 2 * qa::kQ8Block * D, scales = blocks * sizeof(float2), bounds = blocks * 2 * D;
    const size_t tail = heads * 4 * qa::kQ8Block * D * sizeof(__nv_bfloat16), state = heads * sizeof(qa::Q8Tail);
    const size_t tickets = static_cast<size_t>(qa::kMaxSeqPerLaunch) * g.n_kv_heads * sizeof(uint32_t);
    const size_t total = align256(codes) + align256(scales) + align256(bounds) + align256(tail) + align256(state) +
                         align256(tickets) + 256;
    bool ok = cudaGetDevice(&c->device) == cudaSuccess &&
              cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, c->device) == cudaSuccess &&
              cudaDeviceGetAttribute(&c->sm_smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, c->device) == cudaSuccess &&
              cudaDeviceGetAttribute(&c->reserved_smem, cudaDevAttrReservedSharedMemoryPerBlock, c->device) == cudaSuccess &&
              cudaMalloc(&c->mem, total) == cudaSuccess && cudaMemsetAsync(c->mem, 0, total, nullptr) == cudaSuccess;
    ok = ok && no_throw([&] {
        uint8_t *at = static_cast<uint8_t *>(c->mem);
        auto take = [&](size_t bytes) {
            uint8_t *p = at;
            at += align256(bytes);
            return p;
        };
        c->codes = take(codes);
        c->scales = reinterpret_cast<float2 *>(take(scales));
        c->bounds = reinterpret_cast<int8_t *>(take(bounds));
        c->tail = reinterpret_cast<__nv_bfloat16 *>(take(tail));
        c->state = reinterpret_cast<qa::Q8Tail *>(take(state));
        c->tickets = reinterpret_cast<uint32_t *>(take(tickets));
        c->err = reinterpret_cast<uint32_t *>(at);
        if (cudaMemsetAsync(c->state, 0xff, state, nullptr) != cudaSuccess) return QA_ERR_CUDA;  // no rows kept
        c->rope = qa::rope_table_take(c->device, g.rope_theta, g.head_dim, g.capacity);
        return c->rope && cudaStreamSynchronize(nullptr) == cudaSuccess ? QA_OK : QA_ERR_CUDA;
    }) == QA_OK;
    c->ws.init(g, c->num_sms, true);
    c->cache_bytes = codes + scales + bounds + tail + state;
    c->scratch_bytes = 256 + tickets + c->ws.bytes() + static_cast<size_t>(g.capacity) * (g.head_dim / 2) * sizeof(float2);
    if (!ok) {
        free_all(c);
        delete c;
        cudaGetLastError();
        return QA_ERR_CUDA;
    }
    *out = c;
    return QA_OK;
}

QA_API qa_status qa_q8_cache_free(qa_q8_cache *c) {
    if (!c) return QA_OK;
    DeviceScope dev(c->device);
    qa::synchronise_device();
    free_all(c);
    delete c;
    return QA_OK;
}

QA_API qa_status qa_q8_append(qa_q8_cache *c, int layer, int batch, const int32_t *start, const int32_t *ntok,
                              const void *k, const void *v, void *stream) {
    qa_status st = check_layer(c, layer, batch);
    if (st != QA_OK) return st;
    int64_t T = 0;
    st = check_ranges(c, batch, start, ntok, &T);
    if (st != QA_OK) return st;
    if (T == 0) return QA_OK;
    if (!k || !v) return QA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v)) return QA_ERR_ALIGNMENT;
    DeviceScope dev(c->device);
    if (!dev.ok()) return QA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    qa::Q8RowsParams p{};
    p.layer = layer_of(c, layer);
    p.rows[0] = static_cast<__nv_bfloat16 *>(const_cast<void *>(k));
    p.rows[1] = static_cast<__nv_bfloat16 *>(const_cast<void *>(v));
    return no_throw([&] {
        qa::StreamRef at = qa::stream_ref(s, c->device);
        int64_t row0 = 0;
        for (int s0 = 0; s0 < batch; s0 += qa::kQ8MaxSeqPerLaunch) {
            const int n = std::min(qa::kQ8MaxSeqPerLaunch, batch - s0);
            if (fill_packed(p, c->cfg, s0, n, start, ntok, row0, write_items)) {
                if (qa::launch_q8_write(p, c->cfg.head_dim, s) != cudaSuccess) {
                    cudaGetLastError();
                    return QA_ERR_CUDA;
                }
                // It lets the next launch start once it has itself waited, while it writes.
                qa::launch_order().admit(at, c, layer, 1, 1, false, 1);
                qa::note_launch(at, s);
                c->launches[QA_Q8_KERNEL_WRITE]++;
            }
            for (int i = 0; i < n; ++i) row0 += ntok[s0 + i];
        }
        return QA_OK;
    });
}

QA_API qa_status qa_q8_read(qa_q8_cache *c, int layer, int batch, const int32_t *start, const int32_t *ntok,
                            void *k_out, void *v_out, void *stream) {
    qa_status st = check_layer(c, layer, batch);
    if (st != QA_OK) return st;
    int64_t T = 0;
    st = check_ranges(c, batch, start, ntok, &T);
    if (st != QA_OK) return st;
    if (T == 0) return QA_OK;
    if (!k_out && !v_out) return QA_ERR_INVALID_ARG;
    if (!aligned16(k_out) || !aligned16(v_out)) return QA_ERR_ALIGNMENT;
    const int64_t kb = T * c->cfg.n_kv_heads * 2 * c->cfg.head_dim;
    if (overlap({k_out, kb}, {v_out, kb})) return QA_ERR_INVALID_ARG;
    DeviceScope dev(c->device);
    if (!dev.ok()) return QA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    qa::Q8RowsParams p{};
    p.layer = layer_of(c, layer);
    p.rows[0] = static_cast<__nv_bfloat16 *>(k_out);
    p.rows[1] = static_cast<__nv_bfloat16 *>(v_out);
    return no_throw([&] {
        int64_t row0 = 0;
        for (int s0 = 0; s0 < batch; s0 += qa::kQ8MaxSeqPerLaunch) {
            const int n = std::min(qa::kQ8MaxSeqPerLaunch, batch - s0);
            if (fill_packed(p, c->cfg, s0, n, start, ntok, row0, read_items)) {
                if (qa::launch_q8_read(p, c->cfg.head_dim, s) != cudaSuccess) {
                    cudaGetLastError();
                    return QA_ERR_CUDA;
                }
                qa::launch_order().barrier(qa::stream_ref(s, c->device));
                c->launches[QA_Q8_KERNEL_READ]++;
            }
            for (int i = 0; i < n; ++i) row0 += ntok[s0 + i];
        }
        return QA_OK;
    });
}

QA_API qa_status qa_q8_prefill(qa_q8_cache *c, int layer, int batch, const int32_t *start, const int32_t *ntok,
                               const void *q, const void *k, const void *v, const void *q_norm_w, const void *k_norm_w,
                               void *out, void *stream) {
    qa_status st = check_layer(c, layer, batch);
    if (st != QA_OK) return st;
    int64_t T = 0;
    st = check_ranges(c, batch, start, ntok, &T);
    if (st != QA_OK) return st;
    if (T == 0) return QA_OK;
    if (!q || !k || !v || !q_norm_w || !k_norm_w || !out) return QA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_norm_w) || !aligned16(k_norm_w) || !aligned16(out))
        return QA_ERR_ALIGNMENT;
    const qa_config &g = c->cfg;
    const int64_t D2 = 2 * g.head_dim, qb = T * g.n_q_heads * D2, kb = T * g.n_kv_heads * D2;
    if (!apart({Span{q, qb}, Span{k, kb}, Span{v, kb}, Span{q_norm_w, D2}, Span{k_norm_w, D2}}, {Span{out, qb}}))
        return QA_ERR_INVALID_ARG;
    DeviceScope dev(c->device);
    if (!dev.ok()) return QA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // It goes through the cache's one bf16 workspace: a graph could be replayed
    // beside another call that uses it, so it is not captured, and calls on several
    // streams take turns.
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone) {
        cudaGetLastError();
        return QA_ERR_STATE;
    }
    if (!c->ws.take()) {
        cudaGetLastError();
        return QA_ERR_CUDA;
    }
    std::vector<PrefillGroup> groups;
    st = no_throw([&] {
        int64_t row0 = 0;
        for (int s0 = 0; s0 < batch; s0 += c->ws.slots()) {
            const int n = std::min(c->ws.slots(), batch - s0);
            groups.emplace_back();
            if (!plan_prefill(c, layer, s0, n, start, ntok, row0, q, k, v, q_norm_w, k_norm_w, out, groups.back())) {
                cudaGetLastError();
                return QA_ERR_CUDA;
            }
            row0 += groups.back().rows.k1.T;
        }
        return QA_OK;
    });
    if (st != QA_OK) return st;
    if (cudaStreamWaitEvent(s, c->ws.free_event(), 0) != cudaSuccess) return QA_ERR_CUDA;
    const qa::StreamRef at(s, c->device);  // (not being captured)
    auto launch = [&](PrefillGroup &pg) {
        auto done = [&](cudaError_t e, int kernel) {
            if (e != cudaSuccess) {
                cudaGetLastError();
                return false;
            }
            qa::launch_order().barrier(at);
            c->launches[kernel]++;
            return true;
        };
        if (pg.rows.k1.T == 0) return QA_OK;
        if (!done(qa::launch_q8_prefill_rows(pg.rows, g.head_dim, s), QA_Q8_KERNEL_WRITE) ||
            (pg.older.item0[pg.older.nseq] > 0 && !done(qa::launch_q8_read(pg.older, g.head_dim, s), QA_Q8_KERNEL_READ)) ||
            !done(c->ws.launch(pg.k2, s), QA_Q8_KERNEL_PREFILL_ATTN)) {
            // What was enqueued may no longer be followed by a kernel that waits for it: let
            // it finish before anything else is enqueued.
            cudaStreamSynchronize(s);
            return QA_ERR_CUDA;
        }
        return QA_OK;
    };
    for (size_t i = 0; i < groups.size() && st == QA_OK; ++i) st = no_throw([&] { return launch(groups[i]); });
    // After a failure too: what was enqueued uses the workspace.
    if (cudaEventRecord(c->ws.free_event(), s) != cudaSuccess) return QA_ERR_CUDA;
    return st;
}

QA_API qa_status qa_q8_decode_step(qa_q8_cache *c, int layer, int batch, const int32_t *positions, const void *q,
                                   const void *k, const void *v, const void *q_norm_w, const void *k_norm_w, void *out,
                                   void *k_held, void *v_held, void *stream) {
    return step(c, layer, batch, {positions, nullptr, 0, q, k, v, q_norm_w, k_norm_w, out, nullptr, k_held, v_held}, false,
                stream);
}

QA_API qa_status qa_q8_decode_step_device_positions(qa_q8_cache *c, int layer, int batch, const int32_t *positions,
                                                    const void *q, const void *k, const void *v, const void *q_norm_w,
                                                    const void *k_norm_w, void *out, void *k_held, void *v_held,
                                                    void *stream) {
    return step(c, layer, batch, {nullptr, positions, 0, q, k, v, q_norm_w, k_norm_w, out, nullptr, k_held, v_held}, false,
                stream);
}

QA_API qa_status qa_q8_sparse_step(qa_q8_cache *c, int layer, int batch, const int32_t *positions, int n_blocks,
                                   const void *q, const void *k, const void *v, const void *q_norm_w,
                                   const void *k_norm_w, void *out, int32_t *blocks, void *k_held, void *v_held,
                                   void *stream) {
    return step(c, layer, batch, {positions, nullptr, n_blocks, q, k, v, q_norm_w, k_norm_w, out, blocks, k_held, v_held},
                true, stream);
}

QA_API qa_status qa_q8_sparse_step_device_positions(qa_q8_cache *c, int layer, int batch, const int32_t *positions,
                                                    int n_blocks, const void *q, const void *k, const void *v,
                                                    const void *q_norm_w, const void *k_norm_w, void *out,
                                                    int32_t *blocks, void *k_held, void *v_held, void *stream) {
    return step(c, layer, batch, {nullptr, positions, n_blocks, q, k, v, q_norm_w, k_norm_w, out, blocks, k_held, v_held},
                true, stream);
}

QA_API qa_status qa_q8_get_device_error(qa_q8_cache *c, uint32_t *detail) {
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

QA_API qa_status qa_q8_stats(qa_q8_cache *c, uint64_t launches[QA_Q8_NUM_KERNELS]) {
    if (!c || !launches) return QA_ERR_INVALID_ARG;
    for (int i = 0; i < QA_Q8_NUM_KERNELS; ++i) launches[i] = c->launches[i].load();
    return QA_OK;
}

QA_API qa_status qa_q8_memory_info(qa_q8_cache *c, uint64_t *cache_bytes, uint64_t *scratch_bytes) {
    if (!c) return QA_ERR_INVALID_ARG;
    if (cache_bytes) *cache_bytes = c->cache_bytes;
    if (scratch_bytes) *scratch_bytes = c->scratch_bytes;
    return QA_OK;
}
