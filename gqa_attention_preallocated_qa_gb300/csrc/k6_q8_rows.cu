// k6_q8_rows.cu -- K6: rows of keys and values into the 8-bit cache, and back.
//
// A thread block works on one block of 64 positions of one kv head, K and V: the
// largest magnitude of 64 x D values gives the scale, so all of them are loaded
// (32 KB at D = 128, 16-byte loads, all in flight before any arithmetic), reduced,
// and written as codes.  Bound by HBM.
#include <algorithm>
#include <atomic>

#include "q8_device.cuh"

namespace qa {

// The launched sequence of a work item.
__device__ __forceinline__ int q8_sequence(const Q8RowsParams &p, int item) {
    int lo = 0, hi = p.nseq;  // item0[lo] <= item < item0[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.item0[mid] <= item) lo = mid; else hi = mid;
    }
    return lo;
}

template <int D>
__device__ __forceinline__ __nv_bfloat16 *q8_tail_rows(const Q8Layer &l, int64_t sh, int buffer, int kv) {
    return l.tail + ((sh * 2 + buffer) * 2 + kv) * static_cast<int64_t>(kQ8Block * D);
}

template <int D>
__global__ void __launch_bounds__(256) q8_write_kernel(const __grid_constant__ Q8RowsParams p) {
    __shared__ Q8SealSmem<D> sm;
    griddep_wait();
    griddep_launch_dependents();
    const int z = q8_sequence(p, blockIdx.x), h = blockIdx.y;
    const int i = blockIdx.x - p.item0[z];
    const int start = p.start[z], end = start + p.ntok[z], first = start / kQ8Block;
    const int64_t sh = static_cast<int64_t>(p.seq0 + z) * p.layer.Hkv + h;
    const __nv_bfloat16 *src[2] = {p.rows[0] + p.off[z] + h * p.head, p.rows[1] + p.off[z] + h * p.head};
    auto source8 = [&](int kv, int pos, int d0) {
        return *reinterpret_cast<const uint4 *>((kv ? src[1] : src[0]) + static_cast<int64_t>(pos - start) * p.tok + d0);
    };
    const int kv_of_warp = threadIdx.x >> 7, kt = threadIdx.x >> 5 & 3;  // four warps for K, four for V
    uint4 x[D / 16];
    if (i > 0) {  // every row of the block is new
        const int blk = first + i;
        q8_seal_load<D>(kv_of_warp, kt, x, [&](int kv, int r, int d0) { return source8(kv, blk * kQ8Block + r, d0); });
        q8_seal_sums<D>(kv_of_warp, kt, sm, x);
        __syncthreads();
        q8_store<D>(p.layer, sh, blk, kv_of_warp, kt, q8_seal_codes<D>(kv_of_warp, kt, sm, x));
        return;
    }
    const Q8Tail state = p.layer.state[sh];
    const Q8TailPlan plan = q8_plan_tail(state, start, end, false);
    const uint8_t *codes = p.layer.codes + (sh * p.layer.nblk + first) * static_cast<int64_t>(2 * kQ8Block * D);
    const float2 scale = p.layer.scales[sh * p.layer.nblk + first];
    auto row8 = [&](int kv, int r, int d0) {  // of the first block: new, kept, or from the codes
        const int pos = first * kQ8Block + r;
        if (pos >= start) return source8(kv, pos, d0);
        if (r < plan.from_rows)
            return *reinterpret_cast<const uint4 *>(q8_tail_rows<D>(p.layer, sh, plan.from, kv) + r * D + d0);
        return q8_row8<D>(codes + kv * kQ8Block * D, kv != 0, kv ? scale.y : scale.x, r, d0);
    };
    if (plan.dst >= 0) {  // rows of the last block: all of a lane's on the way at once
        const int last = (end - 1) / kQ8Block, rest = end - last * kQ8Block;
        const int from = last == first ? plan.from_rows : 0;  // (below it the buffer has them)
        constexpr int kRows = 256 / (D / 8), kTurns = kQ8Block / kRows;  // rows of a turn of the CTA
        const int d0 = threadIdx.x % (D / 8) * 8;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            uint4 y[kTurns];
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
                const int r = from + k * kRows + threadIdx.x / (D / 8);
                if (r < rest) y[k] = last == first ? row8(kv, r, d0) : source8(kv, last * kQ8Block + r, d0);
            }
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
                const int r = from + k * kRows + threadIdx.x / (D / 8);
                if (r < rest) *reinterpret_cast<uint4 *>(q8_tail_rows<D>(p.layer, sh, plan.dst, kv) + r * D + d0) = y[k];
            }
        }
    }
    if (end >= (first + 1) * kQ8Block) {
        q8_seal_load<D>(kv_of_warp, kt, x, row8);
        q8_seal_sums<D>(kv_of_warp, kt, sm, x);
        __syncthreads();  // (and every warp has read what it needs of the old codes)
        q8_store<D>(p.layer, sh, first, kv_of_warp, kt, q8_seal_codes<D>(kv_of_warp, kt, sm, x));
    }
    __syncthreads();  // every thread has read the state
    if (threadIdx.x == 0) p.layer.state[sh] = plan.next;
}

// -------------------------------------------------------------------- a prefill's rows
// RMSNorm and rotation of a block's keys and of the queries that share its kv head, into
// the attention's workspace and the staging buffer, and the block's codes (or the rows to
// keep) on the way: each row is read once and written once.  A row of keys or queries is
// on four lanes, 8 dims of every 32 each, as the codes' layout has it: a rotated pair is
// in one lane, and the sum of squares adds up in the order of norm_rope_row, so that a key
// gets the same bits from a prefill and from a step.  The rotary rows are shared by the
// block's 1 + G heads through shared memory.
//   K1 and q8_write_kernel after it take one pass more over keys and values and one launch
// more.  A call takes, with them / with this (32/8 heads, D = 128): 1778 tokens of two
// chunks 119 / 113 us, 64 tokens (2/1 heads, D = 64) 13.6 / 12.5, 4 x 2048 171 / 176.  At 8192
// tokens this takes 48 us alone, 4.5 TB/s: two CTAs of 8 warps an SM, for their 128
// registers, fill half of the issue slots; with three of 80 registers that call took 187.
template <int D>
struct alignas(16) Q8RowsSmem {
    // Rotary rows, (cos_a, sin_a, cos_b, sin_b) of two pairs each: pairs 16 c + 4 t + e at
    // 16 c + 4 e + t, and 64 bytes between rows: eight lanes read 128 bytes of all banks.
    float4 cs[kQ8Block][D / 4 + 4];
    uint4 w[2][D / 8];                // norm weights of queries and keys
    Q8SealSmem<D> seal;
};
// A row in x[c], c = 0 .. D/32 - 1; w, cs: weights and its rotary row, in shared memory.
template <int D>
__device__ __forceinline__ void q8_norm_rope(uint4 (&x)[D / 32], const uint4 *w, float eps, const float4 *cs) {
    constexpr int C = D / 32;
    const unsigned FULL = 0xffffffffu;
    float part[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const uint32_t xw[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
        part[c] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) part[c] = fmaf(bf16lo(xw[e]), bf16lo(xw[e]), fmaf(bf16hi(xw[e]), bf16hi(xw[e]), part[c]));
    }
    float ss = C == 4 ? (part[0] + part[C / 2]) + (part[1] + part[C - 1]) : part[0] + part[1];
    ss += __shfl_xor_sync(FULL, ss, 2);
    ss += __shfl_xor_sync(FULL, ss, 1);
    const float r = rsqrtf(ss * (1.0f / D) + eps);
    auto scaled = [&](uint32_t xw, uint32_t ww) {
        return pack_bf16(bf16lo(ww) * round_bf16(bf16lo(xw) * r), bf16hi(ww) * round_bf16(bf16hi(xw) * r));
    };
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int c = 0; c < C / 2; ++c) {  // dims 32 c + 8 t .. of the lower half, and their partners
        const uint4 wa = w[4 * c + t], wc = w[4 * (c + C / 2) + t], xc = x[c + C / 2];
        const uint32_t xl[4] = {x[c].x, x[c].y, x[c].z, x[c].w}, wl[4] = {wa.x, wa.y, wa.z, wa.w};
        const uint32_t xh[4] = {xc.x, xc.y, xc.z, xc.w}, wh[4] = {wc.x, wc.y, wc.z, wc.w};
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 a = cs[16 * c + 4 * e + t];
            const uint32_t u = scaled(xl[e], wl[e]), v = scaled(xh[e], wh[e]);
            lo[e] = pack_bf16(fmaf(-a.y, bf16lo(v), bf16lo(u) * a.x), fmaf(-a.w, bf16hi(v), bf16hi(u) * a.z));
            hi[e] = pack_bf16(fmaf(a.y, bf16lo(u), bf16lo(v) * a.x), fmaf(a.w, bf16hi(u), bf16hi(v) * a.z));
        }
        x[c] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        x[c + C / 2] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
}

template <int D>
__global__ void __launch_bounds__(256, 2) q8_prefill_rows_kernel(const __grid_constant__ Q8PrefillRowsParams p) {
    extern __shared__ uint4 smem[];
    Q8RowsSmem<D> &sm = *reinterpret_cast<Q8RowsSmem<D> *>(smem);
    griddep_wait();
    griddep_launch_dependents();
    const K1Params &k1 = p.k1;
    const int h = blockIdx.y, G = k1.Hq / k1.Hkv;
    int z = 0;
    while (z + 1 < k1.nseq && p.item0[z + 1] <= static_cast<int>(blockIdx.x)) ++z;
    const int start = k1.start[z], end = start + k1.cu[z + 1] - k1.cu[z];
    const int first = start / kQ8Block, last = (end - 1) / kQ8Block, rest = end - last * kQ8Block;
    const int blk = first + static_cast<int>(blockIdx.x) - p.item0[z];
    // The block's new rows are lo .. hi - 1; earlier ones are in its kept rows or codes.
    const int lo = max(start - blk * kQ8Block, 0), hi = min(end - blk * kQ8Block, kQ8Block);
    const int64_t sh = static_cast<int64_t>(p.seq0 + z) * p.layer.Hkv + h;
    const int64_t row0 = k1.cu[z] + static_cast<int64_t>(blk) * kQ8Block - start;  // packed row of the block's row 0
    for (int e = threadIdx.x; e < (hi - lo) * (D / 4); e += 256) {
        const int r = lo + e / (D / 4), i = e % (D / 4);
        q8_copy16(&sm.cs[r][(i & ~15) | (i & 3) << 2 | (i >> 2 & 3)],
                  reinterpret_cast<const float4 *>(k1.rope + static_cast<int64_t>(blk * kQ8Block + r) * (D / 2)) + i);
    }
    if (threadIdx.x < D / 4) {
        const int i = threadIdx.x % (D / 8);
        q8_copy16(&sm.w[threadIdx.x / (D / 8)][i], reinterpret_cast<const uint4 *>(threadIdx.x < D / 8 ? k1.wq : k1.wk) + i);
    }
    // Four warps take K, four V.  Of the 2 G turns of 8 query rows (row g or g + 8 of a warp's
    // 16, of one head) the latter, who norm nothing else, take two more.
    const int kv = threadIdx.x >> 7, kt = threadIdx.x >> 5 & 3;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int turns = kv ? G + 1 : G - 1, turn0 = kv ? 0 : G + 1;
    auto row_of = [&](int turn) { return 16 * kt + g + 8 * ((turn0 + turn) & 1); };
    auto live = [&](int turn) { return row_of(turn) >= lo && row_of(turn) < hi; };
    auto place = [&](int turn) { return ((row0 + row_of(turn)) * k1.Hq + h * G + ((turn0 + turn) >> 1)) * D + 8 * t; };
    auto load = [&](int turn, uint4 (&y)[D / 32]) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            y[c] = make_uint4(0, 0, 0, 0);
            if (turn < turns && live(turn)) y[c] = *reinterpret_cast<const uint4 *>(k1.q + place(turn) + 32 * c);
        }
    };
    const bool mine = blk == first || (blk == last && rest < kQ8Block);  // the kept rows matter here
    Q8TailPlan plan{};
    plan.dst = -1;
    if (mine) plan = q8_plan_tail(p.layer.state[sh], start, end, false);
    const uint8_t *codes = p.layer.codes + (sh * p.layer.nblk + blk) * static_cast<int64_t>(2 * kQ8Block * D);
    uint4 x[D / 16];
    auto row8 = [&](int r, int d0) {
        if (r >= hi) return make_uint4(0, 0, 0, 0);
        if (r >= lo) return *reinterpret_cast<const uint4 *>((kv ? k1.v : k1.k) + ((row0 + r) * k1.Hkv + h) * D + d0);
        if (r < plan.from_rows)
            return *reinterpret_cast<const uint4 *>(q8_tail_rows<D>(p.layer, sh, plan.from, kv) + r * D + d0);
        const float2 s = p.layer.scales[sh * p.layer.nblk + blk];
        return q8_row8<D>(codes + kv * kQ8Block * D, kv != 0, kv ? s.y : s.x, r, d0);
    };
#pragma unroll
    for (int i = 0; i < D / 16; ++i) x[i] = row8(q8_seal_row(kv, kt, i), q8_seal_dim<D>(kv, i));
    uint4 even[D / 32], odd[D / 32];
    load(0, even);
    q8_copy_wait();  // the rotary rows
    __syncthreads();
    if (kv == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 16 * kt + g + 8 * i;
            const bool is_new = r >= lo && r < hi;
            uint4 y[D / 32];
#pragma unroll
            for (int c = 0; c < D / 32; ++c) y[c] = x[2 * c + i];
            q8_norm_rope<D>(y, sm.w[1], k1.eps, sm.cs[is_new ? r : lo]);
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                if (is_new) x[2 * c + i] = y[c];
        }
    }
    __nv_bfloat16 *ws = (kv ? k1.vc : k1.kc) + z * k1.seq_stride + h * k1.head_stride + static_cast<int64_t>(blk) * kQ8Block * D;
    __nv_bfloat16 *kept = blk == last && plan.dst >= 0 ? q8_tail_rows<D>(p.layer, sh, plan.dst, kv) : nullptr;
    const int keep = blk == first && plan.dst == plan.from ? plan.from_rows : 0;  // (the buffer has the rows before)
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const int r = q8_seal_row(kv, kt, i), d0 = q8_seal_dim<D>(kv, i);
        if (r >= hi) continue;
        *reinterpret_cast<uint4 *>(ws + r * D + d0) = x[i];
        if (kept && r >= keep) *reinterpret_cast<uint4 *>(kept + r * D + d0) = x[i];
    }
    if (hi == kQ8Block) {
        q8_seal_sums<D>(kv, kt, sm.seal, x);
        named_bar_sync(1 + kv, 128);  // (and each of the four warps has read what it needs of the old codes)
        q8_store<D>(p.layer, sh, blk, kv, kt, q8_seal_codes<D>(kv, kt, sm.seal, x));
    }
    auto finish = [&](int turn, uint4 (&y)[D / 32]) {
        q8_norm_rope<D>(y, sm.w[0], k1.eps, sm.cs[live(turn) ? row_of(turn) : lo]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            if (live(turn)) *reinterpret_cast<uint4 *>(k1.qp + place(turn) + 32 * c) = y[c];
    };
#pragma unroll 1
    for (int turn = 0; turn < turns; turn += 2) {  // (uniform in a warp)
        load(turn + 1, odd);
        finish(turn, even);
        load(turn + 2, even);
        if (turn + 1 < turns) finish(turn + 1, odd);
    }
    if (mine) {
        __syncthreads();  // every thread has read the state
        if (threadIdx.x == 0) {
            // Two thread blocks may need the state as it was: the second one to get here changes it.
            bool write = last == first || rest == kQ8Block;
            if (!write) {
                uint32_t *ticket = p.tickets + z * k1.Hkv + h;
                __threadfence();
                write = atomicAdd(ticket, 1u) == 1u;
                if (write) *ticket = 0u;
            }
            if (write) p.layer.state[sh] = plan.next;
        }
    }
}

// The codes of a block pass through shared memory, so that both sides move whole lines.
// kFactors: the complete blocks before a chunk of a prefill, into the attention's workspace.
// There a row is its codes (bf16 holds them exactly) and the scales are factors of the
// block; its product with the scale would be rounded once more.  Blocks of zeros and of
// NaN, and those of the chunk's own rows, have the factor 1.
template <int D, bool kFactors>
__global__ void __launch_bounds__(256) q8_read_kernel(const __grid_constant__ Q8RowsParams p) {
    __shared__ alignas(16) uint8_t codes[2][kQ8Block * D];
    // For a prefill it runs beside the kernel of the new rows, which starts after all
    // that came before and touches none of these.  The next kernel waits for this grid,
    // whose last block is not done before the new rows are.
    if (!kFactors || (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1)) griddep_wait();
    griddep_launch_dependents();
    const int z = q8_sequence(p, blockIdx.x), h = blockIdx.y;
    const int start = p.start[z], end = start + p.ntok[z];
    const int blk = start / kQ8Block + blockIdx.x - p.item0[z];
    const int lo = max(start - blk * kQ8Block, 0), hi = min(end - blk * kQ8Block, kQ8Block);
    const int64_t sh = static_cast<int64_t>(p.seq0 + z) * p.layer.Hkv + h;
    const bool held = kFactors && hi == kQ8Block;
    float2 scale = make_float2(0.f, 0.f);
    if (held || !kFactors) scale = p.layer.scales[sh * p.layer.nblk + blk];
    if (kFactors) {
        const bool fk = held && scale.x > 0.f, fv = held && scale.y > 0.f;  // (not 0, not NaN)
        if (threadIdx.x == 0)
            p.factors[(static_cast<int64_t>(z) * p.layer.Hkv + h) * p.factor_stride + blk] =
                make_float4(fk ? scale.x : 1.f, fv ? log2f(scale.y) : 0.f, fv ? 1.f / scale.y : 1.f, 0.f);
        if (!held) return;
        if (fk) scale.x = 1.f;
        if (fv) scale.y = 1.f;
    }
    Q8Tail state{};
    if (!kFactors) state = p.layer.state[sh];
    auto buffer_of = [&](int r) { return kFactors ? -1 : q8_tail_of(state, blk, r, false); };
    if (buffer_of(hi - 1) < 0) {
        const uint4 *from = reinterpret_cast<const uint4 *>(p.layer.codes + (sh * p.layer.nblk + blk) * static_cast<int64_t>(2 * kQ8Block * D));
#pragma unroll
        for (int k = 0; k < 2 * kQ8Block * D / (16 * 256); ++k) {
            const int e = threadIdx.x + 256 * k;
            if (p.rows[e / (kQ8Block * D / 16)]) reinterpret_cast<uint4 *>(codes[0])[e] = from[e];
        }
        __syncthreads();
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        if (!p.rows[kv]) continue;
        __nv_bfloat16 *dst = p.rows[kv] + p.off[z] + h * p.head;
        for (int k = threadIdx.x; k < (hi - lo) * (D / 8); k += 256) {
            const int r = lo + k / (D / 8), d0 = k % (D / 8) * 8;
            const int buffer = buffer_of(r);
            const uint4 x = buffer >= 0 ? *reinterpret_cast<const uint4 *>(q8_tail_rows<D>(p.layer, sh, buffer, kv) + r * D + d0)
                                        : q8_row8<D>(codes[kv], kv != 0, kv ? scale.y : scale.x, r, d0);
            *reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(blk * kQ8Block + r - start) * p.tok + d0) = x;
        }
    }
}

// ------------------------------------------------------------------ launch
static cudaError_t q8_launch_rows(void (*kern)(Q8RowsParams), const Q8RowsParams &p, cudaStream_t stream) {
    const int items = p.item0[p.nseq];
    if (items <= 0) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(items, p.layer.Hkv);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_q8_write(const Q8RowsParams &p, int D, cudaStream_t stream) {
    return q8_launch_rows(D == 128 ? q8_write_kernel<128> : q8_write_kernel<64>, p, stream);
}
template <int D>
static cudaError_t q8_launch_prefill_rows(const Q8PrefillRowsParams &p, cudaStream_t stream) {
    static std::atomic<unsigned> configured{0u};  // devices 0..31 set up (one bit each)
    auto kern = q8_prefill_rows_kernel<D>;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 32 || !((configured.load(std::memory_order_acquire) >> dev) & 1u)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Q8RowsSmem<D>));
        if (e != cudaSuccess) return e;
        if (dev < 32) configured.fetch_or(1u << dev, std::memory_order_release);
    }
    const int items = p.item0[p.k1.nseq];
    if (items <= 0) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(items, p.k1.Hkv);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = sizeof(Q8RowsSmem<D>);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}
cudaError_t launch_q8_prefill_rows(const Q8PrefillRowsParams &p, int D, cudaStream_t stream) {
    return D == 128 ? q8_launch_prefill_rows<128>(p, stream) : q8_launch_prefill_rows<64>(p, stream);
}
cudaError_t launch_q8_read(const Q8RowsParams &p, int D, cudaStream_t stream) {
    if (p.factors) return q8_launch_rows(D == 128 ? q8_read_kernel<128, true> : q8_read_kernel<64, true>, p, stream);
    return q8_launch_rows(D == 128 ? q8_read_kernel<128, false> : q8_read_kernel<64, false>, p, stream);
}

}  // namespace qa
