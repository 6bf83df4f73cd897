// k6_q8_rows.cu -- K6: rows of keys and values into the 8-bit cache, and back.
//
// A thread block works on one block of 64 positions of one kv head, K and V: the
// largest magnitude of 64 x D values gives the scale, so all of them are loaded
// (32 KB at D = 128, 16-byte loads, all in flight before any arithmetic), reduced,
// and written as codes.  Bound by HBM.
#include <algorithm>

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
        return *reinterpret_cast<const uint4 *>((kv ? src[1] : src[0]) + static_cast<int64_t>(pos - p.first[z]) * p.tok + d0);
    };
    const int kv_of_warp = threadIdx.x >> 7, kt = threadIdx.x >> 5 & 3;  // four warps for K, four for V
    uint4 x[D / 16];
    if (i > 0) {  // every row of the block is new
        const int blk = first + i;
        q8_seal_rows<D>(kv_of_warp, kt, sm, x, [&](int kv, int r, int d0) { return source8(kv, blk * kQ8Block + r, d0); });
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
        if (pos >= p.first[z]) return source8(kv, pos, d0);
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
        q8_seal_rows<D>(kv_of_warp, kt, sm, x, row8);
        __syncthreads();  // (and every warp has read what it needs of the old codes)
        q8_store<D>(p.layer, sh, first, kv_of_warp, kt, q8_seal_codes<D>(kv_of_warp, kt, sm, x));
    }
    __syncthreads();  // every thread has read the state
    if (threadIdx.x == 0) p.layer.state[sh] = plan.next;
}

// The codes of a block pass through shared memory, so that both sides move whole lines.
// kFactors: the rows before a chunk of a prefill, into the attention's workspace.
// There a row of a complete block is its codes (bf16 holds them exactly) and the
// scales are factors of the block; its product with the scale would be rounded once
// more.  Blocks of zeros and of NaN, and rows in bf16, have the factor 1.
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
    const bool held = kFactors && hi == kQ8Block;  // complete, for the chunk
    float2 scale = make_float2(0.f, 0.f);
    if (hi > lo) scale = p.layer.scales[sh * p.layer.nblk + blk];
    if (kFactors) {
        const bool fk = held && scale.x > 0.f, fv = held && scale.y > 0.f;  // (not 0, not NaN)
        if (threadIdx.x == 0)
            p.factors[(static_cast<int64_t>(z) * p.layer.Hkv + h) * p.factor_stride + blk] =
                make_float4(fk ? scale.x : 1.f, fv ? log2f(scale.y) : 0.f, fv ? 1.f / scale.y : 1.f, 0.f);
        if (hi <= lo) return;
        if (fk) scale.x = 1.f;
        if (fv) scale.y = 1.f;
    }
    const Q8Tail state = p.layer.state[sh];
    auto buffer_of = [&](int r) { return held ? -1 : q8_tail_of(state, blk, r, kFactors); };
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
            *reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(blk * kQ8Block + r - p.first[z]) * p.tok + d0) = x;
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
cudaError_t launch_q8_read(const Q8RowsParams &p, int D, cudaStream_t stream) {
    if (p.factors) return q8_launch_rows(D == 128 ? q8_read_kernel<128, true> : q8_read_kernel<64, true>, p, stream);
    return q8_launch_rows(D == 128 ? q8_read_kernel<128, false> : q8_read_kernel<64, false>, p, stream);
}

}  // namespace qa
