// k4_q4_rows.cu -- K4: quantising rows of keys and values into the 4-bit cache,
// and reading them back.
//
// Both directions move each byte once and are bound by HBM: a row of D values
// is 2 D bytes in bf16 and D/2 + D/32 in the cache.  A warp owns 16 (D = 128)
// or 32 (D = 64) consecutive tokens of one head of K or of V: its rows lie next
// to each other in the cache, so the codes of the block are one contiguous run
// and the scale bytes another.  D/8 lanes hold a row, 8 values each; a group of
// 32 is four lanes, whose largest magnitude takes two shuffles.  All the warp's
// loads are issued before any arithmetic (128 bytes a lane).
#include <algorithm>

#include "q4_device.cuh"

namespace qa {

constexpr int kQ4Unroll = 8;  // rows per lane group

// The block of tokens, head and tensor of a warp.
struct Q4Task {
    int z, kv, h, tok0, n;  // launched sequence, K/V, head, first token, tokens (0: none)
};

template <int D>
__device__ __forceinline__ Q4Task q4_task(const Q4RowsParams &p) {
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
    Q4Task t{0, 0, 0, 0, 0};
    const int per = p.Hkv * p.kv_count;
    const int64_t blk64 = w / per;
    if (blk64 >= p.nblocks) return t;
    const int blk = static_cast<int>(blk64), r = static_cast<int>(w - blk64 * per);
    t.kv = p.kv_first + r / p.Hkv;
    t.h = r % p.Hkv;
    int lo = 0, hi = p.nseq;  // block0[lo] <= blk < block0[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.block0[mid] <= blk) lo = mid; else hi = mid;
    }
    t.z = lo;
    t.tok0 = (blk - p.block0[lo]) * q4_block_tokens(D);
    t.n = min(q4_block_tokens(D), p.ntok[lo] - t.tok0);
    return t;
}

template <int D, bool kHeld>
__global__ void __launch_bounds__(256) q4_quantise_kernel(const __grid_constant__ Q4RowsParams p) {
    constexpr int LPR = D / 8;  // lanes per row
    constexpr int GR = D / kQ4Group;
    const unsigned FULL = 0xffffffffu;
    const Q4Task t = q4_task<D>(p);
    if (t.n <= 0) return;
    const int lane = threadIdx.x & 31, sub = lane % LPR, half = lane / LPR;
    const __nv_bfloat16 *src = p.src[t.kv] + p.src_off[t.z] + t.h * p.src_head;
    uint4 x[kQ4Unroll];
#pragma unroll
    for (int u = 0; u < kQ4Unroll; ++u) {
        const int i = half * kQ4Unroll + u;
        x[u] = make_uint4(0, 0, 0, 0);
        if (i < t.n)
            x[u] = *(reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(t.tok0 + i) * p.src_tok) + sub);
    }
    const int64_t row = static_cast<int64_t>(p.seq0 + t.z) * p.row_seq + t.h * p.row_head +
                        p.start[t.z] + t.tok0;
    uint32_t *codes = reinterpret_cast<uint32_t *>(p.codes[t.kv]) + row * (D / 8);
    uint8_t *scales = p.scales[t.kv] + row * GR;
    uint32_t mine = 0;
#pragma unroll
    for (int u = 0; u < kQ4Unroll; ++u) {
        if (u >= t.n) break;  // no lane group has a row u
        const int i = half * kQ4Unroll + u;
        uint32_t byte;
        uint4 held;
        const uint32_t w = q4_quantise8<kHeld>(x[u], byte, held);
        // The row's scale bytes gathered in one word, kept by lane u of the row's lanes.
        uint32_t s = byte << (8 * (sub / 4));
        s |= __shfl_xor_sync(FULL, s, 4);
        if (GR == 4) s |= __shfl_xor_sync(FULL, s, 8);
        if (sub == u) mine = s;
        if (i < t.n) {
            codes[static_cast<int64_t>(i) * LPR + sub] = w;
            if (kHeld)
                *(reinterpret_cast<uint4 *>(p.dst[t.kv] + p.dst_off[t.z] + t.h * p.dst_head +
                                            static_cast<int64_t>(t.tok0 + i) * p.dst_tok) + sub) = held;
        }
    }
    const int i = half * kQ4Unroll + sub;
    if (sub < kQ4Unroll && i < t.n) {
        if (GR == 4) reinterpret_cast<uint32_t *>(scales)[i] = mine;
        else reinterpret_cast<uint16_t *>(scales)[i] = static_cast<uint16_t>(mine);
    }
}

template <int D>
__global__ void __launch_bounds__(256) q4_dequantise_kernel(const __grid_constant__ Q4RowsParams p) {
    constexpr int LPR = D / 8;
    constexpr int GR = D / kQ4Group;
    const Q4Task t = q4_task<D>(p);
    if (t.n <= 0) return;
    const int lane = threadIdx.x & 31, sub = lane % LPR, half = lane / LPR;
    const int64_t row = static_cast<int64_t>(p.seq0 + t.z) * p.row_seq + t.h * p.row_head +
                        p.start[t.z] + t.tok0;
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(p.codes[t.kv]) + row * (D / 8);
    const uint8_t *scales = p.scales[t.kv] + row * GR;
    __nv_bfloat16 *dst = p.dst[t.kv] + p.dst_off[t.z] + t.h * p.dst_head;
    uint32_t w[kQ4Unroll], s[kQ4Unroll];
#pragma unroll
    for (int u = 0; u < kQ4Unroll; ++u) {
        const int i = half * kQ4Unroll + u;
        w[u] = s[u] = 0;
        if (i < t.n) {
            w[u] = codes[static_cast<int64_t>(i) * LPR + sub];
            s[u] = scales[i * GR + sub / 4];
        }
    }
#pragma unroll
    for (int u = 0; u < kQ4Unroll; ++u) {
        const int i = half * kQ4Unroll + u;
        if (i < t.n)
            *(reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(t.tok0 + i) * p.dst_tok) + sub) =
                q4_values8(w[u], s[u]);
    }
}

static bool q4_rows_grid(const Q4RowsParams &p, unsigned &blocks) {
    const int64_t warps = static_cast<int64_t>(p.nblocks) * p.Hkv * p.kv_count;
    const int64_t n = (warps + 7) / 8;
    blocks = static_cast<unsigned>(n);
    return n > 0 && n <= 0x7fffffff;
}

cudaError_t launch_q4_quantise(const Q4RowsParams &p, int D, cudaStream_t stream) {
    if (p.nblocks <= 0) return cudaSuccess;
    unsigned blocks;
    if (!q4_rows_grid(p, blocks)) return cudaErrorInvalidConfiguration;
    if (D == 128) {
        if (p.dst[0]) q4_quantise_kernel<128, true><<<blocks, 256, 0, stream>>>(p);
        else q4_quantise_kernel<128, false><<<blocks, 256, 0, stream>>>(p);
    } else {
        if (p.dst[0]) q4_quantise_kernel<64, true><<<blocks, 256, 0, stream>>>(p);
        else q4_quantise_kernel<64, false><<<blocks, 256, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t launch_q4_dequantise(const Q4RowsParams &p, int D, cudaStream_t stream) {
    if (p.nblocks <= 0) return cudaSuccess;
    unsigned blocks;
    if (!q4_rows_grid(p, blocks)) return cudaErrorInvalidConfiguration;
    if (D == 128) q4_dequantise_kernel<128><<<blocks, 256, 0, stream>>>(p);
    else q4_dequantise_kernel<64><<<blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace qa
