// k8_q8_select.cu -- K8: the blocks of the 8-bit cache that a decode step attends to.
//
// A block keeps the least and the largest code of each dim of its keys (lo, hi).
// With c the group's queries as integers in -127..127 (one scale for the group),
//   score_j = s_j sum over heads and dims of max(c lo_j, c hi_j)
//           = s_j sum over dims of (C+ hi_j + C- lo_j),
// C+ and C- the sums over the heads of c's positive and negative parts: what the
// group's products with the block's keys can come to at most ("Quest: Query-Aware
// Sparsity for Efficient Long-Context LLM Inference", Tang et al., 2024, has such
// bounds for each head).  All sums are of integers and below 2^24, so the one
// rounding is that of the product with s_j, and the choice does not depend on the
// order of anything.
//
// Bound by the bounds' bytes, 2 D a block and kv head (1/64 of its codes): 16 lanes
// (D = 128) take a block, 16 bytes each, in 8 two-way integer dot products.  The
// blocks of a kv head are shared out over a cluster; its first CTA gathers the scores
// in shared memory and finds the n-th largest by halving the range of their bits.
#include <algorithm>
#include <atomic>

#include "q8_step.cuh"

namespace qa {

constexpr int kQ8SelectThreads = 256;

// Scores as unsigned integers in their order (NaN does not occur).
__device__ __forceinline__ uint32_t q8_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // (-0 is 0)
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int D>
struct alignas(16) Q8SelectSmem {
    __nv_bfloat16 q[8][D];
    short up[D], down[D];           // C+, C-
    uint32_t top[kQ8SelectThreads / 32];
    int part[2][kQ8SelectThreads / 32];
};

// Sum of x over the block's threads; `turn` alternates between calls.
__device__ __forceinline__ int q8_block_sum(int x, int (&part)[2][kQ8SelectThreads / 32], int turn) {
    x = __reduce_add_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = x;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kQ8SelectThreads / 32; ++w) sum += part[turn][w];
    return sum;
}

template <int D>
__global__ void __launch_bounds__(kQ8SelectThreads) q8_select_kernel(const __grid_constant__ Q8StepParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const unsigned FULL = 0xffffffffu;
    extern __shared__ uint32_t keys[];       // of every complete block, in the cluster's first CTA
    __shared__ Q8SelectSmem<D> sm;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int C = p.cluster, rank = blockIdx.x, h = blockIdx.y, b = p.b0 + blockIdx.z;
    const int64_t sh = static_cast<int64_t>(b) * p.layer.Hkv + h;
    griddep_wait();
    griddep_launch_dependents();
    const int pos = q8_position(p, blockIdx.z, kKernQ8Select);
    const int full = pos < 0 ? 0 : pos / kQ8Block;
    int32_t *list = p.blocks + sh * p.n_blocks;
    if (full <= p.n_blocks) {  // all of them (no scores)
        if (rank == 0)
            for (int i = threadIdx.x; i < p.n_blocks; i += kQ8SelectThreads) list[i] = i < full ? i : -1;
        return;
    }
    if (C > 1) cluster_arrive();  // peers may write into this CTA once they have waited on this

    // ---------------------------------------------------------------- the queries' integers
    uint32_t mx = 0;
    if (warp * RPW < 8) {
        const int r = warp * RPW + lane / LPR, sub = lane % LPR;
        const uint4 x = q8_step_row<D>(p, b, h, r, pos, sub);
        *reinterpret_cast<uint4 *>(&sm.q[r][8 * sub]) = x;
        mx = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
        mx = __reduce_max_sync(FULL, max(mx & 0xffffu, mx >> 16));
    }
    if (lane == 0) sm.top[warp] = mx;
    __syncthreads();
    for (int w = 0; w < kQ8SelectThreads / 32; ++w) mx = max(mx, sm.top[w]);
    const float a = __uint_as_float(mx << 16);
    const float inv = mx < 0x7F80u && a >= kQ8Small ? __fdiv_rn(127.f, a) : 0.f;
    if (threadIdx.x < D / 2) {
        int up[2] = {0, 0}, down[2] = {0, 0};
        if (inv > 0.f) {
            for (int r = 0; r < p.G; ++r) {
                const uint32_t c = q8_code2(*reinterpret_cast<const uint32_t *>(&sm.q[r][2 * threadIdx.x]), inv);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int n = static_cast<int>((c >> (8 * e)) & 255u) - 128;
                    up[e] += max(n, 0);
                    down[e] += min(n, 0);
                }
            }
        }
        *reinterpret_cast<short2 *>(&sm.up[2 * threadIdx.x]) = make_short2(up[0], up[1]);
        *reinterpret_cast<short2 *>(&sm.down[2 * threadIdx.x]) = make_short2(down[0], down[1]);
    }
    __syncthreads();
    if (C > 1) cluster_wait();

    // ---------------------------------------------------------------- scores
    // A lane holds 16 codes of a block's 2 D: lo's in the first half of its lanes, hi's in the other.
    constexpr int LPB = D / 8, BPW = 32 / LPB, U = 4;  // lanes a block, blocks a warp, loads ahead
    {
        const int sub = lane % LPB, d0 = sub % (D / 16) * 16;
        const uint4 *w4 = reinterpret_cast<const uint4 *>(sub < D / 16 ? &sm.down[d0] : &sm.up[d0]);
        const uint4 wa = w4[0], wb = w4[1];
        const int per = (full + C - 1) / C, lo = rank * per, hi = min(full, lo + per);
        const int8_t *bounds = p.layer.bounds + sh * p.layer.nblk * (2 * D) + sub * 16;
        const float2 *scales = p.layer.scales + sh * p.layer.nblk;
        const uint32_t to = C > 1 ? map_rank(smem_u32(keys), 0) : smem_u32(keys);
        for (int j0 = lo + warp * BPW; j0 < hi; j0 += U * BPW * (kQ8SelectThreads / 32)) {
            uint4 x[U];
            float s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + u * BPW * (kQ8SelectThreads / 32) + lane / LPB;
                x[u] = make_uint4(0, 0, 0, 0);
                s[u] = 0.f;
                if (j < hi) {
                    x[u] = __ldg(reinterpret_cast<const uint4 *>(bounds + static_cast<int64_t>(j) * (2 * D)));
                    s[u] = __ldg(&scales[j].x);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + u * BPW * (kQ8SelectThreads / 32) + lane / LPB;
                int dot = 0;
                dot = __dp2a_lo(static_cast<int>(wa.x), static_cast<int>(x[u].x), dot);
                dot = __dp2a_hi(static_cast<int>(wa.y), static_cast<int>(x[u].x), dot);
                dot = __dp2a_lo(static_cast<int>(wa.z), static_cast<int>(x[u].y), dot);
                dot = __dp2a_hi(static_cast<int>(wa.w), static_cast<int>(x[u].y), dot);
                dot = __dp2a_lo(static_cast<int>(wb.x), static_cast<int>(x[u].z), dot);
                dot = __dp2a_hi(static_cast<int>(wb.y), static_cast<int>(x[u].z), dot);
                dot = __dp2a_lo(static_cast<int>(wb.z), static_cast<int>(x[u].w), dot);
                dot = __dp2a_hi(static_cast<int>(wb.w), static_cast<int>(x[u].w), dot);
#pragma unroll
                for (int o = LPB / 2; o >= 1; o >>= 1) dot += __shfl_xor_sync(FULL, dot, o);
                if (sub == 0 && j < hi) {
                    float score = __fmul_rn(static_cast<float>(dot), s[u]);
                    if (j == 0 || j == full - 1 || s[u] != s[u]) score = INFINITY;
                    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + 4 * j), "r"(q8_key(score)) : "memory");
                }
            }
        }
    }
    if (C > 1) cluster_sync_all(); else __syncthreads();
    if (rank != 0) return;  // (nobody writes into this CTA's shared memory)

    // ---------------------------------------------------------------- the n-th largest
    // Built from its highest bit: a bit stays when at least n keys reach the value with it.
    const int n = p.n_blocks;
    constexpr int R = 8;  // keys of a thread in registers; the others are read again
    uint32_t mine[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int j = threadIdx.x + i * kQ8SelectThreads;
        mine[i] = j < full ? keys[j] : 0u;  // (0 is below every score's key)
    }
    auto count = [&](uint32_t least) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) c += mine[i] >= least;
        for (int j = threadIdx.x + R * kQ8SelectThreads; j < full; j += kQ8SelectThreads) c += keys[j] >= least;
        return c;
    };
    uint32_t nth = 0;
    int reach = full, turn = 0;  // keys that are at least nth
    for (int bit = 31; bit >= 0 && reach != n; --bit, turn ^= 1) {
        const uint32_t with = nth | (1u << bit);
        const int c = q8_block_sum(count(with), sm.part, turn);
        if (c >= n) {
            nth = with;
            reach = c;
        }
    }
    // All above it, and of those that equal it the first ones: in order, a run of
    // blocks for each thread.
    int equal_take = 1 << 30;
    if (reach != n) {
        const int above = q8_block_sum(nth == 0xffffffffu ? 0 : count(nth + 1u), sm.part, turn);
        turn ^= 1;
        equal_take = n - above;
    }
    const int run = (full + kQ8SelectThreads - 1) / kQ8SelectThreads;
    const int j_lo = min(full, static_cast<int>(threadIdx.x) * run), j_hi = min(full, j_lo + run);
    int above = 0, equal = 0;
    for (int j = j_lo; j < j_hi; ++j) {
        above += keys[j] > nth;
        equal += keys[j] == nth;
    }
    // Exclusive sums over the threads of both counts (each at most 2^14).
    int both = above << 16 | equal, before = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) sm.part[turn][warp] = before;
    __syncthreads();
    before -= both;
    for (int w = 0; w < warp; ++w) before += sm.part[turn][w];
    int equals = before & 0xffff, at = (before >> 16) + min(equals, equal_take);
    for (int j = j_lo; j < j_hi; ++j) {
        const uint32_t key = keys[j];
        if (key > nth || (key == nth && equals < equal_take)) list[at++] = j;
        equals += key == nth;
    }
}

// ------------------------------------------------------------------ launch
template <int D>
static cudaError_t q8_launch_select(const Q8StepParams &p, int batch, cudaStream_t stream) {
    static std::atomic<unsigned> configured{0u};  // devices 0..31 set up (one bit each)
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 32 || !((configured.load(std::memory_order_acquire) >> dev) & 1u)) {
        const cudaError_t e = cudaFuncSetAttribute(q8_select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kQ8MaxBlocks * sizeof(uint32_t));
        if (e != cudaSuccess) return e;
        if (dev < 32) configured.fetch_or(1u << dev, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.cluster, p.layer.Hkv, batch);
    cfg.blockDim = dim3(kQ8SelectThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.layer.nblk) * sizeof(uint32_t);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, q8_select_kernel<D>, p);
}

cudaError_t launch_q8_select(const Q8StepParams &p, int D, int batch, cudaStream_t stream) {
    return D == 128 ? q8_launch_select<128>(p, batch, stream) : q8_launch_select<64>(p, batch, stream);
}

}  // namespace qa
