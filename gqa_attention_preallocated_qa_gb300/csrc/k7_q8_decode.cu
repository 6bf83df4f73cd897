// k7_q8_decode.cu -- K7: one decode step over the 8-bit cache, dense or sparse.
//
// For each sequence and query head, with q' the normed and rotated query and
// n_j, s the codes and scale of a block's keys (likewise of its values):
//   t_j = log2(e) / sqrt(D) * s * (q' . n_j),  out = sum_j 2^t_j V_j / sum_j 2^t_j
// over the complete blocks (or the chosen ones of them), and over the bf16 rows of
// the block that the new token is in, itself among them.
//
// Bound by the bytes of the codes: a block of K and V is 16 KB (D = 128), and
// each is read once, by one warp, straight into the registers that feed the MMAs
// (the codes lie in fragment order): no shared memory, no barrier between warps.
// A warp loads the next block's K while it computes with V, and its V after, so
// that 8 to 16 KB a warp are on the way.
//   Keys are the M side (S^T = K q'^T, O^T += V^T P^T, m16n8k16, N = the group's
// up to 8 heads).  A code becomes fp16 by half a byte permute: n + 128 as the
// subnormal (n + 128) 2^-24.  The offset is taken away by the accumulators' start:
// -128 2^-24 sum q' for S, and for O -128 2^-24 sum_j p_j, which one more MMA (the
// constant times P) gives in every lane of a column, together with the sum of the
// weights as they were rounded to fp16.  Scales multiply the block's sums: one FMA
// per accumulator and 64 keys.
//   The running maximum lags: weights are 2^(t - ref), and ref moves only when one would
// pass 2^15, which fp16 still holds, to where the largest is 2^7.  So a warp's largest
// weight is 2^7 at least, and what fp16 cannot hold of another is below 2^-32 of it
// (a step of its smallest numbers is 2^-24).  Outputs are summed 2^32 times too small, so
// that 2^17 keys of the largest bf16 numbers stay in range.
//   S CTAs (a power of two) of a cluster share a (sequence, kv head); each sends its
// sums to the CTAs that finish them, through distributed shared memory.
//
// A sparse step first chooses its blocks.  A block keeps the least and the largest
// code of each dim of its keys (lo, hi).  With c the group's queries as integers in
// -127..127 (one scale for the group),
//   score_j = s_j sum over heads and dims of max(c lo_j, c hi_j)
//           = s_j sum over dims of (C+ hi_j + C- lo_j),
// C+ and C- the sums over the heads of c's positive and negative parts: what the
// group's products with the block's keys can come to at most ("Quest: Query-Aware
// Sparsity for Efficient Long-Context LLM Inference", Tang et al., 2024, has such
// bounds for each head).  All sums are of integers and below 2^24, so the one
// rounding is that of the product with s_j, and the choice does not depend on the
// order of anything.  The bounds are 2 D bytes a block and kv head (1/64 of its
// codes): 16 lanes (D = 128) take a block, in 8 two-way integer dot products each.
// Every CTA of a (sequence, kv head) scores a share, sends the scores to the others,
// and finds the n-th largest for itself.
#include <algorithm>
#include <atomic>

#include "norm_rope.cuh"
#include "q8_device.cuh"

namespace qa {

constexpr int kQ8Warps = 4, kQ8Threads = kQ8Warps * 32;
constexpr float kQ8NoRef = -3e38f;   // no key yet
constexpr float kQ8Lift = 7.f;       // the largest weight's exponent where ref is set,
constexpr float kQ8Most = 15.f;      // and the one that it may grow to

// A (16x16 fp16) * B (16x8 fp16), fp32 accumulators.
__device__ __forceinline__ void q8_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void q8_mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8x8 matrix of 16-bit values, a row on four lanes.
__device__ __forceinline__ uint32_t q8_transpose(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t q8_pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float q8_exp2(float x) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Codes are read once per step: past L1.  (volatile: loads stay where they are issued.)
__device__ __forceinline__ uint4 q8_load(const uint8_t *p) {
    uint4 x;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "l"(p));
    return x;
}
// Four bytes into the shared memory of a CTA of the cluster, counted on an mbarrier there.
__device__ __forceinline__ void q8_send(uint32_t addr, uint32_t x, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(addr), "r"(x), "r"(bar)
                 : "memory");
}

// Sums of a warp: columns (heads) 2 t and 2 t + 1 of the MMAs (t = lane % 4); o[m] holds
// dims (D / 8) g + 2 m and + 1 of both heads, 2^32 times too small.
template <int D>
struct Q8Acc {
    float ref[2], l[2];
    float o[D / 16][4];
};

template <int D>
__device__ __forceinline__ void q8_raise(Q8Acc<D> &a, float m0, float m1) {
    // m0, m1: this lane's largest scores of its two heads
    const unsigned FULL = 0xffffffffu;
    // (The differences are the weights' exponents, and exact for scores of any size; a sum with
    // the limit is not, and from 2^24 on would let a weight pass fp16's largest number.)
    if (!__any_sync(FULL, m0 - a.ref[0] > kQ8Most || m1 - a.ref[1] > kQ8Most)) return;
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(FULL, m0, o));
        m1 = fmaxf(m1, __shfl_xor_sync(FULL, m1, o));
    }
    const float r0 = m0 - a.ref[0] > kQ8Most ? m0 - kQ8Lift : a.ref[0], r1 = m1 - a.ref[1] > kQ8Most ? m1 - kQ8Lift : a.ref[1];
    const float f0 = q8_exp2(a.ref[0] - r0), f1 = q8_exp2(a.ref[1] - r1);
    a.ref[0] = r0;
    a.ref[1] = r1;
    a.l[0] *= f0;
    a.l[1] *= f1;
#pragma unroll
    for (int m = 0; m < D / 16; ++m) {
        a.o[m][0] *= f0;
        a.o[m][1] *= f1;
        a.o[m][2] *= f0;
        a.o[m][3] *= f1;
    }
}

// Scores as unsigned integers in their order (NaN does not occur).
__device__ __forceinline__ uint32_t q8_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // (-0 is 0)
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int D>
struct alignas(16) Q8StepSmem {
    __half qh[8][D + 8];            // queries, each row times a power of two
    __nv_bfloat16 qb[8][D + 8];     // queries as they are
    float qscale[8], qstart[8];     // log2(e) / sqrt(D) over that power; what S starts from
    __nv_bfloat16 rows[2][kQ8Block][D + 8];   // K and V of the block that the new token is in
    float o[kQ8Warps][8][D + 8];    // a warp's sums; slot 16 m + 2 g + e of a head's row: dim (D / 8) g + 2 m + e
    union {
        alignas(16) uint32_t hist[4][256];   // a sparse step's, for its choice
        Q8SealSmem<D> seal;               // at its end
    };
    float ref[kQ8Warps][8], l[kQ8Warps][8];
    // From the CTAs of the (sequence, kv head): references and sums of weights (of a
    // head), and this CTA's share of the outputs.
    float2 got_l[kQ8MaxSplits][8];
    float got_o[8 * D];
    // A sparse step's
    uint32_t top[kQ8Warps];
    alignas(16) short up[D], down[D];             // C+, C-
    alignas(16) uint32_t part[kQ8Warps][4];
    uint32_t runs[32];
    // Transactions of what the other CTAs send: sums, scores.
    alignas(8) uint64_t bar[2];
    int abort;
};

// Waits for the sums of the others.  A CTA that has given up waiting, for these or for the
// scores, stays as long again: what a late one still sends may not find it gone.  (One
// that missed scores sends no sums, so nothing is sent later than that.)
__device__ __noinline__ void q8_wait_sums(uint32_t bar, volatile int *abort, uint32_t *err, uint64_t wait_ns) {
    if (mbar_wait_cluster(bar, 0, abort, err, kKernQ8Decode, 3, wait_ns)) return;
    int alone = 0;
    mbar_wait_cluster(bar, 0, &alone, err, kKernQ8Decode, 4, wait_ns);
}

template <int D>
__device__ __forceinline__ int q8_slot(int d) {
    const int g = d / (D / 8), r = d % (D / 8);
    return (r >> 1) * 16 + 2 * g + (r & 1);
}

// The bounds of a batch of blocks of this CTA's share, 16 bytes a lane: lo's in the first
// half of a block's lanes, hi's in the other.  Eight loads a lane; the sum over a block's
// lanes leaves block kMine of the eight in the lane, whose scale it has.
template <int D>
struct Q8Bounds {
    static constexpr int kLanes = D / 8, kPer = 32 / kLanes, kAhead = 8;  // lanes a block, blocks a warp and load, loads
    static constexpr int kBatch = kAhead * kPer * kQ8Warps;
    static constexpr int kSame = kLanes / kAhead;  // lanes with the same block of the eight
    uint4 x[kAhead];
    float s;

    __device__ __forceinline__ static int block(int first, int u) {
        return first + ((u * kQ8Warps + (threadIdx.x >> 5)) * kPer) + (threadIdx.x & 31) / kLanes;
    }
    __device__ __forceinline__ static int mine(int first) { return block(first, threadIdx.x % kLanes / kSame); }
    // Of blocks first .. first + kBatch - 1, below hi.
    __device__ __forceinline__ void load(const Q8Layer &l, int64_t base, int first, int hi) {
        const int8_t *bounds = l.bounds + base * (2 * D) + (threadIdx.x % kLanes) * 16;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int j = block(first, u);
            x[u] = make_uint4(0, 0, 0, 0);
            if (j < hi) x[u] = *reinterpret_cast<const uint4 *>(bounds + static_cast<int64_t>(j) * (2 * D));
        }
        s = mine(first) < hi ? l.scales[base + mine(first)].x : 0.f;
    }
};

// Scores blocks lo .. hi - 1 and sends them to keys[] of all S CTAs (to none: withhold); at:
// their first two batches, both on the way before the queries are normed.  (That, one shuffle
// a block instead of four and one barrier a round of the choice: B 4, 60 to 65 thousand
// positions, 64 blocks 12.65 -> 11.2 us; B 8, 32768 positions 15.3 -> 13.5.)
template <int D>
__device__ __forceinline__ void q8_score(const Q8Layer &l, int64_t base, int full, int lo, int hi, int S,
                                         uint32_t first_rank, bool withhold, Q8StepSmem<D> &sm, uint32_t *keys,
                                         Q8Bounds<D> (&at)[2]) {
    using B = Q8Bounds<D>;
    constexpr int LPB = B::kLanes;
    const int sub = threadIdx.x % LPB, d0 = sub % (D / 16) * 16;
    const uint4 *w4 = reinterpret_cast<const uint4 *>(sub < D / 16 ? &sm.down[d0] : &sm.up[d0]);
    const uint4 wa = w4[0], wb = w4[1];
    const uint32_t to = smem_u32(keys), bar = smem_u32(&sm.bar[1]);
    auto batch = [&](int first, B &in) {
        int dot[B::kAhead];
        const float s = in.s;
#pragma unroll
        for (int u = 0; u < B::kAhead; ++u) {
            const uint4 x = in.x[u];
            dot[u] = __dp2a_lo(static_cast<int>(wa.x), static_cast<int>(x.x), 0);
            dot[u] = __dp2a_hi(static_cast<int>(wa.y), static_cast<int>(x.x), dot[u]);
            dot[u] = __dp2a_lo(static_cast<int>(wa.z), static_cast<int>(x.y), dot[u]);
            dot[u] = __dp2a_hi(static_cast<int>(wa.w), static_cast<int>(x.y), dot[u]);
            dot[u] = __dp2a_lo(static_cast<int>(wb.x), static_cast<int>(x.z), dot[u]);
            dot[u] = __dp2a_hi(static_cast<int>(wb.y), static_cast<int>(x.z), dot[u]);
            dot[u] = __dp2a_lo(static_cast<int>(wb.z), static_cast<int>(x.w), dot[u]);
            dot[u] = __dp2a_hi(static_cast<int>(wb.w), static_cast<int>(x.w), dot[u]);
        }
        if (first + 2 * B::kBatch < hi) in.load(l, base, first + 2 * B::kBatch, hi);
        // Half of the sums go to the lane across, half of its come here.
#pragma unroll
        for (int n = B::kAhead / 2, o = LPB / 2; n >= 1; n /= 2, o /= 2) {
            const bool upper = (sub & o) != 0;
#pragma unroll
            for (int u = 0; u < n; ++u) {
                const int keep = upper ? dot[u + n] : dot[u], give = upper ? dot[u] : dot[u + n];
                dot[u] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        }
        if (B::kSame == 2) dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], 1);
        const int j = B::mine(first);
        if (j >= hi) return;
        float score = __fmul_rn(static_cast<float>(dot[0]), s);
        if (j == 0 || j == full - 1 || s != s) score = INFINITY;
        const uint32_t key = q8_key(score);
        if (S == 1) {
            if (sub % B::kSame == 0) keys[j] = key;
        } else if (!withhold) {
            for (int r = sub % B::kSame; r < S; r += B::kSame)
                q8_send(map_rank(to + 4 * j, first_rank + r), key, map_rank(bar, first_rank + r));
        }
    };
    for (int j0 = lo; j0 < hi; j0 += 2 * B::kBatch) {
        batch(j0, at[0]);
        if (j0 + B::kBatch < hi) batch(j0 + B::kBatch, at[1]);
    }
}

// The n blocks of the largest of keys[0 .. full - 1] (full > n), in rising order: those at
// places lo .. hi - 1 go to list[].
//   The n-th largest key is found by counting keys in 256 equal steps of the range that
// holds it, which then shrinks to one step: two or three times for scores as they come,
// four at most, each time in counters of its own and found by every warp for itself, for
// one barrier.  Infinite ones are set apart, so that the first range is that of numbers.
template <int D>
__device__ __forceinline__ void q8_select(const uint32_t *keys, int full, int n, int lo, int hi, Q8StepSmem<D> &sm,
                                          uint16_t *list) {
    const unsigned FULL = 0xffffffffu;
    constexpr uint32_t kInf = 0xff800000u;  // q8_key(INFINITY)
    constexpr int R = 8, kHeld = R * kQ8Threads;  // keys of a thread in registers: the first of all
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t mine[R];
    auto take_keys = [&](int first) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int j = first + i * kQ8Threads + threadIdx.x;
            mine[i] = j < full ? keys[j] : 0u;  // (0 is below every score's key)
        }
    };
    auto each = [&](auto &&f) {
#pragma unroll
        for (int i = 0; i < R; ++i) f(mine[i]);
        for (int j = kHeld + threadIdx.x; j < full; j += kQ8Threads) f(keys[j]);
    };
    take_keys(0);
    uint32_t least = kInf, most = 0, infinite = 0;
    each([&](uint32_t key) {
        infinite += key >= kInf;
        least = min(least, key == 0u ? kInf : key);
        most = max(most, key >= kInf ? 0u : key);
    });
    least = __reduce_min_sync(FULL, least);
    most = __reduce_max_sync(FULL, most);
    infinite = __reduce_add_sync(FULL, infinite);
    if (lane == 0) *reinterpret_cast<uint4 *>(sm.part[warp]) = make_uint4(least, most, infinite, 0);
    for (int i = threadIdx.x; i < 256; i += kQ8Threads) reinterpret_cast<uint4 *>(sm.hist[0])[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    infinite = 0;
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) {
        const uint4 x = *reinterpret_cast<const uint4 *>(sm.part[w]);
        least = min(least, x.x);
        most = max(most, x.y);
        infinite += x.z;
    }
    // All keys above nth belong to them, and the first `take` of those that equal it.
    uint32_t nth = kInf;
    int need = n - static_cast<int>(infinite), take = n;
    for (uint32_t *hist = sm.hist[0]; need > 0; hist += 256) {
        const int shift = max(0, 24 - __clz(most - least));  // (most - least) >> shift is below 256
        each([&](uint32_t key) {
            if (key >= least && key <= most) atomicAdd(&hist[(key - least) >> shift], 1u);
        });
        __syncthreads();
        // A lane has 8 steps, the last lane the largest.
        const uint4 a = *reinterpret_cast<const uint4 *>(&hist[8 * lane]), b = *reinterpret_cast<const uint4 *>(&hist[8 * lane + 4]);
        const int c[8] = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w),
                          static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w)};
        const int all = c[0] + c[1] + c[2] + c[3] + c[4] + c[5] + c[6] + c[7];
        int from = all;  // keys in this lane's steps and higher ones
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_down_sync(FULL, from, o);
            if (lane + o < 32) from += y;
        }
        // The n-th largest is in the steps of one lane: its step, the keys above, those in it.
        int above = from - all, at = 0, in = 0;
        const int src = __ffs(__ballot_sync(FULL, above < need && from >= need)) - 1;
        bool found = false;
#pragma unroll
        for (int step = 7; step >= 0; --step) {
            if (!found && above + c[step] >= need) {
                found = true;
                at = 8 * lane + step;
                in = c[step];
            }
            if (!found) above += c[step];
        }
        at = __shfl_sync(FULL, at, src);
        above = __shfl_sync(FULL, above, src);
        in = __shfl_sync(FULL, in, src);
        least += static_cast<uint32_t>(at) << shift;
        need -= above;
        if (need == in || shift == 0) {  // all keys of the step, or equal ones
            nth = need == in ? least - 1 : least;
            take = need == in ? 0 : need;
            break;
        }
        most = min(most, least + ((1u << shift) - 1u));
    }
    // In order, kHeld blocks at a time: a warp has 32 of them for each of its registers.
    int above_before = 0, equal_before = 0;
    const uint32_t below = (1u << lane) - 1u;
    for (int first = 0; first < full; first += kHeld) {
        if (first > 0) take_keys(first);
        uint32_t above[R], equal[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            above[i] = __ballot_sync(FULL, mine[i] > nth);
            equal[i] = __ballot_sync(FULL, mine[i] == nth);
            if (lane == 0) sm.runs[i * kQ8Warps + warp] = __popc(above[i]) | __popc(equal[i]) << 16;
        }
        __syncthreads();
        uint32_t run = sm.runs[lane], upto = run;  // R * kQ8Warps = 32 of them
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(FULL, upto, o);
            if (lane >= o) upto += y;
        }
        const uint32_t total = __shfl_sync(FULL, upto, 31);
        upto -= run;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint32_t runs = __shfl_sync(FULL, upto, i * kQ8Warps + warp);
            const int equals = equal_before + static_cast<int>(runs >> 16) + __popc(equal[i] & below);
            const int at = above_before + static_cast<int>(runs & 0xffff) + __popc(above[i] & below) + min(equals, take);
            if ((mine[i] > nth || (mine[i] == nth && equals < take)) && at >= lo && at < hi)
                list[at - lo] = static_cast<uint16_t>(first + i * kQ8Threads + threadIdx.x);
        }
        above_before += total & 0xffff;
        equal_before += total >> 16;
        __syncthreads();
    }
}

template <int D, bool kSparse>
__global__ void __launch_bounds__(kQ8Threads, 2) q8_decode_kernel(const __grid_constant__ Q8StepParams p) {
    constexpr int NV = D / 8;   // 16-byte vectors of a lane for K, and for V, of a block
    constexpr int NB = 128 / D; // blocks that a warp has in hand: independent chains at D = 64
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const unsigned FULL = 0xffffffffu;
    extern __shared__ uint4 smem[];
    Q8StepSmem<D> &sm = *reinterpret_cast<Q8StepSmem<D> *>(smem);
    // Sparse: the scores of every block (n_scores); behind them the chosen blocks of this CTA.
    uint32_t *keys = reinterpret_cast<uint32_t *>(&sm + 1);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;

    // ---------------------------------------------------------------- this CTA's share
    // An early launch signals at once, reads and computes beside its predecessors, which
    // write nothing that it reads, and waits for them before it writes.
    if (!p.early) griddep_wait();
    griddep_launch_dependents();
    int z = 0, pos = -1;
    if (static_cast<int>(blockIdx.x) < p.ctas) {
        if (p.per_seq > 0) {
            z = blockIdx.x / static_cast<uint32_t>(p.per_seq);
        } else {
            int hi = p.nseq;  // seq[z].cta0 <= blockIdx.x < seq[hi].cta0
            while (hi - z > 1) {
                const int mid = (z + hi) / 2;
                if (p.seq[mid].cta0 <= static_cast<int>(blockIdx.x)) z = mid; else hi = mid;
            }
        }
        pos = p.pos_dev ? p.pos_dev[p.seq[z].slot] : p.seq[z].pos;
        if (pos < 0 || pos >= p.cap) {
            if (threadIdx.x == 0) set_error(p.err, kErrBounds, kKernQ8Decode, 1);
            pos = -1;
        }
    }
    const int b = p.seq[z].slot, log_S = p.seq[z].log_S, S = 1 << log_S;
    const int unit = static_cast<int>(blockIdx.x) - p.seq[z].cta0, me = unit & (S - 1), h = unit >> log_S;
    __syncwarp();  // (thread 0 may have been setting the error: the cluster's barriers want whole warps)
    if (pos < 0) {  // nothing to do here
        if (p.cluster > 1) cluster_arrive();
        griddep_wait();
        if (kSparse && me == 0 && static_cast<int>(blockIdx.x) < p.ctas) {
            for (int i = threadIdx.x; i < p.n_blocks; i += kQ8Threads)
                p.blocks[(static_cast<int64_t>(b) * p.layer.Hkv + h) * p.n_blocks + i] = -1;
        }
        __syncwarp();
        if (p.cluster > 1) cluster_wait();
        return;
    }
    const uint32_t first_rank = cluster_ctarank() - me;
    const int64_t sh = static_cast<int64_t>(b) * p.layer.Hkv + h, base = sh * p.layer.nblk;
    const int full = static_cast<uint32_t>(pos) / kQ8Block, row = static_cast<uint32_t>(pos) % kQ8Block;
    const bool choose = kSparse && full > p.n_blocks;
    bool listed = true;  // (false: a wait ran out)
    const bool withhold = p.fault != 0 && z == 0 && unit == S - 1;  // (test hook)
    const int items = choose ? p.n_blocks : full;
    const int item_lo = items * me >> log_S, item_hi = items * (me + 1) >> log_S;  // (at most 2^18)
    int item = item_lo + warp;
    uint16_t *list = reinterpret_cast<uint16_t *>(keys + p.n_scores);
    const uint8_t *codes = p.layer.codes + base * (2 * kQ8Block * D) + lane * 16;
    uint4 k[NB][NV], v[NB][NV];
    float2 scale[NB];
    int blk[NB];
    // The next blocks of the warp, -1 where there is none.
    auto next_blocks = [&](int (&j)[NB]) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            j[n] = item >= item_hi ? -1 : choose ? static_cast<int>(list[item - item_lo]) : item;
            item += kQ8Warps;
        }
    };
    auto load_k = [&](const int (&j)[NB]) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            if (j[n] < 0) continue;
            const uint8_t *c = codes + static_cast<int64_t>(j[n]) * (2 * kQ8Block * D);
#pragma unroll
            for (int i = 0; i < NV; ++i) k[n][i] = q8_load(c + i * 512);
            scale[n] = p.layer.scales[base + j[n]];
        }
    };
    auto load_v = [&](const int (&j)[NB]) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            if (j[n] < 0) continue;
            const uint8_t *c = codes + static_cast<int64_t>(j[n]) * (2 * kQ8Block * D) + kQ8Block * D;
#pragma unroll
            for (int i = 0; i < NV; ++i) v[n][i] = q8_load(c + i * 512);
        }
    };
    auto load_first = [&]() {
        next_blocks(blk);
        load_k(blk);
        load_v(blk);
    };
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        blk[n] = -1;
        scale[n] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) k[n][i] = v[n][i] = make_uint4(0, 0, 0, 0);
    }
    // The blocks that this CTA scores.
    const int score_lo = full * me >> log_S, score_hi = full * (me + 1) >> log_S;
    Q8Bounds<D> bounds[2];
    // What the other CTAs of the S send: sums of weights and outputs, scores.
    if (p.cluster > 1) {
        if (threadIdx.x == 0) {
            sm.abort = 0;
            mbar_init(smem_u32(&sm.bar[0]), 1);
            mbar_init(smem_u32(&sm.bar[1]), 1);
            fence_mbar_init();
            mbar_expect_tx(smem_u32(&sm.bar[0]), p.G * D * 4 + S * p.G * 8);
            if (choose) mbar_expect_tx(smem_u32(&sm.bar[1]), full * 4);
        }
        __syncwarp();
        cluster_arrive();  // peers send once they have waited on this
    }

    // ---------------------------------------------------------------- query rows, and the new token's
    // Their loads go out first, before the codes', which would hold them up.  CTA 0 of the
    // S has the rows of the block that the token is in.
    const int sub = lane % LPR, key_row = p.G < 8 ? p.G : 8;
    const bool two = p.G == 8 && kQ8Warps * RPW < 9;  // a second turn, for the key alone
    auto is_key = [&](int r) { return r == key_row && me == 0; };
    auto load_row = [&](int r, NormRow &in) {
        const bool is_q = r < p.G;
        in.x = in.w = in.v = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) in.cs[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!is_q && !is_key(r)) return;
        in.x = __ldg(reinterpret_cast<const uint4 *>(is_q ? p.q + (static_cast<int64_t>(b) * p.Hq + h * p.G + r) * D : p.k + sh * D) + sub);
        if (!is_q) in.v = __ldg(reinterpret_cast<const uint4 *>(p.v + sh * D) + sub);
        if (!p.wq) return;
        in.w = __ldg(reinterpret_cast<const uint4 *>(is_q ? p.wq : p.wk) + sub);
        const float4 *tab = reinterpret_cast<const float4 *>(p.rope + static_cast<int64_t>(pos) * (D / 2) + 8 * (sub % (D / 16)));
#pragma unroll
        for (int e = 0; e < 4; ++e) in.cs[e] = __ldg(tab + e);
    };
    NormRow in;
    load_row(warp * RPW + lane / LPR, in);
    Q8TailPlan plan;
    __nv_bfloat16 *tail = nullptr;   // where they are kept: 64 rows of K, then of V
    if (me == 0) plan.next = p.layer.state[sh];
    if (choose) {
        bounds[0].load(p.layer, base, score_lo, score_hi);
        bounds[1].load(p.layer, base, score_lo + Q8Bounds<D>::kBatch, score_hi);
    } else if (!kSparse) {
        load_first();
    }
    if (me == 0) {
        plan = q8_plan_tail(plan.next, pos, pos + 1, true);
        tail = p.layer.tail + (sh * 2 + plan.dst) * static_cast<int64_t>(2 * kQ8Block * D);
        for (int e = threadIdx.x; e < plan.from_rows * LPR; e += kQ8Threads) {
            const int r = e / LPR, d0 = e % LPR * 8;
            q8_copy16(&sm.rows[0][r][d0], tail + r * D + d0);
            q8_copy16(&sm.rows[1][r][d0], tail + (kQ8Block + r) * D + d0);
        }
    }
    uint32_t top = 0;
#pragma unroll 1
    for (int turn = 0; turn <= (two ? 1 : 0); ++turn) {  // (uniform in a warp)
        const int r = (turn * kQ8Warps + warp) * RPW + lane / LPR;
        if (turn > 0) load_row(r, in);
        uint4 x = p.wq ? norm_rope_row<D>(in, p.eps, sub) : in.x;
        if (r >= p.G && !is_key(r)) x = make_uint4(0, 0, 0, 0);
        if (is_key(r)) {
            *reinterpret_cast<uint4 *>(&sm.rows[0][row][8 * sub]) = x;
            *reinterpret_cast<uint4 *>(&sm.rows[1][row][8 * sub]) = in.v;
            x = make_uint4(0, 0, 0, 0);
        }
        // fp16 with one power of two per row: the largest magnitude goes to [256, 512),
        // so bf16's 8 bits survive down to 2^-22 of it.
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
        uint32_t mx = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = __vmaxu2(mx, xw[e] & 0x7fff7fffu);
        mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) mx = max(mx, __shfl_xor_sync(FULL, mx, o));
        top = max(top, mx);
        const int ex = min(max(static_cast<int>(mx >> 7), 20), 254) - 127;
        const float by = __uint_as_float(static_cast<uint32_t>(127 + 8 - ex) << 23);
        uint32_t hw[4];
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hw[e] = q8_pack_f16(bf16lo(xw[e]) * by, bf16hi(xw[e]) * by);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hw[e]));
            sum += f.x + f.y;
        }
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
        if (r < 8) {
            *reinterpret_cast<uint4 *>(&sm.qh[r][8 * sub]) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            *reinterpret_cast<uint4 *>(&sm.qb[r][8 * sub]) = x;
            if (sub == 0) {
                sm.qscale[r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
                sm.qstart[r] = sum * -7.62939453125e-06f;  // 128 * 2^-24
            }
        }
    }
    if (kSparse) {
        top = __reduce_max_sync(FULL, top);
        if (lane == 0) sm.top[warp] = top;
    }
    if (me == 0) {
        if (plan.from_rows < row) {  // earlier rows of the block are in its codes alone
            griddep_wait();
            const uint8_t *c = p.layer.codes + (base + full) * (2 * kQ8Block * D);
            const float2 s = p.layer.scales[base + full];
            for (int e = threadIdx.x; e < (row - plan.from_rows) * 2 * LPR; e += kQ8Threads) {
                const int kv = e / ((row - plan.from_rows) * LPR), w = e % ((row - plan.from_rows) * LPR);
                const int rr = plan.from_rows + w / LPR, d0 = w % LPR * 8;
                const uint4 x = q8_row8<D>(c + kv * kQ8Block * D, kv != 0, kv ? s.y : s.x, rr, d0);
                *reinterpret_cast<uint4 *>(&sm.rows[kv][rr][d0]) = x;
                *reinterpret_cast<uint4 *>(tail + (kv * kQ8Block + rr) * D + d0) = x;
            }
        }
    }
    __syncthreads();
    if (p.cluster > 1) cluster_wait();

    // ---------------------------------------------------------------- the choice
    if (kSparse) {
        if (choose) {
            uint32_t mx = sm.top[0];
#pragma unroll
            for (int w = 1; w < kQ8Warps; ++w) mx = max(mx, sm.top[w]);
            const float a = __uint_as_float(mx << 16);
            const float inv = mx < 0x7F80u && a >= kQ8Small ? __fdiv_rn(127.f, a) : 0.f;
            if (threadIdx.x < D / 2) {
                int up[2] = {0, 0}, down[2] = {0, 0};
                if (inv > 0.f) {
                    for (int r = 0; r < p.G; ++r) {
                        const uint32_t c = q8_code2(*reinterpret_cast<const uint32_t *>(&sm.qb[r][2 * threadIdx.x]), inv);
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
            q8_score<D>(p.layer, base, full, score_lo, score_hi, S, first_rank, withhold, sm, keys, bounds);
            const bool ok = S == 1 || mbar_wait_cluster(smem_u32(&sm.bar[1]), 0, &sm.abort, p.err, kKernQ8Decode, 2, p.wait_ns);
            if (__syncthreads_and(ok)) {
                q8_select<D>(keys, full, p.n_blocks, item_lo, item_hi, sm, list);
            } else {
                listed = false;
            }
        }
        if (listed) load_first();  // (its registers held the bounds; also where nothing was to choose)
    }

    // ---------------------------------------------------------------- complete blocks
    Q8Acc<D> a;
    a.ref[0] = a.ref[1] = kQ8NoRef;
    a.l[0] = a.l[1] = 0.f;
#pragma unroll
    for (int m = 0; m < D / 16; ++m) a.o[m][0] = a.o[m][1] = a.o[m][2] = a.o[m][3] = 0.f;
    const float qs0 = sm.qscale[2 * t], qs1 = sm.qscale[2 * t + 1];
    const float st0 = sm.qstart[2 * t], st1 = sm.qstart[2 * t + 1];
    while (blk[0] >= 0) {
        int ahead[NB];
        next_blocks(ahead);
        float s[NB][4][4];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                s[n][kt][0] = s[n][kt][2] = st0;
                s[n][kt][1] = s[n][kt][3] = st1;
            }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const uint4 q = *reinterpret_cast<const uint4 *>(&sm.qh[g][32 * c + 8 * t]);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
#pragma unroll
                for (int kt = 0; kt < 4; ++kt) {
                    const uint4 w = k[n][kt * (D / 32) + c];
                    q8_mma(s[n][kt], q8_lo(w.x), q8_hi(w.x), q8_lo(w.y), q8_hi(w.y), q.x, q.y);
                    q8_mma(s[n][kt], q8_lo(w.z), q8_hi(w.z), q8_lo(w.w), q8_hi(w.w), q.z, q.w);
                }
            }
        }
        float2 sc[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) sc[n] = blk[n] >= 0 ? scale[n] : make_float2(0.f, 0.f);
        load_k(ahead);
        float m0 = kQ8NoRef, m1 = kQ8NoRef;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            // S is 2^24 times too small, and 2^8 too large by the queries' power of two.  (The
            // 2^16 last: the scale alone may be near fp32's largest numbers.)
            const float c0 = sc[n].x * qs0 * 65536.f, c1 = sc[n].x * qs1 * 65536.f;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                s[n][kt][0] *= c0;
                s[n][kt][1] *= c1;
                s[n][kt][2] *= c0;
                s[n][kt][3] *= c1;
                if (n > 0 && blk[n] < 0) s[n][kt][0] = s[n][kt][1] = s[n][kt][2] = s[n][kt][3] = -INFINITY;
                m0 = fmaxf(m0, fmaxf(s[n][kt][0], s[n][kt][2]));
                m1 = fmaxf(m1, fmaxf(s[n][kt][1], s[n][kt][3]));
            }
        }
        q8_raise<D>(a, m0, m1);
        uint32_t pb[NB][4][2];
        float acc[NB][D / 16][4];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            float start[4] = {0.f, 0.f, 0.f, 0.f};  // -128 2^-24 times the sum of the weights
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                pb[n][kt][0] = q8_transpose(q8_pack_f16(q8_exp2(s[n][kt][0] - a.ref[0]), q8_exp2(s[n][kt][1] - a.ref[1])));
                pb[n][kt][1] = q8_transpose(q8_pack_f16(q8_exp2(s[n][kt][2] - a.ref[0]), q8_exp2(s[n][kt][3] - a.ref[1])));
                q8_mma(start, kQ8Zero, kQ8Zero, kQ8Zero, kQ8Zero, pb[n][kt][0], pb[n][kt][1]);  // 0x8080: -2^-17 in fp16
            }
            a.l[0] = fmaf(start[0], -131072.f, a.l[0]);
            a.l[1] = fmaf(start[1], -131072.f, a.l[1]);
#pragma unroll
            for (int m = 0; m < D / 16; ++m) {
                acc[n][m][0] = acc[n][m][2] = start[0];
                acc[n][m][1] = acc[n][m][3] = start[1];
            }
        }
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
#pragma unroll
            for (int n = 0; n < NB; ++n) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint4 w = v[n][kt * (D / 32) + i];
                    q8_mma(acc[n][2 * i], q8_lo(w.x), q8_hi(w.x), q8_lo(w.y), q8_hi(w.y), pb[n][kt][0], pb[n][kt][1]);
                    q8_mma(acc[n][2 * i + 1], q8_lo(w.z), q8_hi(w.z), q8_lo(w.w), q8_hi(w.w), pb[n][kt][0], pb[n][kt][1]);
                }
            }
        }
        load_v(ahead);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const float by = sc[n].y * 0.00390625f;  // (acc is 2^24 times too small)
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.o[m][e] = fmaf(acc[n][m][e], by, a.o[m][e]);
            blk[n] = ahead[n];
        }
    }

    // ---------------------------------------------------------------- rows in bf16
    // 16 of them a warp, the last warps (which have the fewest blocks) first.  Weights as
    // the sum of two bf16 numbers, 2^32 times too small.
    const int tile = kQ8Warps - 1 - warp;
    if (me == 0) {
        q8_copy_wait();
        __syncthreads();
    }
    if (me == 0 && 16 * tile <= row) {
        const int r0 = 16 * tile + g, r8 = r0 + 8;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const int d0 = 32 * c + 8 * t;
            const uint4 q = *reinterpret_cast<const uint4 *>(&sm.qb[g][d0]);
            const uint4 x = r0 <= row ? *reinterpret_cast<const uint4 *>(&sm.rows[0][r0][d0]) : zero;
            const uint4 y = r8 <= row ? *reinterpret_cast<const uint4 *>(&sm.rows[0][r8][d0]) : zero;
            q8_mma_bf16(s, x.x, y.x, x.y, y.y, q.x, q.y);
            q8_mma_bf16(s, x.z, y.z, x.w, y.w, q.z, q.w);
        }
        s[0] = r0 <= row ? s[0] * p.scale_log2 : -INFINITY;
        s[1] = r0 <= row ? s[1] * p.scale_log2 : -INFINITY;
        s[2] = r8 <= row ? s[2] * p.scale_log2 : -INFINITY;
        s[3] = r8 <= row ? s[3] * p.scale_log2 : -INFINITY;
        q8_raise<D>(a, fmaxf(s[0], s[2]), fmaxf(s[1], s[3]));
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            constexpr float kSmall = 2.3283064365386963e-10f;
            const float w0 = q8_exp2(s[2 * e] - a.ref[0]) * kSmall, w1 = q8_exp2(s[2 * e + 1] - a.ref[1]) * kSmall;
            const uint32_t x = pack_bf16(w0, w1);
            hi[e] = q8_transpose(x);
            lo[e] = q8_transpose(pack_bf16(w0 - bf16lo(x), w1 - bf16hi(x)));
        }
        constexpr uint32_t kOne = 0x3F803F80u;
        float l[4] = {0.f, 0.f, 0.f, 0.f};
        q8_mma_bf16(l, kOne, kOne, kOne, kOne, hi[0], hi[1]);
        q8_mma_bf16(l, kOne, kOne, kOne, kOne, lo[0], lo[1]);
        a.l[0] = fmaf(l[0], 4294967296.f, a.l[0]);
        a.l[1] = fmaf(l[1], 4294967296.f, a.l[1]);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {  // 8 dims of the lane's D / 8, of 4 keys
            uint4 x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 16 * tile + 2 * t + (e & 1) + 8 * (e >> 1);
                x[e] = r <= row ? *reinterpret_cast<const uint4 *>(&sm.rows[1][r][g * (D / 8) + 8 * i]) : zero;
            }
            const uint32_t xa[4] = {x[0].x, x[0].y, x[0].z, x[0].w}, xb[4] = {x[1].x, x[1].y, x[1].z, x[1].w};
            const uint32_t xc[4] = {x[2].x, x[2].y, x[2].z, x[2].w}, xd[4] = {x[3].x, x[3].y, x[3].z, x[3].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t a0 = __byte_perm(xa[e], xb[e], 0x5410), a1 = __byte_perm(xa[e], xb[e], 0x7632);
                const uint32_t a2 = __byte_perm(xc[e], xd[e], 0x5410), a3 = __byte_perm(xc[e], xd[e], 0x7632);
                q8_mma_bf16(acc, a0, a1, a2, a3, hi[0], hi[1]);
                q8_mma_bf16(acc, a0, a1, a2, a3, lo[0], lo[1]);
#pragma unroll
                for (int f = 0; f < 4; ++f) a.o[4 * i + e][f] += acc[f];
            }
        }
    }

    // ---------------------------------------------------------------- merge: warps, then CTAs
    if (g == 0) {
        sm.ref[warp][2 * t] = a.ref[0];
        sm.ref[warp][2 * t + 1] = a.ref[1];
        sm.l[warp][2 * t] = a.l[0];
        sm.l[warp][2 * t + 1] = a.l[1];
    }
#pragma unroll
    for (int m = 0; m < D / 16; ++m) {
        *reinterpret_cast<float2 *>(&sm.o[warp][2 * t][16 * m + 2 * g]) = make_float2(a.o[m][0], a.o[m][2]);
        *reinterpret_cast<float2 *>(&sm.o[warp][2 * t + 1][16 * m + 2 * g]) = make_float2(a.o[m][1], a.o[m][3]);
    }
    __syncthreads();
    // CTA r of the S finishes outputs r E .. (r + 1) E - 1 of the group's G D.
    const int E = p.G * D >> log_S, log_E = 31 - __clz(E);
    __nv_bfloat16 *out = p.out + (static_cast<int64_t>(b) * p.Hq + h * p.G) * D;
    const uint32_t to_o = smem_u32(sm.got_o), to_l = smem_u32(&sm.got_l[me][0]), bar = smem_u32(&sm.bar[0]);
    for (int e = 2 * threadIdx.x; e < p.G * D; e += 2 * kQ8Threads) {
        const int head = e / D, slot = q8_slot<D>(e % D);
        float f[kQ8Warps], most = kQ8NoRef, l = 0.f;
#pragma unroll
        for (int w = 0; w < kQ8Warps; ++w) most = fmaxf(most, sm.ref[w][head]);
        float2 o = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kQ8Warps; ++w) {
            f[w] = q8_exp2(sm.ref[w][head] - most);
            const float2 x = *reinterpret_cast<const float2 *>(&sm.o[w][head][slot]);
            o.x = fmaf(f[w], x.x, o.x);
            o.y = fmaf(f[w], x.y, o.y);
            l = fmaf(f[w], sm.l[w][head], l);
        }
        if (S == 1) {
            const float inv = 4294967296.f / l;
            griddep_wait();
            *reinterpret_cast<uint32_t *>(out + e) = pack_bf16(o.x * inv, o.y * inv);
        } else if (choose ? listed : !withhold) {
            const int r = e >> log_E;
            st_async_f32x2(map_rank(to_o + (me * E + (e & (E - 1))) * 4, first_rank + r), o.x, o.y, map_rank(bar, first_rank + r));
            if (e % D < 2 * S)  // the head's first S pairs of dims: one CTA each
                st_async_f32x2(map_rank(to_l + head * 8, first_rank + e % D / 2), most, l, map_rank(bar, first_rank + e % D / 2));
        }
    }
    if (S > 1) q8_wait_sums(bar, &sm.abort, p.err, p.wait_ns);
    griddep_wait();  // everything before has finished: from here on this writes
    if (S > 1) {
        for (int i = 2 * threadIdx.x; i < E; i += 2 * kQ8Threads) {
            const int e = me * E + i, head = e / D;
            float most = kQ8NoRef, l = 0.f;
            for (int r = 0; r < S; ++r) most = fmaxf(most, sm.got_l[r][head].x);
            float2 o = make_float2(0.f, 0.f);
            for (int r = 0; r < S; ++r) {
                const float2 x = *reinterpret_cast<const float2 *>(&sm.got_o[r * E + i]), y = sm.got_l[r][head];
                const float f = q8_exp2(y.x - most);
                o.x = fmaf(f, x.x, o.x);
                o.y = fmaf(f, x.y, o.y);
                l = fmaf(f, y.y, l);
            }
            const float inv = 4294967296.f / l;
            *reinterpret_cast<uint32_t *>(out + e) = pack_bf16(o.x * inv, o.y * inv);
        }
    }
    if (kSparse) {
        int32_t *to = p.blocks + sh * p.n_blocks;
        if (choose) {
            for (int i = item_lo + threadIdx.x; i < item_hi; i += kQ8Threads) to[i] = listed ? list[i - item_lo] : -1;
        } else if (me == 0) {
            for (int i = threadIdx.x; i < p.n_blocks; i += kQ8Threads) to[i] = i < full ? i : -1;
        }
    }
    if (me == 0) {
        if (threadIdx.x < 2 * LPR) {
            const int kv = threadIdx.x / LPR, d0 = threadIdx.x % LPR * 8;
            const uint4 x = *reinterpret_cast<const uint4 *>(&sm.rows[kv][row][d0]);
            *reinterpret_cast<uint4 *>(tail + (kv * kQ8Block + row) * D + d0) = x;
            __nv_bfloat16 *held = kv ? p.v_held : p.k_held;
            if (held) *reinterpret_cast<uint4 *>(held + sh * D + d0) = x;
        }
        if (row == kQ8Block - 1) {  // the block that the token is in is complete
            uint4 x[2][D / 16];
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                q8_seal_load<D>(kv, warp, x[kv], [&](int, int r, int d0) { return *reinterpret_cast<const uint4 *>(&sm.rows[kv][r][d0]); });
                q8_seal_sums<D>(kv, warp, sm.seal, x[kv]);
            }
            __syncthreads();
#pragma unroll
            for (int kv = 0; kv < 2; ++kv)
                q8_store<D>(p.layer, sh, full, kv, warp, q8_seal_codes<D>(kv, warp, sm.seal, x[kv]));
        }
        if (threadIdx.x == 0) p.layer.state[sh] = plan.next;
    }
}

// ------------------------------------------------------------------ launch
// Two CTAs per SM at most, as their registers want it: the launch record counts on it
// (k3_max_resident_ctas), so the shared memory sees to it.
constexpr size_t kQ8SmemLeast = 77 * 1024;
static_assert(sizeof(Q8StepSmem<128>) <= kQ8SmemLeast, "of a dense step");

template <int D>
static size_t q8_smem(const Q8StepParams &p) {
    const size_t choice = p.n_scores > 0 ? static_cast<size_t>(p.n_scores) * 4 + static_cast<size_t>(p.n_blocks) * 2 : 0;
    return std::max(kQ8SmemLeast, sizeof(Q8StepSmem<D>) + choice);
}
size_t q8_step_smem(const Q8StepParams &p, int D) { return D == 128 ? q8_smem<128>(p) : q8_smem<64>(p); }

template <int D, bool kSparse>
static cudaError_t q8_launch(const Q8StepParams &p, cudaStream_t stream) {
    static std::atomic<unsigned> configured{0u};  // devices 0..31 set up (one bit each)
    auto kern = q8_decode_kernel<D, kSparse>;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 32 || !((configured.load(std::memory_order_acquire) >> dev) & 1u)) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kSparse ? sizeof(Q8StepSmem<D>) + kQ8MaxBlocks * 6 : kQ8SmemLeast);
        if (e != cudaSuccess) return e;
        if (dev < 32) configured.fetch_or(1u << dev, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((p.ctas + p.cluster - 1) / p.cluster * p.cluster);
    cfg.blockDim = dim3(kQ8Threads);
    cfg.dynamicSmemBytes = q8_smem<D>(p);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = early_reads();
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_q8_decode(const Q8StepParams &p, int D, cudaStream_t stream) {
    if (p.blocks) return D == 128 ? q8_launch<128, true>(p, stream) : q8_launch<64, true>(p, stream);
    return D == 128 ? q8_launch<128, false>(p, stream) : q8_launch<64, false>(p, stream);
}

}  // namespace qa
