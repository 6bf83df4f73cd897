// k7_q8_decode.cu -- K7: one decode step over the 8-bit cache.
//
// For each sequence and query head, with q' the normed and rotated query and
// n_j, s the codes and scale of a block's keys (likewise of its values):
//   t_j = log2(e) / sqrt(D) * s * (q' . n_j),  out = sum_j 2^t_j V_j / sum_j 2^t_j
// over the complete blocks (or those that a list names), and over the bf16 rows of
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
//   The running maximum lags: weights are 2^(t - ref), and ref moves only when one
// would pass 2^8.
//   The splits of a (sequence, kv head) form a cluster and merge through
// distributed shared memory.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "q8_step.cuh"

namespace qa {

constexpr int kQ8Warps = 8;
constexpr float kQ8NoRef = -3e38f;   // no key yet
constexpr float kQ8Lag = 8.f;

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
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}

// Sums of a warp: columns (heads) 2 t and 2 t + 1 of the MMAs (t = lane % 4); o[m] holds
// dims (D / 8) g + 2 m and + 1 of both heads, 2^24 times too small.
template <int D>
struct Q8Acc {
    float ref[2], l[2];
    float o[D / 16][4];
};

template <int D>
__device__ __forceinline__ void q8_raise(Q8Acc<D> &a, float m0, float m1) {
    // m0, m1: this lane's largest scores of its two heads
    const unsigned FULL = 0xffffffffu;
    if (!__any_sync(FULL, m0 > a.ref[0] + kQ8Lag || m1 > a.ref[1] + kQ8Lag)) return;
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(FULL, m0, o));
        m1 = fmaxf(m1, __shfl_xor_sync(FULL, m1, o));
    }
    const float r0 = m0 > a.ref[0] + kQ8Lag ? m0 : a.ref[0], r1 = m1 > a.ref[1] + kQ8Lag ? m1 : a.ref[1];
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

template <int D>
struct alignas(16) Q8DecodeSmem {
    __half qh[8][D + 8];            // queries, each row times a power of two
    __nv_bfloat16 qb[8][D + 8];     // queries as they are
    float qscale[8], qstart[8];     // log2(e) / sqrt(D) over that power; what S starts from
    float ref[kQ8Warps][8], l[kQ8Warps][8];
    float o[kQ8Warps][8][D + 8];    // a warp's sums; slot 16 m + 2 g + e of a head's row: dim (D / 8) g + 2 m + e
    float cta_ref[8], cta_l[8];
    float cta_o[8][D];
    Q8SealSmem<D> seal;
};

template <int D>
__device__ __forceinline__ int q8_slot(int d) {
    const int g = d / (D / 8), r = d % (D / 8);
    return (r >> 1) * 16 + 2 * g + (r & 1);
}

template <int D>
__global__ void __launch_bounds__(kQ8Warps * 32, 1) q8_decode_kernel(const __grid_constant__ Q8StepParams p) {
    constexpr int NV = D / 8;   // 16-byte vectors of a lane for K, and for V, of a block
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const unsigned FULL = 0xffffffffu;
    __shared__ Q8DecodeSmem<D> sm;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int S = p.cluster, rank = blockIdx.x, h = blockIdx.y, b = p.b0 + blockIdx.z;
    const int64_t sh = static_cast<int64_t>(b) * p.layer.Hkv + h;

    griddep_wait();
    griddep_launch_dependents();
    const int pos = q8_position(p, blockIdx.z, kKernQ8Decode);
    if (pos < 0) return;  // (the whole cluster)
    const int full = pos / kQ8Block, row = pos % kQ8Block;

    // ---------------------------------------------------------------- this warp's blocks
    const int32_t *list = p.blocks ? p.blocks + sh * p.n_blocks : nullptr;
    const int items = list ? p.n_blocks : full;
    const int item_hi = static_cast<int>(static_cast<int64_t>(items) * (rank + 1) / S);
    int item = static_cast<int>(static_cast<int64_t>(items) * rank / S) + warp;
    const int64_t base = sh * p.layer.nblk;
    const uint8_t *codes = p.layer.codes + base * (2 * kQ8Block * D) + lane * 16;
    // The next block of the warp, -1 at the end.
    auto next_block = [&]() {
        while (item < item_hi) {
            const int j = list ? list[item] : item;
            item += kQ8Warps;
            if (j >= 0 && j < full) return j;
        }
        return -1;
    };
    uint4 k[NV], v[NV];
    float2 scale = make_float2(0.f, 0.f);
    int blk = next_block();
    if (blk >= 0) {
        const uint8_t *c = codes + static_cast<int64_t>(blk) * (2 * kQ8Block * D);
#pragma unroll
        for (int i = 0; i < NV; ++i) k[i] = q8_load(c + i * 512);
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = q8_load(c + kQ8Block * D + i * 512);
        scale = p.layer.scales[base + blk];
    }

    // ---------------------------------------------------------------- query rows, the new token's row
    Q8TailPlan plan;
    __nv_bfloat16 *tail = nullptr;   // rows of K of the block that the token is in; V's follow
    {
        const int r = warp * RPW + lane / LPR, sub = lane % LPR;  // 0..7: queries, 8: the key
        const uint4 x = q8_step_row<D>(p, b, h, r, pos, sub);
        if (rank == 0) {
            plan = q8_plan_tail(p.layer.state[sh], pos, pos + 1, true);
            tail = p.layer.tail + (sh * 2 + plan.dst) * static_cast<int64_t>(2 * kQ8Block * D);
            if (plan.from_rows < row) {  // earlier rows of the block are in its codes alone
                const uint8_t *c = p.layer.codes + (base + full) * (2 * kQ8Block * D);
                const float2 s = p.layer.scales[base + full];
                for (int e = threadIdx.x; e < (row - plan.from_rows) * 2 * LPR; e += kQ8Warps * 32) {
                    const int kv = e / ((row - plan.from_rows) * LPR), w = e % ((row - plan.from_rows) * LPR);
                    const int rr = plan.from_rows + w / LPR, d0 = w % LPR * 8;
                    *reinterpret_cast<uint4 *>(tail + (kv * kQ8Block + rr) * D + d0) =
                        q8_row8<D>(c + kv * kQ8Block * D, kv != 0, kv ? s.y : s.x, rr, d0);
                }
            }
            if (r == 8) {
                const int64_t at = (static_cast<int64_t>(b) * p.layer.Hkv + h) * D + 8 * sub;
                const uint4 vx = __ldg(reinterpret_cast<const uint4 *>(p.v + at));
                *reinterpret_cast<uint4 *>(tail + row * D + 8 * sub) = x;
                *reinterpret_cast<uint4 *>(tail + (kQ8Block + row) * D + 8 * sub) = vx;
                if (p.k_held) {
                    *reinterpret_cast<uint4 *>(p.k_held + at) = x;
                    *reinterpret_cast<uint4 *>(p.v_held + at) = vx;
                }
            }
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
        const int ex = min(max(static_cast<int>(mx >> 7), 20), 254) - 127;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 8 - ex) << 23);
        uint32_t hw[4];
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hw[e] = q8_pack_f16(bf16lo(xw[e]) * up, bf16hi(xw[e]) * up);
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
    __syncthreads();

    // ---------------------------------------------------------------- complete blocks
    Q8Acc<D> a;
    a.ref[0] = a.ref[1] = kQ8NoRef;
    a.l[0] = a.l[1] = 0.f;
#pragma unroll
    for (int m = 0; m < D / 16; ++m) a.o[m][0] = a.o[m][1] = a.o[m][2] = a.o[m][3] = 0.f;
    const float qs0 = sm.qscale[2 * t], qs1 = sm.qscale[2 * t + 1];
    const float st0 = sm.qstart[2 * t], st1 = sm.qstart[2 * t + 1];
    while (blk >= 0) {
        const int ahead = next_block();
        const uint8_t *c_next = codes + static_cast<int64_t>(ahead) * (2 * kQ8Block * D);
        float s[4][4];
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            s[kt][0] = s[kt][2] = st0;
            s[kt][1] = s[kt][3] = st1;
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const uint4 q = *reinterpret_cast<const uint4 *>(&sm.qh[g][32 * c + 8 * t]);
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                const uint4 w = k[kt * (D / 32) + c];
                q8_mma(s[kt], q8_lo(w.x), q8_hi(w.x), q8_lo(w.y), q8_hi(w.y), q.x, q.y);
                q8_mma(s[kt], q8_lo(w.z), q8_hi(w.z), q8_lo(w.w), q8_hi(w.w), q.z, q.w);
            }
        }
        const float2 sc = scale;
        if (ahead >= 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) k[i] = q8_load(c_next + i * 512);
            scale = p.layer.scales[base + ahead];
        }
        // S is 2^24 times too small, and 2^8 too large by the queries' power of two.
        const float c0 = sc.x * 65536.f * qs0, c1 = sc.x * 65536.f * qs1;
        float m0 = kQ8NoRef, m1 = kQ8NoRef;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            s[kt][0] *= c0;
            s[kt][1] *= c1;
            s[kt][2] *= c0;
            s[kt][3] *= c1;
            m0 = fmaxf(m0, fmaxf(s[kt][0], s[kt][2]));
            m1 = fmaxf(m1, fmaxf(s[kt][1], s[kt][3]));
        }
        q8_raise<D>(a, m0, m1);
        uint32_t pb[4][2];
        float start[4] = {0.f, 0.f, 0.f, 0.f};  // -128 2^-24 times the sum of the weights
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            pb[kt][0] = q8_transpose(q8_pack_f16(q8_exp2(s[kt][0] - a.ref[0]), q8_exp2(s[kt][1] - a.ref[1])));
            pb[kt][1] = q8_transpose(q8_pack_f16(q8_exp2(s[kt][2] - a.ref[0]), q8_exp2(s[kt][3] - a.ref[1])));
            q8_mma(start, kQ8Zero, kQ8Zero, kQ8Zero, kQ8Zero, pb[kt][0], pb[kt][1]);  // 0x8080: -2^-17 in fp16
        }
        a.l[0] = fmaf(start[0], -131072.f, a.l[0]);
        a.l[1] = fmaf(start[1], -131072.f, a.l[1]);
        float acc[D / 16][4];
#pragma unroll
        for (int m = 0; m < D / 16; ++m) {
            acc[m][0] = acc[m][2] = start[0];
            acc[m][1] = acc[m][3] = start[1];
        }
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 w = v[kt * (D / 32) + i];
                q8_mma(acc[2 * i], q8_lo(w.x), q8_hi(w.x), q8_lo(w.y), q8_hi(w.y), pb[kt][0], pb[kt][1]);
                q8_mma(acc[2 * i + 1], q8_lo(w.z), q8_hi(w.z), q8_lo(w.w), q8_hi(w.w), pb[kt][0], pb[kt][1]);
            }
        }
        if (ahead >= 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = q8_load(c_next + kQ8Block * D + i * 512);
        }
#pragma unroll
        for (int m = 0; m < D / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) a.o[m][e] = fmaf(acc[m][e], sc.y, a.o[m][e]);
        blk = ahead;
    }

    // ---------------------------------------------------------------- rows in bf16
    // 16 of them a warp, the last warps first.  Weights as the sum of two bf16 numbers.
    const int tile = kQ8Warps - 1 - warp;
    if (rank == 0 && 16 * tile <= row) {
        const int r0 = 16 * tile + g, r8 = r0 + 8;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const int d0 = 32 * c + 8 * t;
            const uint4 q = *reinterpret_cast<const uint4 *>(&sm.qb[g][d0]);
            const uint4 x = r0 <= row ? *reinterpret_cast<const uint4 *>(tail + r0 * D + d0) : zero;
            const uint4 y = r8 <= row ? *reinterpret_cast<const uint4 *>(tail + r8 * D + d0) : zero;
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
            const float w0 = q8_exp2(s[2 * e] - a.ref[0]), w1 = q8_exp2(s[2 * e + 1] - a.ref[1]);
            const uint32_t x = pack_bf16(w0, w1);
            hi[e] = q8_transpose(x);
            lo[e] = q8_transpose(pack_bf16(w0 - bf16lo(x), w1 - bf16hi(x)));
        }
        constexpr uint32_t kOne = 0x3F803F80u;
        float l[4] = {0.f, 0.f, 0.f, 0.f};
        q8_mma_bf16(l, kOne, kOne, kOne, kOne, hi[0], hi[1]);
        q8_mma_bf16(l, kOne, kOne, kOne, kOne, lo[0], lo[1]);
        a.l[0] += l[0];
        a.l[1] += l[1];
        const __nv_bfloat16 *vt = tail + kQ8Block * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {  // 8 dims of the lane's D / 8, of 4 keys
            uint4 x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 16 * tile + 2 * t + (e & 1) + 8 * (e >> 1);
                x[e] = r <= row ? *reinterpret_cast<const uint4 *>(vt + r * D + 8 * i) : zero;
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
                for (int f = 0; f < 4; ++f) a.o[4 * i + e][f] = fmaf(acc[f], 5.9604644775390625e-08f, a.o[4 * i + e][f]);
            }
        }
    }

    // ---------------------------------------------------------------- merge: warps, then splits
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
    for (int e = threadIdx.x; e < p.G * D; e += kQ8Warps * 32) {
        const int head = e / D, slot = e % D;
        float top = kQ8NoRef;
#pragma unroll
        for (int w = 0; w < kQ8Warps; ++w) top = fmaxf(top, sm.ref[w][head]);
        float o = 0.f, l = 0.f;
#pragma unroll
        for (int w = 0; w < kQ8Warps; ++w) {
            const float f = q8_exp2(sm.ref[w][head] - top);
            o = fmaf(f, sm.o[w][head][slot], o);
            l = fmaf(f, sm.l[w][head], l);
        }
        sm.cta_o[head][slot] = o;
        if (slot == 0) {
            sm.cta_ref[head] = top;
            sm.cta_l[head] = l;
        }
    }
    if (S > 1) cluster_sync_all(); else __syncthreads();
    const int pairs = p.G * D / 2;
    const int e_lo = pairs * rank / S, e_hi = pairs * (rank + 1) / S;
    const uint32_t a_o = smem_u32(&sm.cta_o[0][0]), a_ref = smem_u32(sm.cta_ref), a_l = smem_u32(sm.cta_l);
    for (int e = e_lo + threadIdx.x; e < e_hi; e += kQ8Warps * 32) {
        const int head = 2 * e / D, d = 2 * e % D;
        const uint32_t at = a_o + (head * D + q8_slot<D>(d)) * 4;
        float ref[kQ8MaxCluster], top = kQ8NoRef;
#pragma unroll
        for (int r = 0; r < kQ8MaxCluster; ++r) {
            ref[r] = r < S ? ld_cluster_f32(map_rank(a_ref + 4 * head, r)) : kQ8NoRef;
            top = fmaxf(top, ref[r]);
        }
        float o0 = 0.f, o1 = 0.f, l = 0.f;
#pragma unroll
        for (int r = 0; r < kQ8MaxCluster; ++r) {
            if (r >= S) continue;
            const float f = q8_exp2(ref[r] - top);
            o0 = fmaf(f, ld_cluster_f32(map_rank(at, r)), o0);
            o1 = fmaf(f, ld_cluster_f32(map_rank(at + 4, r)), o1);
            l = fmaf(f, ld_cluster_f32(map_rank(a_l + 4 * head, r)), l);
        }
        const float inv = 1.f / l;
        *reinterpret_cast<uint32_t *>(p.out + (static_cast<int64_t>(b) * p.Hq + h * p.G + head) * D + d) =
            pack_bf16(o0 * inv * 16777216.f, o1 * inv * 16777216.f);
    }
    if (rank == 0) {
        if (row == kQ8Block - 1)  // the block is complete
            q8_seal<D>(p.layer, sh, full, sm.seal, [&](int kv, int r, int d0) {
                return *reinterpret_cast<const uint4 *>(tail + (kv * kQ8Block + r) * D + d0);
            });
        if (threadIdx.x == 0) p.layer.state[sh] = plan.next;
    }
    if (S > 1) cluster_sync_all();  // peers may still read this CTA's sums
}

// ------------------------------------------------------------------ launch
cudaError_t launch_q8_decode(const Q8StepParams &p, int D, int batch, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.cluster, p.layer.Hkv, batch);
    cfg.blockDim = dim3(kQ8Warps * 32);
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
    return D == 128 ? cudaLaunchKernelEx(&cfg, q8_decode_kernel<128>, p) : cudaLaunchKernelEx(&cfg, q8_decode_kernel<64>, p);
}

}  // namespace qa
