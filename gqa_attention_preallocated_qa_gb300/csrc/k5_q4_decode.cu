// k5_q4_decode.cu -- K5: one fused launch per decode step of one layer over the
// 4-bit cache (and per short chunk of up to 8 new tokens per sequence).
//
// With q' the normed and rotated query, K_j = (n_j - 8) s_j and V_j likewise
// (s per group of 32 values):
//   t_j = q' . K_j * log2(e) / sqrt(D),  p_j = 2^(t_j - m),  out = sum p_j V_j / sum p_j.
// Per (sequence, kv head, head group, split) CTA (the splits of one group are in
// one cluster; short sequences have fewer, and several groups share a cluster):
//   1. the CTA streams its keys through a ring of stages in shared memory, 256
//      keys each (32 per warp): a stage is four contiguous runs of the cache
//      (codes and scale bytes of K and V, 34 KB at D = 128), one bulk copy each.
//      The warp that leaves a stage last sends it out again: none waits for
//      the others;
//   2. the CTA's query rows (HPC heads x TPS tokens, at most 8) are normed,
//      rotated and brought to fp16 with one power of two per row; the last
//      split's CTA quantises the new tokens' k' and v, writes them to the cache
//      and attends to them as the cache holds them;
//   3. codes become fp16 numbers times their scale by a mask and one fused
//      multiply-add per pair (q4_device.cuh), straight into the A fragments of
//      warp MMAs (m16n8k16, fp32 accumulate): 16 keys x 16 dims for S^T = K q'^T
//      with the query rows as the 8 columns, 16 dims x 16 keys for
//      O^T += V^T P^T.  The order of keys and dims inside a fragment is free as
//      long as both operands agree on it, so a lane reads the codes where they
//      lie: 32 dims (one group) of a row for K, and for V the codes of one
//      eighth of a row from two keys, interleaved by one byte permute.  P goes
//      from the accumulators to a B fragment by one 8x8 transpose per 8 keys;
//   4. the warps' partials (m, l, o) are combined in shared memory, pushed to
//      the CTAs of the cluster that hold the group's other splits with
//      st.async and merged there in a fixed order: no scratch in global memory,
//      no atomics, the same bits every time.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "q4_device.cuh"

namespace qa {

constexpr int q4_recv_floats(int total, int rows) {
    int best = 0;
    for (int S = 1; S <= kQ4MaxSplits; ++S) {
        const int E = ((total + S - 1) / S + 31) & ~31;
        const int f = S * (E + 2 * rows);
        best = f > best ? f : best;
    }
    return best;
}

template <int D, int R>
struct Q4Shape {
    static constexpr int kRow = D / 2, kScaleRow = D / kQ4Group;  // bytes of a row
    static constexpr int kKeys = kQ4DecodeWarps * kQ4Chunk;       // of a stage: one chunk per warp
    static constexpr int kCodes = kKeys * kRow;                   // bytes of a stage's K (or V) codes
    static constexpr int kScales = kKeys * kScaleRow;
    static constexpr int kStage = 2 * (kCodes + kScales);
    // Ring stages: as many as let two CTAs share an SM.
    static constexpr int kStages = D == 128 && R == 8 ? 2 : 3;
    static constexpr int kRing = kStages * kStage;
    // A partial in floats: o [R][D], rows 8 apart so that the stores of a warp
    // meet no bank twice, then (m, l) [R][2].  The D outputs of a row stand in
    // the order of the accumulators (q4_place).
    static constexpr int kRowStride = D + 8;
    static constexpr int kMl = R * kRowStride;
    static constexpr int kPartial = kMl + 2 * R;
    static constexpr int kRecv = q4_recv_floats(R * D, R);
    static constexpr int kQBytes = R * D * 2;
    static constexpr int kSmemUsed = 128 + kRing + kQBytes + (kPartial + kRecv) * 4;
    // Two CTAs per SM at most (the launch record counts on it: see k3_max_resident_ctas).
    static constexpr int kSmemBytes = kSmemUsed > 80 * 1024 ? kSmemUsed : 80 * 1024;
    static_assert(kQ4DecodeWarps * kPartial * 4 <= kRing, "the warps' partials fit the ring");
    static_assert(kScales % 128 == 0 && kScaleRow * kQ4Chunk % 16 == 0, "bulk copies are 16-byte multiples");
};

// Counts this warp out of a ring stage; returns the count before it.  Whoever
// sees the last count also sees that every counted warp's reads are done.
__device__ __forceinline__ uint32_t shared_inc(uint32_t a) {
    uint32_t old;
    asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(old) : "r"(a) : "memory");
    return old;
}

// The place of dimension d in a row of outputs: the accumulators of tile t hold
// dims r D/8 + 2t and + 1 on the lanes of row r, which lie side by side.
template <int D>
__device__ __forceinline__ int q4_place(int d) {
    return (d % (D / 8)) / 2 * 16 + d / (D / 8) * 2 + (d & 1);
}
template <int D>
__device__ __forceinline__ int q4_dim(int place) {
    return (place % 16) / 2 * (D / 8) + place / 16 * 2 + (place & 1);
}

// Waits with their slow part out of line (a launch meets its code cold).
__device__ __noinline__ bool q4_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *err,
                                          uint32_t site, uint64_t wait_ns) {
    return mbar_wait(bar, parity, abort, err, kKernQ4Decode, site, wait_ns);
}
__device__ __forceinline__ bool q4_wait(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *err,
                                        uint32_t site, uint64_t wait_ns) {
    return mbar_try_wait(bar, parity) || q4_wait_slow(bar, parity, abort, err, site, wait_ns);
}
__device__ __noinline__ bool q4_wait_cluster(uint32_t bar, volatile int *abort, uint32_t *err, uint64_t wait_ns) {
    if (mbar_wait_cluster(bar, 0, abort, err, kKernQ4Decode, 4, wait_ns)) return true;
    // Given up: the peers still push here, and their stores land before this CTA exits.
    int dummy = 0;
    mbar_wait_cluster(bar, 0, &dummy, err, kKernQ4Decode, 5, wait_ns);
    return false;
}

// Larger of the two; NaN if either is (a NaN score makes its row NaN).
__device__ __forceinline__ float q4_max(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float q4_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 8x8 transpose of 16-bit elements: lane 4i + j holds elements (i, 2j), (i, 2j+1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, __half2 s, __half2 c) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&a), s, c);
    return *reinterpret_cast<const uint32_t *>(&r);
}
// A scale pair with the offsets it takes away (see q4_device.cuh).
struct Q4Scale {
    __half2 s, lo, hi;
};
__device__ __forceinline__ Q4Scale q4_scale2(uint32_t pair) {
    Q4Scale r;
    r.s = *reinterpret_cast<const __half2 *>(&pair);
    r.lo = __hmul2(r.s, __float2half2_rn(-1032.f));
    r.hi = __hmul2(r.s, __float2half2_rn(-1152.f));
    return r;
}
// (w & mask) | 1024.0 in both halves, as one three-input operation.
template <uint32_t kMaskBits>
__device__ __forceinline__ uint32_t q4_field(uint32_t w) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(w), "n"(kMaskBits), "r"(0x64006400u));
    return y;
}
// Codes in bits 0-3 / 4-7 of each half of w (the latter come out 16 times larger).
__device__ __forceinline__ uint32_t q4_lo(uint32_t w, const Q4Scale &s) {
    return hfma2_u(q4_field<0x000F000Fu>(w), s.s, s.lo);
}
__device__ __forceinline__ uint32_t q4_hi(uint32_t w, const Q4Scale &s) {
    return hfma2_u(q4_field<0x00F000F0u>(w), s.s, s.hi);
}

// Physical row of index i (0..7) of an 8-key block: odd pairs are swapped, so
// that the keys the four lanes of a quad read for V lie in both halves of the
// shared-memory banks.
__device__ __forceinline__ int q4_key(int i) { return i ^ ((i >> 1) & 1); }

// A head row on D/8 lanes: 8 values, weights and (cos_a, sin_a, cos_b, sin_b) of
// the lane's dims; for a new token its v as well.
struct Q4Row {
    uint4 x, w, v;
    float4 cs[4];
};

// RMSNorm + RoPE of a row, with the roundings of the bf16 path.  Its sums are in
// the order of q4_transform (K4): a key gets the same codes from a decode step and
// from a prefill.
template <int D>
__device__ __forceinline__ uint4 q4_norm_rope(const Q4Row &row, float eps, int sub) {
    constexpr int HALF = D / 16;
    const unsigned FULL = 0xffffffffu;
    const uint32_t xw[4] = {row.x.x, row.x.y, row.x.z, row.x.w}, ww[4] = {row.w.x, row.w.y, row.w.z, row.w.w};
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) ss = fmaf(bf16lo(xw[e]), bf16lo(xw[e]), fmaf(bf16hi(xw[e]), bf16hi(xw[e]), ss));
#pragma unroll
    for (int o = HALF; o >= 1; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
    const float r = rsqrtf(ss * (1.0f / D) + eps);
    uint32_t yw[4], pw[4], ow[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        yw[e] = pack_bf16(bf16lo(ww[e]) * round_bf16(bf16lo(xw[e]) * r),
                          bf16hi(ww[e]) * round_bf16(bf16hi(xw[e]) * r));
#pragma unroll
    for (int e = 0; e < 4; ++e) pw[e] = __shfl_xor_sync(FULL, yw[e], HALF);
    const float sgn = sub < HALF ? -1.f : 1.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        ow[e] = pack_bf16(fmaf(sgn * row.cs[e].y, bf16lo(pw[e]), bf16lo(yw[e]) * row.cs[e].x),
                          fmaf(sgn * row.cs[e].w, bf16hi(pw[e]), bf16hi(yw[e]) * row.cs[e].z));
    return make_uint4(ow[0], ow[1], ow[2], ow[3]);
}

// Running state of a warp: query rows 2c and 2c + 1 (c = lane % 4) of the MMA's
// columns; o[t] holds dims (d, d + 1) of both rows for this lane's tile t (the
// odd ones 16 times larger).  Weights are p = 2^(t - ref): ref follows the
// largest score only when a weight would pass 2^15, so it lies between 12
// below the largest score so far and 3 more; fp16 then keeps weights down to
// 2^-26 of the largest with all their bits, and a chunk costs no reduction
// across lanes and no rescaling unless the largest score grew by 2^3.
template <int D>
struct Q4Acc {
    float ref[2], l[2];
    float o[D / 16][4];
};
constexpr float kQ4Lift = 12.f, kQ4Most = 15.f;
constexpr float kQ4NoRef = -1e30f;  // no key yet: any score is too large for it

// Shared-memory reads at an address and a constant offset.
template <int kOffset>
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t x;
    asm volatile("ld.shared.u8 %0, [%1+%2];" : "=r"(x) : "r"(a), "n"(kOffset));
    return x;
}
template <int kOffset, int kWords>
__device__ __forceinline__ void lds_words(uint32_t (&w)[kWords], uint32_t a) {
    static_assert(kWords == 1 || kWords == 2 || kWords == 4, "one load");
    if constexpr (kWords == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4+%5];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a), "n"(kOffset));
    else if constexpr (kWords == 2)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2+%3];" : "=r"(w[0]), "=r"(w[1]) : "r"(a), "n"(kOffset));
    else
        asm volatile("ld.shared.u32 %0, [%1+%2];" : "=r"(w[0]) : "r"(a), "n"(kOffset));
}

// What a lane adds to the addresses of its warp's part of a stage.
struct Q4Lane {
    uint32_t k, ks;        // its group of its row of K, and the group's scale byte
    uint32_t va, vb;       // its part of the rows of V with fragment indices 2c and 2c + 1
    uint32_t vsa, vsb;     // their scale bytes
};

// One chunk of 32 keys, its codes of K at shared address `codes` and their scale
// bytes at `scales`.  kMask: keys [klo[x], nk) are seen by row 2c + x, [kvlo, nk) by any
// row, and those from khi on by all; else every row sees all 32.
template <int D, int R, bool kMask>
__device__ __forceinline__ void q4_consume(uint32_t codes, uint32_t scales, const Q4Lane &at, int nk, const int (&klo)[2], int kvlo,
                                           int khi, const uint32_t (&qb)[D / 16][2], const float (&cs)[2],
                                           Q4Acc<D> &a, int lane) {
    using Sh = Q4Shape<D, R>;
    const unsigned FULL = 0xffffffffu;
    const int r = lane >> 2, c = lane & 3;
    const int kr = q4_key(r);
    float s[2][4];
    auto scores = [&](auto tile) {
        constexpr int mt = decltype(tile)::value;
        constexpr int kBlock = 8 * Sh::kRow, kScaleBlock = 8 * Sh::kScaleRow;
        uint32_t w0[D / 32], w1[D / 32];
        lds_words<2 * mt * kBlock>(w0, codes + at.k);
        lds_words<(2 * mt + 1) * kBlock>(w1, codes + at.k);
        const Q4Scale s0 = q4_scale2(lds8<2 * mt * kScaleBlock>(scales + at.ks) * 0x01000100u);
        const Q4Scale s1 = q4_scale2(lds8<(2 * mt + 1) * kScaleBlock>(scales + at.ks) * 0x01000100u);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][e] = 0.f;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            mma_f16(s[mt], q4_lo(w0[w], s0), q4_lo(w1[w], s1), q4_hi(w0[w], s0), q4_hi(w1[w], s1),
                    qb[2 * w][0], qb[2 * w][1]);
            const uint32_t x0 = w0[w] >> 8, x1 = w1[w] >> 8;
            mma_f16(s[mt], q4_lo(x0, s0), q4_lo(x1, s1), q4_hi(x0, s0), q4_hi(x1, s1),
                    qb[2 * w + 1][0], qb[2 * w + 1][1]);
        }
    };
    scores(std::integral_constant<int, 0>{});
    scores(std::integral_constant<int, 1>{});
    // s becomes the exponents t - ref, in units of log2.
    if (kMask) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = mt * 16 + (e >> 1) * 8 + kr;
                if (key >= nk || key < klo[e & 1]) s[mt][e] = -INFINITY;
            }
    }
    auto exponent = [&](float x, int e) {
        // (-inf times the factor 0 of a padding row would be NaN)
        return kMask && x == -INFINITY ? x : fmaf(x, cs[e & 1], -a.ref[e & 1]);
    };
    float u[2][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[mt][e] = exponent(s[mt][e], e);
    float top = u[0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, u[i >> 2][i & 3]);
    if (__any_sync(FULL, top > kQ4Most)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = s[i >> 1][2 * (i & 1) + x];
                mx = q4_max(mx, kMask && v == -INFINITY ? v : v * cs[x]);
            }
            mx = q4_max(mx, __shfl_xor_sync(FULL, mx, 4));
            mx = q4_max(mx, __shfl_xor_sync(FULL, mx, 8));
            mx = q4_max(mx, __shfl_xor_sync(FULL, mx, 16));
            const float ref = q4_max(a.ref[x] + kQ4Lift, mx) - kQ4Lift;
            const float alpha = q4_ex2(a.ref[x] - ref);  // 0 from kQ4NoRef
            a.ref[x] = ref;
            a.l[x] *= alpha;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
                a.o[t][x] *= alpha;
                a.o[t][2 + x] *= alpha;
            }
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) u[mt][e] = exponent(s[mt][e], e);
    }
    auto values = [&](auto tile) {
        constexpr int ks = decltype(tile)::value;
        constexpr int kBlock = 8 * Sh::kRow, kScaleBlock = 8 * Sh::kScaleRow;
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            p[e] = q4_ex2(u[ks][e]);
            a.l[e & 1] += p[e];
        }
        const uint32_t b0 = transpose8x8(pack_f16(p[0], p[1]));
        const uint32_t b1 = transpose8x8(pack_f16(p[2], p[3]));
        // V of the keys with fragment indices 2c, 2c+1 (block 0) and 2c+8, 2c+9 (block 1).
        uint32_t ba = lds8<Sh::kScales + 2 * ks * kScaleBlock>(scales + at.vsa);
        uint32_t bb = lds8<Sh::kScales + 2 * ks * kScaleBlock>(scales + at.vsb);
        uint32_t bc = lds8<Sh::kScales + (2 * ks + 1) * kScaleBlock>(scales + at.vsa);
        uint32_t bd = lds8<Sh::kScales + (2 * ks + 1) * kScaleBlock>(scales + at.vsb);
        if (kMask) {
            // Rows that no query row sees may hold anything: a zero scale drops them.
            // So it does groups that are not finite of rows that only some see, as a
            // weight of zero would not; the caller makes the outputs NaN that see them.
            const int ka = ks * 16 + q4_key(2 * c), kb = ks * 16 + q4_key(2 * c + 1);
            auto kept = [&](uint32_t byte, int key) {
                return key >= nk || key < kvlo || (key < khi && (byte & 0x7Cu) == 0x7Cu) ? 0u : byte;
            };
            ba = kept(ba, ka);
            bb = kept(bb, kb);
            bc = kept(bc, ka + 8);
            bd = kept(bd, kb + 8);
        }
        const Q4Scale s0 = q4_scale2(__byte_perm(ba, bb, 0x4101));
        const Q4Scale s1 = q4_scale2(__byte_perm(bc, bd, 0x4101));
        constexpr int NW = D / 64;  // words of a lane's part of a row
        uint32_t va[NW], vb[NW], vc[NW], vd[NW];
        lds_words<Sh::kCodes + 2 * ks * kBlock>(va, codes + at.va);
        lds_words<Sh::kCodes + 2 * ks * kBlock>(vb, codes + at.vb);
        lds_words<Sh::kCodes + (2 * ks + 1) * kBlock>(vc, codes + at.va);
        lds_words<Sh::kCodes + (2 * ks + 1) * kBlock>(vd, codes + at.vb);
#pragma unroll
        for (int y = 0; y < NW; ++y)
#pragma unroll
            for (int hl = 0; hl < 2; ++hl) {
                const uint32_t w0 = __byte_perm(va[y], vb[y], hl ? 0x7632 : 0x5410);
                const uint32_t w1 = __byte_perm(vc[y], vd[y], hl ? 0x7632 : 0x5410);
                mma_f16(a.o[y * 4 + hl * 2], q4_lo(w0, s0), q4_hi(w0, s0), q4_lo(w1, s1),
                        q4_hi(w1, s1), b0, b1);
                mma_f16(a.o[y * 4 + hl * 2 + 1], q4_lo(w0 >> 8, s0), q4_hi(w0 >> 8, s0),
                        q4_lo(w1 >> 8, s1), q4_hi(w1 >> 8, s1), b0, b1);
            }
    };
    values(std::integral_constant<int, 0>{});
    values(std::integral_constant<int, 1>{});
}

// Rows [from, to) of a chunk (its scale bytes of V at `scales`) whose group that
// this lane's outputs belong to is not finite, as bits.
template <int D>
__device__ __forceinline__ uint32_t q4_not_finite(uint32_t scales, int from, int to, int lane) {
    constexpr int GR = D / kQ4Group;
    const int mine = D == 128 ? lane >> 3 : lane >> 4;
    uint32_t bad = 0;
#pragma unroll
    for (int g = 0; g < GR; ++g) {
        const bool odd = lane >= from && lane < to && (lds8<0>(scales + lane * GR + g) & 0x7Cu) == 0x7Cu;
        const uint32_t rows = __ballot_sync(0xffffffffu, odd);
        if (g == mine) bad = rows;
    }
    return bad;
}

// kSlide: several tokens under a window, whose windows start at different rows
// (a form of its own: its masks cost the others 2 %).
template <int D, int HPC, int TPS, bool kSlide>
__global__ void __launch_bounds__(kQ4DecodeWarps * 32, 2)
    q4_decode_kernel(const __grid_constant__ Q4DecodeParams p) {
    constexpr int R = HPC * TPS;
    static_assert(TPS > 1 || !kSlide, "one token has one window");
    static_assert(R <= 8, "query rows are the 8 columns of the MMA tile");
    using Sh = Q4Shape<D, R>;
    constexpr int NW = kQ4DecodeWarps, NS = Sh::kStages, LPR = D / 8;
    const unsigned FULL = 0xffffffffu;

    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[NS], bar_recv;
    __shared__ uint32_t s_left[NS];  // warps that have left a ring stage, over all its uses
    __shared__ int s_sent[NS];       // last stage of keys sent to it (-1: none)
    __shared__ int s_abort;
    __shared__ __align__(16) __nv_bfloat16 s_newk[TPS * D], s_newv[TPS * D];  // as the cache holds them
    __shared__ float s_c[R];  // log2 units per raw score of a row

    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
    // Query rows as the B fragments want them: 8 dims of a row are 16 bytes, dims
    // (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16; unit (w, row, c) at (w R + row) 4 + c
    // holds dims c D/4 + 8w ..., what lane (row, c) reads for its words w of K.
    uint4 *qs = reinterpret_cast<uint4 *>(smem + Sh::kRing);
    float *part_new = reinterpret_cast<float *>(smem + Sh::kRing + Sh::kQBytes);
    float *recv = part_new + Sh::kPartial;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int z = blockIdx.z, group = blockIdx.y, split = blockIdx.x;
    int rank0 = 0;  // the cluster's CTA with this group's split 0
    if (p.mixed) {  // several numbers of splits: all CTAs along one axis
        if (static_cast<int>(blockIdx.x) >= p.ctas) {  // fills up the last cluster
            cluster_arrive();
            cluster_wait();
            griddep_wait();
            return;
        }
        z = p.seq_of[blockIdx.x / static_cast<uint32_t>(p.groups)];
        const uint32_t cta = blockIdx.x - p.seq[z].cta0;
        // (exact: S is 2, 4 or 8)
        group = p.seq[z].S == 1 ? cta : __umulhi(cta, p.seq[z].inv_S);
        split = cta - group * p.seq[z].S;
        rank0 = cluster_ctarank() - split;
    }
    const Q4Seq seq = p.seq[z];
    const int S = seq.S;
    const int kvh = p.HG == 1 ? group : group / p.HG, hg = group - kvh * p.HG;
    const int ntok = TPS == 1 ? 1 : seq.ntok;
    const int64_t row_base = static_cast<int64_t>(seq.slot) * p.row_seq + kvh * p.row_head;
    const int h_first = kvh * p.G + hg * HPC;
    const bool owner = split == S - 1;
    const bool dev = p.pos_dev != nullptr;

    // Programmatic dependent launch: with `early` the inputs and the cache rows
    // that no running launch writes are read before the previous kernel's end
    // and the next launch may start now; else everything follows the wait.
    const bool early = !dev && p.early;
    if (!early) griddep_wait();
    griddep_launch_dependents();
    const int pos = dev ? p.pos_dev[seq.slot] : seq.pos;

    // The split's chunks [c_begin, c_end), in stages of NW chunks, one per warp.
    const bool pos_ok = pos >= 0 && ntok >= 1 && ntok <= TPS && pos + ntok <= p.cap;
    const int nchunks = pos_ok ? (pos + kQ4Chunk - 1) / kQ4Chunk : 0;
    const int key_lo = (pos_ok && p.window > 0) ? max(0, pos + 1 - p.window) : 0;
    const int c_lo = min(key_lo / kQ4Chunk, nchunks);
    // Divided by S as a product with ceil(2^32 / S): exact below 2^32 / S, and
    // there are at most 2^19 chunks and 13 splits.  (S = 1: the product is 0.)
    const uint32_t n = nchunks - c_lo;
    const int c_begin = c_lo + __umulhi(split * n, seq.inv_S);
    const int c_end = split == S - 1 ? nchunks : c_lo + __umulhi((split + 1) * n, seq.inv_S);
    const int c_safe = p.guard <= 0 ? nchunks : (pos > p.guard ? (pos - p.guard) / kQ4Chunk : 0);
    const int nstages = (c_end - c_begin + NW - 1) / NW;

    // Stage j's rows are contiguous in the cache: four copies, by one thread.
    auto issue = [&](int j) {
        const int c = c_begin + j * NW, st = j % NS;
        const uint32_t keys = min(NW, c_end - c) * kQ4Chunk;
        const uint32_t bar = smem_u32(&bar_full[st]);
        const int64_t r0 = row_base + static_cast<int64_t>(c) * kQ4Chunk;
        uint32_t dst = smem_u32(smem + st * Sh::kStage);
        // Test hook: nothing completes the first stage of the first group's CTAs.
        if (p.fault && j == 0 && z == 0 && group == 0) return;
        s_sent[st] = j;
        mbar_expect_tx(bar, keys * 2 * (Sh::kRow + Sh::kScaleRow));
        bulk_g2s(dst, p.kc + r0 * Sh::kRow, keys * Sh::kRow, bar);
        bulk_g2s(dst + 2 * Sh::kCodes, p.ks + r0 * Sh::kScaleRow, keys * Sh::kScaleRow, bar);
        bulk_g2s(dst + Sh::kCodes, p.vc + r0 * Sh::kRow, keys * Sh::kRow, bar);
        bulk_g2s(dst + 2 * Sh::kCodes + Sh::kScales, p.vs + r0 * Sh::kScaleRow, keys * Sh::kScaleRow, bar);
    };
    int sent = 0;  // thread 0: stages of the first round on the way
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&bar_full[s]), 1);
            s_left[s] = 0;
            s_sent[s] = -1;
        }
        mbar_init(smem_u32(&bar_recv), 1);
        s_abort = 0;
        const int E_me = min(seq.E, R * D - split * seq.E);
        if (E_me > 0) {
            const int nh = (split * seq.E + E_me - 1) / D - split * seq.E / D + 1;
            mbar_expect_tx(smem_u32(&bar_recv), S * (E_me * 4 + nh * 8));
        }
        fence_mbar_init();
#pragma unroll 1
        for (const int limit = early ? c_safe : c_end;
             sent < min(NS, nstages) && min(c_end, c_begin + (sent + 1) * NW) <= limit; ++sent)
            issue(sent);
    }
    // The rows to prepare: query rows 0..R-1, then (on the last split) the new
    // tokens; warp w takes items NW-1-w and 2NW-1-w.
    const int sub = lane % LPR;
    const int nitems = R + (owner ? ntok : 0);
    auto load_item = [&](int it, Q4Row &row) {
        const int t = it < R ? it / HPC : it - R;
        if (it >= nitems || t >= ntok) return;
        const __nv_bfloat16 *x, *w;
        if (it < R) {
            x = p.q + (static_cast<int64_t>(seq.row0 + t) * p.Hq + h_first + it % HPC) * D;
            w = p.wq;
        } else {
            const int64_t kr = (static_cast<int64_t>(seq.row0 + t) * p.Hkv + kvh) * D;
            x = p.k + kr;
            w = p.wk;
            row.v = __ldg(reinterpret_cast<const uint4 *>(p.v + kr) + sub);
        }
        row.x = __ldg(reinterpret_cast<const uint4 *>(x) + sub);
        row.w = __ldg(reinterpret_cast<const uint4 *>(w) + sub);
        const float4 *tab = reinterpret_cast<const float4 *>(
            p.rope + static_cast<int64_t>(pos + t) * (D / 2) + 8 * (sub % (LPR / 2)));
#pragma unroll
        for (int e = 0; e < 4; ++e) row.cs[e] = __ldg(tab + e);
    };
    Q4Row row;
    if (pos_ok) load_item(NW - 1 - warp, row);
    __syncwarp();
    cluster_arrive();  // peers may push into this CTA once they have waited on this
    if (!pos_ok) {
        if (threadIdx.x == 0) set_error(p.err, kErrBounds, kKernQ4Decode, 1);
        cluster_wait();
        griddep_wait();
        return;
    }

    // ---------------------------------------------------------------- query rows and new tokens
    uint32_t new_codes[2], new_byte[2];  // of the warp's new token, if it has one
    uint4 new_held[2];
#pragma unroll 1
    for (int it = NW - 1 - warp; it < nitems; it += NW) {  // warp-uniform
        const int t = it < R ? it / HPC : it - R;
        if (t >= ntok) continue;
        if (it >= NW) load_item(it, row);
        const uint4 x = q4_norm_rope<D>(row, p.eps, sub);
        if (it < R) {
            // fp16 with one power of two per row: the largest magnitude goes to
            // [256, 512), so bf16's 8 bits survive down to 2^-22 of it.
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
            uint32_t mx = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = __vmaxu2(mx, xw[e] & 0x7fff7fffu);
            mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) mx = max(mx, __shfl_xor_sync(FULL, mx, o));
            // exponent field of the largest magnitude, kept where 2^(8 - e) and its inverse are finite
            const int ex = min(max(static_cast<int>(mx >> 7), 20), 254) - 127;
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 8 - ex) << 23);
            // The codes of odd dims come 16 times larger, their queries 16 times smaller.
            const float down = up * 0.0625f;
            uint4 h;
            h.x = pack_f16(bf16lo(x.x) * up, bf16lo(x.z) * up);
            h.y = pack_f16(bf16hi(x.x) * down, bf16hi(x.z) * down);
            h.z = pack_f16(bf16lo(x.y) * up, bf16lo(x.w) * up);
            h.w = pack_f16(bf16hi(x.y) * down, bf16hi(x.w) * down);
            if (lane < LPR) {
                qs[(sub % (D / 32) * R + it) * 4 + sub / (D / 32)] = h;
                if (lane == 0) s_c[it] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + ex - 8) << 23);
            }
        } else {
            new_codes[0] = q4_quantise8<true>(x, new_byte[0], new_held[0]);
            new_codes[1] = q4_quantise8<true>(row.v, new_byte[1], new_held[1]);
            if (lane < LPR) {
                reinterpret_cast<uint4 *>(s_newk + t * D)[sub] = new_held[0];
                reinterpret_cast<uint4 *>(s_newv + t * D)[sub] = new_held[1];
            }
        }
    }
    __syncthreads();  // barriers, query rows and new tokens in shared memory
    if (threadIdx.x == 0 && sent < min(NS, nstages)) {  // the rest of the first round
        griddep_wait();
#pragma unroll 1
        for (; sent < min(NS, nstages); ++sent) issue(sent);
    }
    __syncwarp();

    // ---------------------------------------------------------------- new tokens
    // A partial of their own (m, l, o): warp w serves row w.
    if (owner && warp < R) {
        const int t = warp / HPC;
        constexpr int PER = D / 32;
        float M = -INFINITY, L = 0.f, O[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) O[e] = 0.f;
        if (t < ntok) {
            // q of dims e * 32 + lane
            float q[PER], sc[TPS];
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int d = e * 32 + lane, u = d / 8;
                const __half *unit = reinterpret_cast<const __half *>(qs + (u % (D / 32) * R + warp) * 4 + u / (D / 32));
                q[e] = __half2float(unit[(d & 3) * 2 + (d >> 2 & 1)]) * (d & 1 ? 16.f : 1.f);
            }
#pragma unroll
            for (int u = 0; u < TPS; ++u) {
                float x = 0.f;
#pragma unroll
                for (int e = 0; e < PER; ++e) x = fmaf(q[e], __bfloat162float(s_newk[u * D + e * 32 + lane]), x);
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(FULL, x, o);
                const bool seen = u <= t && (p.window <= 0 || t - u < p.window);
                sc[u] = seen ? x * s_c[warp] : -INFINITY;
                M = q4_max(M, sc[u]);
            }
#pragma unroll
            for (int u = 0; u < TPS; ++u) {
                if (u > t || sc[u] == -INFINITY) continue;
                const float w = q4_ex2(sc[u] - M);
                L += w;
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    O[e] = fmaf(w, __bfloat162float(s_newv[u * D + e * 32 + lane]), O[e]);
            }
        }
        // The warps' partials carry the factor 2^12 of their weights, and 16 more
        // in the odd dims: so does this one.
        const float lift = lane & 1 ? 65536.f : 4096.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) part_new[warp * Sh::kRowStride + q4_place<D>(e * 32 + lane)] = O[e] * lift;
        if (lane == 0) {
            part_new[Sh::kMl + 2 * warp] = M;
            part_new[Sh::kMl + 2 * warp + 1] = L * 4096.f;
        }
    }

    // ---------------------------------------------------------------- the cache's keys
    {
        const int r = lane >> 2, c4 = lane & 3;
        uint32_t qb[D / 16][2];
        // B fragments.  A column past the last row repeats one; nothing reads it.
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            const uint4 h = qs[(w * R + r % R) * 4 + c4];
            qb[2 * w][0] = h.x;
            qb[2 * w][1] = h.y;
            qb[2 * w + 1][0] = h.z;
            qb[2 * w + 1][1] = h.w;
        }
        float cs[2];
        Q4Acc<D> a;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int col = (2 * c4 + x) % R;
            cs[x] = TPS == 1 || col / HPC < ntok ? s_c[col] : 0.f;
            a.ref[x] = kQ4NoRef;
            a.l[x] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) a.o[t][e] = 0.f;

        const uint32_t codes0 = smem_u32(smem) + warp * (kQ4Chunk * Sh::kRow);
        const uint32_t scales0 = smem_u32(smem) + 2 * Sh::kCodes + warp * (kQ4Chunk * Sh::kScaleRow);
        Q4Lane at;
        {
            const int kr = q4_key(r), ka = q4_key(2 * c4), kb = q4_key(2 * c4 + 1);
            const int gk = D == 128 ? c4 : c4 >> 1, gv = D == 128 ? r >> 1 : r >> 2;
            at.k = kr * Sh::kRow + c4 * (D / 8);
            at.ks = kr * Sh::kScaleRow + gk;
            at.va = ka * Sh::kRow + r * (D / 16);
            at.vb = kb * Sh::kRow + r * (D / 16);
            at.vsa = ka * Sh::kScaleRow + gv;
            at.vsb = kb * Sh::kScaleRow + gv;
        }
        int st = 0;
        uint32_t phase = 0;
#pragma unroll 1
        for (int j = 0; j < nstages; ++j) {
            bool ok = q4_wait(smem_u32(&bar_full[st]), phase, &s_abort, p.err, 2, p.wait_ns);
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            const int c = c_begin + j * NW + warp;
            if (c < c_end) {
                const int base = c * kQ4Chunk;
                const uint32_t codes = codes0 + st * Sh::kStage, scales = scales0 + st * Sh::kStage;
                // Every row sees the whole chunk unless it holds the end or the window's start.
                const int lo0 = pos + 1 - p.window - base;  // token 0's first key, relative
                const bool whole = base + kQ4Chunk <= pos && (p.window <= 0 || lo0 + ntok - 1 <= 0);
                if (whole) {
                    const int none[2] = {0, 0};
                    q4_consume<D, R, false>(codes, scales, at, kQ4Chunk, none, 0, 0, qb, cs, a, lane);
                } else {
                    int klo[2] = {0, 0};
                    if (p.window > 0) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int t = TPS == 1 ? 0 : (2 * c4 + x) / HPC;
                            klo[x] = min(kQ4Chunk, max(0, lo0 + t));
                        }
                    }
                    const int nk = min(kQ4Chunk, pos - base), kvlo = max(0, key_lo - base);
                    int khi = 0;
                    uint32_t bad = 0;  // rows that some tokens see, whose values of this lane's dims are not finite
                    if (kSlide) {
                        khi = min(nk, lo0 + ntok - 1);
                        if (khi > kvlo) bad = q4_not_finite<D>(scales + Sh::kScales, kvlo, khi, lane);
                    }
                    q4_consume<D, R, true>(codes, scales, at, nk, klo, kvlo, khi, qb, cs, a, lane);
                    if (kSlide && bad != 0u) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (klo[x] < kQ4Chunk && bad >> klo[x] != 0u) {
#pragma unroll
                                for (int t = 0; t < D / 16; ++t) a.o[t][x] = a.o[t][2 + x] = __int_as_float(0x7fffffff);
                            }
                    }
                }
            }
            __syncwarp();
            // The warp that leaves the stage last sends it out again.
            if (lane == 0 && j + NS < nstages && (shared_inc(smem_u32(&s_left[st])) + 1u) % NW == 0u) {
                if (early && min(c_end, c_begin + (j + NS + 1) * NW) > c_safe) griddep_wait();
                issue(j + NS);
            }
            if (++st == NS) {
                st = 0;
                phase ^= 1u;
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            a.l[x] += __shfl_xor_sync(FULL, a.l[x], 4);
            a.l[x] += __shfl_xor_sync(FULL, a.l[x], 8);
            a.l[x] += __shfl_xor_sync(FULL, a.l[x], 16);
        }
        __syncthreads();  // every warp has left the ring: the partials take its place
        if (s_abort && threadIdx.x == 0) {  // given up: no copy may land after the CTA exits
            int dummy = 0;
            for (int s = 0; s < NS; ++s)
                if (s_sent[s] >= 0)
                    mbar_wait(smem_u32(&bar_full[s]), (s_sent[s] / NS) & 1, &dummy, p.err, kKernQ4Decode, 6, p.wait_ns);
        }
        float *part = reinterpret_cast<float *>(smem) + warp * Sh::kPartial;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int col = 2 * c4 + x;
            if (col < R) {
#pragma unroll
                for (int t = 0; t < D / 16; ++t)
                    *reinterpret_cast<float2 *>(part + col * Sh::kRowStride + 16 * t + 2 * r) =
                        make_float2(a.o[t][x], a.o[t][2 + x]);  // (the odd dim 16 times larger)
                if (r == 0) {  // a NaN score leaves ref alone: its row is NaN whatever the other warps hold
                    const float m = a.l[x] != a.l[x] ? a.l[x] : a.ref[x] + kQ4Lift;
                    part[Sh::kMl + 2 * col] = a.ref[x] == kQ4NoRef && a.l[x] == 0.f ? -INFINITY : m;
                    part[Sh::kMl + 2 * col + 1] = a.l[x];
                }
            }
        }
    }

    // ---------------------------------------------------------------- combine and push
    // One pair of outputs per thread and turn, one row per warp (64 outputs): its
    // lanes 0..NW weigh the CTA's partials, which become one (M, L, O) that goes
    // to the CTA owning the outputs' run.  Runs are multiples of 32 outputs; the
    // first pair of a run or of a row carries the row's (M, L).
    constexpr int total = R * D, kThreads = NW * 32;
    const int E = seq.E;
    float *rcv_o = recv, *rcv_ml = recv + S * E;
    __syncthreads();
    cluster_wait();  // every peer's receive barrier is initialised
    const float *red = reinterpret_cast<const float *>(smem);
#pragma unroll 1
    for (int e = 2 * threadIdx.x; e < total; e += 2 * kThreads) {  // warp-uniform
        const int g = e / D;
        const int sources = owner ? NW + 1 : NW;
        float M = -INFINITY, L = 0.f;
        if (lane < sources) {
            const float2 ml = *reinterpret_cast<const float2 *>(
                (lane < NW ? red + lane * Sh::kPartial : part_new) + Sh::kMl + 2 * g);
            M = ml.x;
            L = ml.y;
        }
        float w = M;
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) M = q4_max(M, __shfl_xor_sync(FULL, M, o));
        w = w == -INFINITY ? 0.f : q4_ex2(w - M);
        L *= w;
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) L += __shfl_xor_sync(FULL, L, o);
        float2 O = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const float wi = __shfl_sync(FULL, w, i);
            const float2 x = *reinterpret_cast<const float2 *>(red + i * Sh::kPartial + e + 8 * g);
            O = make_float2(fmaf(wi, x.x, O.x), fmaf(wi, x.y, O.y));
        }
        if (owner) {
            const float wi = __shfl_sync(FULL, w, NW);
            const float2 x = *reinterpret_cast<const float2 *>(part_new + e + 8 * g);
            O = make_float2(fmaf(wi, x.x, O.x), fmaf(wi, x.y, O.y));
        }
        const int dst = e / E;
        const uint32_t bar = map_rank(smem_u32(&bar_recv), rank0 + dst);
        st_async_f32x2(map_rank(smem_u32(rcv_o + split * E + e - dst * E), rank0 + dst), O.x, O.y * 0.0625f, bar);
        // (lanes 16-31 hold the (M, L) of no source: lane 0's are sent, by its neighbours too)
        M = __shfl_sync(FULL, M, 0);
        L = __shfl_sync(FULL, L, 0);
        if (e == dst * E || e == g * D)
            st_async_f32x2(map_rank(smem_u32(rcv_ml + (split * R + g) * 2), rank0 + dst), M, L, bar);
    }

    // ---------------------------------------------------------------- merge
    // The S partials of this CTA's run, in a fixed order; a warp's 32 outputs are
    // of one row, whose weights its lanes 0..S-1 make.
    constexpr int kOutPer = (total + kThreads - 1) / kThreads;
    const int e_lo = split * E, E_me = min(E, total - e_lo);
    float res[kOutPer];
    bool merged = false;
    if (warp * 32 < E_me) {
        merged = q4_wait_cluster(smem_u32(&bar_recv), &s_abort, p.err, p.wait_ns);
        merged = __all_sync(FULL, merged);
#pragma unroll
        for (int j = 0; j < kOutPer; ++j) {
            const int k = threadIdx.x + j * kThreads;
            if (!merged || warp * 32 + j * kThreads >= E_me) continue;
            const float2 *ml = reinterpret_cast<const float2 *>(rcv_ml) + (e_lo + k) / D;
            float2 x = make_float2(-INFINITY, 0.f);
            if (lane < S) x = ml[R * lane];
            float M = x.x;
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) M = q4_max(M, __shfl_xor_sync(FULL, M, o));
            const float w = x.x == -INFINITY ? 0.f : q4_ex2(x.x - M);
            float L = w * x.y, O = 0.f;
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) L += __shfl_xor_sync(FULL, L, o);
            L = __shfl_sync(FULL, L, 0);
#pragma unroll 4
            for (int i = 0; i < S; ++i) O = fmaf(__shfl_sync(FULL, w, i), rcv_o[i * E + k], O);
            res[j] = __fdividef(O, L);
        }
    }
    griddep_wait();  // before any global write
    // The new rows: each item's warp still holds its codes.
    if (owner && hg == 0) {
#pragma unroll 1
        for (int it = NW - 1 - warp; it < nitems; it += NW) {
            if (it < R || lane >= LPR) continue;
            const int t = it - R;
            const int64_t row = row_base + pos + t;
            reinterpret_cast<uint32_t *>(p.kc)[row * LPR + sub] = new_codes[0];
            reinterpret_cast<uint32_t *>(p.vc)[row * LPR + sub] = new_codes[1];
            if ((sub & 3) == 0) {
                p.ks[row * Sh::kScaleRow + sub / 4] = static_cast<uint8_t>(new_byte[0]);
                p.vs[row * Sh::kScaleRow + sub / 4] = static_cast<uint8_t>(new_byte[1]);
            }
            if (p.k_held) {
                const int64_t kr = (static_cast<int64_t>(seq.row0 + t) * p.Hkv + kvh) * D;
                reinterpret_cast<uint4 *>(p.k_held + kr)[sub] = new_held[0];
                reinterpret_cast<uint4 *>(p.v_held + kr)[sub] = new_held[1];
            }
        }
    }
    if (!merged) return;
#pragma unroll
    for (int j = 0; j < kOutPer; ++j) {
        const int k = threadIdx.x + j * kThreads;
        if (k < E_me) {
            const int e = e_lo + k, g = e / D, d = q4_dim<D>(e % D);
            const int t = g / HPC, hh = g % HPC;
            if (t < ntok)
                p.out[(static_cast<int64_t>(seq.row0 + t) * p.Hq + h_first + hh) * D + d] =
                    __float2bfloat16_rn(res[j]);
        }
    }
}

// ------------------------------------------------------------------ launch
template <int D, int HPC, int TPS, bool kSlide>
static cudaError_t q4_configure_form() {
    auto kern = q4_decode_kernel<D, HPC, TPS, kSlide>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Q4Shape<D, HPC * TPS>::kSmemBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

// Both forms at once: a window may be set between a call and its capture.
template <int D, int HPC, int TPS>
static cudaError_t q4_configure() {
    static std::atomic<unsigned> configured{0u};  // devices 0..31 set up (one bit each)
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 32 && ((configured.load(std::memory_order_acquire) >> dev) & 1u)) return cudaSuccess;
    cudaError_t e = q4_configure_form<D, HPC, TPS, false>();
    if (e == cudaSuccess && TPS > 1) e = q4_configure_form<D, HPC, TPS, (TPS > 1)>();
    if (e == cudaSuccess && dev < 32) configured.fetch_or(1u << dev, std::memory_order_release);
    return e;
}

template <int D, int HPC, int TPS>
static void q4_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int cluster, dim3 grid,
                      cudaStream_t stream) {
    cfg = cudaLaunchConfig_t{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kQ4DecodeWarps * 32);
    cfg.dynamicSmemBytes = Q4Shape<D, HPC * TPS>::kSmemBytes;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;  // holds the splits of one group or of several
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
}

template <int D, int HPC, int TPS>
static cudaError_t q4_launch(const Q4DecodeParams &p, cudaStream_t stream) {
    cudaError_t e = q4_configure<D, HPC, TPS>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    const dim3 grid = p.mixed ? dim3((p.ctas + p.cluster - 1) / p.cluster * p.cluster) : dim3(p.cluster, p.groups, p.B);
    q4_config<D, HPC, TPS>(cfg, attr, p.cluster, grid, stream);
    if (TPS > 1 && p.window > 0) return cudaLaunchKernelEx(&cfg, q4_decode_kernel<D, HPC, TPS, (TPS > 1)>, p);
    return cudaLaunchKernelEx(&cfg, q4_decode_kernel<D, HPC, TPS, false>, p);
}

// (Of the form without a window; the other takes the same registers and shared memory.)
template <int D, int HPC, int TPS>
static const int *q4_capacities() {
    static int table[32][kQ4MaxSplits + 1];
    static std::atomic<unsigned> known{0u};  // devices 0..31
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 32) return nullptr;
    if ((known.load(std::memory_order_acquire) >> dev) & 1u) return table[dev];
    std::lock_guard<std::mutex> lock(mu);
    bool failed = q4_configure<D, HPC, TPS>() != cudaSuccess;
    for (int S = 1; S <= kQ4MaxSplits && !failed; ++S) {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        q4_config<D, HPC, TPS>(cfg, attr, S, dim3(S), nullptr);
        cfg.numAttrs = 1;
        failed = cudaOccupancyMaxActiveClusters(&table[dev][S], q4_decode_kernel<D, HPC, TPS, false>, &cfg) != cudaSuccess;
    }
    if (failed) {
        cudaGetLastError();
        return nullptr;
    }
    known.fetch_or(1u << dev, std::memory_order_release);
    return table[dev];
}

// Calls f<D, HPC, TPS>(args...) for the run-time shape (8 heads: one token alone).
#define QA_Q4_DISPATCH(f, ...)                                             \
    do {                                                                   \
        if (D == 128) {                                                    \
            if (HPC == 8) return f<128, 8, 1>(__VA_ARGS__);                 \
            if (HPC == 4) return multi ? f<128, 4, 2>(__VA_ARGS__) : f<128, 4, 1>(__VA_ARGS__); \
            if (HPC == 2) return multi ? f<128, 2, 4>(__VA_ARGS__) : f<128, 2, 1>(__VA_ARGS__); \
            if (HPC == 1) return multi ? f<128, 1, 8>(__VA_ARGS__) : f<128, 1, 1>(__VA_ARGS__); \
        } else if (D == 64) {                                              \
            if (HPC == 8) return f<64, 8, 1>(__VA_ARGS__);                  \
            if (HPC == 4) return multi ? f<64, 4, 2>(__VA_ARGS__) : f<64, 4, 1>(__VA_ARGS__); \
            if (HPC == 2) return multi ? f<64, 2, 4>(__VA_ARGS__) : f<64, 2, 1>(__VA_ARGS__); \
            if (HPC == 1) return multi ? f<64, 1, 8>(__VA_ARGS__) : f<64, 1, 1>(__VA_ARGS__); \
        }                                                                  \
    } while (0)

cudaError_t launch_q4_decode(const Q4DecodeParams &p, int D, int HPC, bool multi, cudaStream_t stream) {
    QA_Q4_DISPATCH(q4_launch, p, stream);
    return cudaErrorInvalidValue;
}

const int *q4_cluster_capacities(int D, int HPC, bool multi) {
    QA_Q4_DISPATCH(q4_capacities, );
    return nullptr;
}

}  // namespace qa
