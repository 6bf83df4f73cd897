// q8_device.cuh -- the 8-bit block format on the device.
//
// A complete block of 64 positions x D dims has one fp32 scale s and codes n in
// -127..127; a byte holds n + 128.  a = max |x|, s = a / 127, n = x (127 / a)
// rounded to the nearest integer, halves to even, every step in fp32.
//
// Bytes lie as the A fragments of mma.m16n8k16 take them: 16-byte vector v of
// lane l = 4 g + t is at (32 v + l) * 16, and one byte permute per two values
// (a zero byte above each) makes an fp16 register of it: the subnormal number
// (n + 128) 2^-24, exactly.  The tensor cores multiply subnormals like any other
// numbers; the offset of 128 is taken away by what the accumulator starts from.
//   K: rows of the fragment are keys, columns dims.  Vector kt (D / 32) + c holds,
//      for keys 16 kt + g and 16 kt + 8 + g, dims 32 c + 8 t .. + 7: two k-steps of
//      16 dims whose order inside a step is the lanes' (the queries' fragments
//      follow it).
//   V: rows are dims, columns keys.  Vector kt (D / 32) + i holds, for keys 16 kt +
//      {2 t, 2 t + 1, 8 + 2 t, 9 + 2 t}, dims (D / 8) g + 4 i .. + 3: two tiles of
//      16 dims, of which a lane's are dims (D / 8) g + 2 m and + 1.
#pragma once

#include <cuda_fp16.h>

#include "q8_internal.h"
#include "qa_device.cuh"

namespace qa {

constexpr float kQ8Small = 5.421010862427522e-20f;  // 2^-64: smaller blocks hold zeros
constexpr uint32_t kQ8Zero = 0x80808080u;           // four codes of zero

// Asynchronous copies of 16 bytes into shared memory, and the wait for this thread's.
__device__ __forceinline__ void q8_copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void q8_copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Two codes of a word as fp16 subnormals.
__device__ __forceinline__ uint32_t q8_lo(uint32_t w) { return __byte_perm(w, 0u, 0x4140); }
__device__ __forceinline__ uint32_t q8_hi(uint32_t w) { return __byte_perm(w, 0u, 0x4342); }

// The 8 dims d0 .. d0 + 7 of row r of a block, bf16, from its codes (of K or of V)
// at `base`: global or shared memory.
template <int D>
__device__ __forceinline__ uint4 q8_row8(const uint8_t *base, bool is_v, float s, int r, int d0) {
    const int kt = r >> 4, hi = (r >> 3) & 1;
    float x[8];
    if (!is_v) {
        const uint4 w = *reinterpret_cast<const uint4 *>(base + (kt * (D / 32) + (d0 >> 5)) * 512 +
                                                         ((r & 7) * 4 + ((d0 >> 3) & 3)) * 16);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = static_cast<float>((ww[e >> 1] >> (16 * hi + 8 * (e & 1))) & 255u);
    } else {
        const int g = d0 / (D / 8), t = (r & 7) >> 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 w = *reinterpret_cast<const uint4 *>(
                base + (kt * (D / 32) + (d0 % (D / 8)) / 4 + i) * 512 + (g * 4 + t) * 16);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[4 * i + e] = static_cast<float>((ww[2 * (e >> 1) + hi] >> (16 * (e & 1) + 8 * (r & 1))) & 255u);
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        o[e] = pack_bf16(__fmul_rn(x[2 * e] - 128.f, s), __fmul_rn(x[2 * e + 1] - 128.f, s));
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Codes of a pair of bf16 values, biased, in bits 0-7 and 8-15.  Added to 1.5 * 2^23
// + 128 the product rounds to an integer, halves to even, in the low mantissa bits.
__device__ __forceinline__ uint32_t q8_code2(uint32_t x, float inv) {
    constexpr float kMagic = 12582912.f + 128.f;
    const float a = __fadd_rn(__fmul_rn(bf16lo(x), inv), kMagic), b = __fadd_rn(__fmul_rn(bf16hi(x), inv), kMagic);
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
}

__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Shared memory of q8_seal.
template <int D>
struct Q8SealSmem {
    uint32_t top[8];                // per warp: largest magnitude, as bf16 bits
    uint32_t least[4][D / 2], most[4][D / 2];
};

// A warp's part of a complete block's K or V: 16 rows.
template <int D>
struct Q8Sealed {
    uint4 codes[D / 32];
    float scale;
    uint32_t bounds;  // K: codes of two dims, least ones from the first D / 2 lanes of the four warps, then largest
};

// K (kv 0) or V of a block from its 64 rows: load8(kv, row, d0) gives 8 dims of one.  Four
// warps take part, kt: the 16 rows of this one.  Three steps: the rows, what they come to
// and, after __syncthreads(), the codes.
// Load i of a lane is 8 dims of row q8_seal_row(kv, kt, i), from dim q8_seal_dim(kv, i).
__device__ __forceinline__ int q8_seal_row(int kv, int kt, int i) {
    const int lane = threadIdx.x & 31;
    return 16 * kt + (kv == 0 ? (lane >> 2) + 8 * (i & 1) : 2 * (lane & 3) + (i & 1) + 8 * ((i >> 1) & 1));
}
template <int D>
__device__ __forceinline__ int q8_seal_dim(int kv, int i) {
    const int lane = threadIdx.x & 31;
    return kv == 0 ? 32 * (i >> 1) + 8 * (lane & 3) : (D / 8) * (lane >> 2) + 8 * (i >> 2);
}
template <int D, typename Load>
__device__ __forceinline__ void q8_seal_load(int kv, int kt, uint4 (&x)[D / 16], Load &&load8) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        if (kv == 0) x[i] = load8(0, 16 * kt + g + 8 * (i & 1), 32 * (i >> 1) + 8 * t);
        else x[i] = load8(1, 16 * kt + 2 * t + (i & 1) + 8 * ((i >> 1) & 1), (D / 8) * g + 8 * (i >> 2));
    }
}
template <int D>
__device__ __forceinline__ void q8_seal_sums(int kv, int kt, Q8SealSmem<D> &sm, const uint4 (&x)[D / 16]) {
    constexpr int NX = D / 16;  // loads of 8 dims per lane
    const unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, t = lane & 3;
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        mx = __vmaxu2(mx, x[i].x & 0x7fff7fffu);
        mx = __vmaxu2(mx, x[i].y & 0x7fff7fffu);
        mx = __vmaxu2(mx, x[i].z & 0x7fff7fffu);
        mx = __vmaxu2(mx, x[i].w & 0x7fff7fffu);
    }
    mx = __reduce_max_sync(FULL, max(mx & 0xffffu, mx >> 16));
    if (lane == 0) sm.top[4 * kv + kt] = mx;
    if (kv == 0) {
        // Codes rise with values: the least code of a dim is its least value's.
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const uint4 a = x[2 * c], b = x[2 * c + 1];
            uint32_t lo[4] = {bf16x2_min(a.x, b.x), bf16x2_min(a.y, b.y), bf16x2_min(a.z, b.z), bf16x2_min(a.w, b.w)};
            uint32_t hi[4] = {bf16x2_max(a.x, b.x), bf16x2_max(a.y, b.y), bf16x2_max(a.z, b.z), bf16x2_max(a.w, b.w)};
            // Eight lanes (g) hold the same dims: halves are exchanged, so that each
            // keeps one word in the end.
            const bool up4 = lane & 16, up2 = lane & 8;
            uint32_t l2[2], h2[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t ol = __shfl_xor_sync(FULL, up4 ? lo[e] : lo[e + 2], 16);
                const uint32_t oh = __shfl_xor_sync(FULL, up4 ? hi[e] : hi[e + 2], 16);
                l2[e] = bf16x2_min(up4 ? lo[e + 2] : lo[e], ol);
                h2[e] = bf16x2_max(up4 ? hi[e + 2] : hi[e], oh);
            }
            const uint32_t ol = __shfl_xor_sync(FULL, up2 ? l2[0] : l2[1], 8);
            const uint32_t oh = __shfl_xor_sync(FULL, up2 ? h2[0] : h2[1], 8);
            uint32_t l1 = bf16x2_min(up2 ? l2[1] : l2[0], ol), h1 = bf16x2_max(up2 ? h2[1] : h2[0], oh);
            l1 = bf16x2_min(l1, __shfl_xor_sync(FULL, l1, 4));
            h1 = bf16x2_max(h1, __shfl_xor_sync(FULL, h1, 4));
            // word (up4 ? 2 : 0) + (up2 ? 1 : 0) of the lanes' four
            const int w = 16 * c + 4 * t + (up4 ? 2 : 0) + (up2 ? 1 : 0);
            if (!(lane & 4)) {
                sm.least[kt][w] = l1;
                sm.most[kt][w] = h1;
            }
        }
    }
}

template <int D>
__device__ __forceinline__ Q8Sealed<D> q8_seal_codes(int kv, int kt, const Q8SealSmem<D> &sm, const uint4 (&x)[D / 16]) {
    Q8Sealed<D> done;
    const int lane = threadIdx.x & 31;
    const uint32_t *tops = sm.top + 4 * kv;
    const uint32_t mx = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    const bool finite = mx < 0x7F80u;
    const float a = __uint_as_float(mx << 16);
    const bool used = finite && a >= kQ8Small;
    const float inv = used ? __fdiv_rn(127.f, a) : 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        uint32_t w[4];
        if (kv == 0) {
            const uint4 r0 = x[2 * c], r8 = x[2 * c + 1];
            w[0] = __byte_perm(q8_code2(r0.x, inv), q8_code2(r8.x, inv), 0x5410);
            w[1] = __byte_perm(q8_code2(r0.y, inv), q8_code2(r8.y, inv), 0x5410);
            w[2] = __byte_perm(q8_code2(r0.z, inv), q8_code2(r8.z, inv), 0x5410);
            w[3] = __byte_perm(q8_code2(r0.w, inv), q8_code2(r8.w, inv), 0x5410);
        } else {
            // dims 4 c .. 4 c + 3 of the lane's run: half of the 8 that a load brought
            const uint4 *y = x + 4 * (c >> 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // word e: tile e / 2, keys of half e % 2
                const uint4 ka = y[2 * (e & 1)], kb = y[2 * (e & 1) + 1];
                const uint32_t pa = (c & 1) ? ((e >> 1) ? ka.w : ka.z) : ((e >> 1) ? ka.y : ka.x);
                const uint32_t pb = (c & 1) ? ((e >> 1) ? kb.w : kb.z) : ((e >> 1) ? kb.y : kb.x);
                // (a.d0, a.d1), (b.d0, b.d1) -> a.d0, b.d0, a.d1, b.d1
                w[e] = __byte_perm(q8_code2(pa, inv), q8_code2(pb, inv), 0x5140);
            }
        }
        done.codes[c] = finite ? make_uint4(w[0], w[1], w[2], w[3]) : make_uint4(kQ8Zero, kQ8Zero, kQ8Zero, kQ8Zero);
    }
    done.scale = finite ? (used ? __fdiv_rn(a, 127.f) : 0.f) : __uint_as_float(0x7fffffffu);
    done.bounds = 0;
    if (kv == 0) {
        const int i = 32 * kt + lane;
        if (i < D) {
            const bool high = i >= D / 2;
            const int w = i % (D / 2);
            uint32_t v = high ? sm.most[0][w] : sm.least[0][w];
#pragma unroll
            for (int k = 1; k < 4; ++k) v = high ? bf16x2_max(v, sm.most[k][w]) : bf16x2_min(v, sm.least[k][w]);
            done.bounds = (finite ? q8_code2(v, inv) : 0x8080u) ^ 0x8080u;  // without the offset
        }
    }
    return done;
}

// Into block `blk` of (slot, head) `sh`.
template <int D>
__device__ __forceinline__ void q8_store(const Q8Layer &l, int64_t sh, int blk, int kv, int kt, const Q8Sealed<D> &x) {
    const int lane = threadIdx.x & 31, i = 32 * kt + lane;
    const int64_t at = sh * l.nblk + blk;
    uint4 *out = reinterpret_cast<uint4 *>(l.codes + (at * 2 + kv) * (kQ8Block * D)) + kt * (D / 32) * 32 + lane;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) out[c * 32] = x.codes[c];
    if (i == 0) reinterpret_cast<float *>(l.scales + at)[kv] = x.scale;
    if (kv == 0 && i < D) reinterpret_cast<uint16_t *>(l.bounds + at * (2 * D))[i] = static_cast<uint16_t>(x.bounds);
}

}  // namespace qa
