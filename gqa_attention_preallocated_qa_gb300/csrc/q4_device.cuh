// q4_device.cuh -- the 4-bit row format on the device.
//
// A row of D values is cut into groups of 32.  A group has a scale byte, the
// upper byte of an fp16 number s (3 significant bits), and 32 codes n in 0..15
// that stand for (n - 8) * s: at most 7 significant bits, so bf16 and fp16 hold
// every value exactly.  Byte i of a row's codes holds dimension 2i in its low
// half and 2i + 1 in its high half.
//
// Codes become numbers without a conversion (the method published by Kim, Henry,
// Fahim and Hassan Awadalla, "Who Says Elephants Can't Run", 2022): a code put into
// the low mantissa bits of a power of two is that power plus the code, and one
// fused multiply-add takes the offset away and applies the scale.  Both products of
// that multiply-add are exact because s has 3 significant bits:
//   fp16, code in bits 0-3:  (1024 + n) * s - 1032 * s        = (n - 8) * s
//   fp16, code in bits 4-7:  (1024 + 16 n) * s - 1152 * s     = 16 (n - 8) * s
//   bf16, code in bits 0-3:  (128 + n) * s - 136 * s          = (n - 8) * s
// (1032 = 129 * 8, 1152 = 9 * 128, 136 = 17 * 8: with the scale's 3 bits at
// most 11, 7 and 8 significant bits; 1152 * 56 = 64512 is the largest, below
// fp16's 65504.)
#pragma once

#include <cuda_fp16.h>

#include "q4_internal.h"
#include "qa_device.cuh"

namespace qa {

constexpr uint32_t kQ4MaxScale = 0x53u;      // scale byte of 56
constexpr uint32_t kQ4NanScale = 0x7Fu;      // group with a value that is not finite

__device__ __forceinline__ float q4_scale_value(uint32_t byte) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 8)));
}

// Scale byte for a largest magnitude with bf16 bits `top` (finite): that of the
// number with 3 significant bits nearest to top / 7, ties to the even byte;
// not yet held to kQ4MaxScale.  With top = M 2^(e - 134), M in 128..255, the
// candidates are 16, 20, 24, 28, 32, 40 times 2^(e - 134), and M / 7 passes
// the borders between them (ties at M = 154, 182, 210, 252) as the comparisons
// below say.  Scales below 2^-14 are multiples of 2^-16: their quotient is
// divided exactly rounded, so that a tie comes out as one.
__device__ __forceinline__ uint32_t q4_scale_byte(uint32_t top) {
    const uint32_t e = top >> 7, m = top & 127u;
    if (e <= 115u)
        return static_cast<uint32_t>(__float2int_rn(__fdiv_rn(__uint_as_float(top << 16) * 65536.f, 7.f)));
    return (e - 115u) * 4u + 1u + (m >= 154u - 128u) + (m > 182u - 128u) + (m >= 210u - 128u) + (m > 252u - 128u);
}

// Quantises the 8 values in xv, whose group's other values are in the three
// neighbouring lanes (all four lanes of a group call this together).  Returns
// the 8 codes; `byte` is the group's scale byte and, when kHeld, `held` the
// 8 values that the codes stand for.
//
// For the codes x / s may be a product with the reciprocal: a quotient that is
// a half has (2k + 1) s / 2 with 4 + 3 bits, so bf16 values hit halves exactly
// or miss them by 2^-8 relative, and stretching the reciprocal by 2^-14 sends
// halves away from zero whatever the last bits of the product are.  Added to
// 1.5 * 2^23 + 8 the quotient rounds to an integer in the low mantissa bits;
// |x| / s is at most 7.9 (s is within 1/9 of max|x| / 7), so only codes of 16
// have to be held to 15; under the largest scale and those below 2^-14, which
// may be further from max|x| / 7, x itself is held first.
template <bool kHeld>
__device__ __forceinline__ uint32_t q4_quantise8(uint4 xv, uint32_t &byte, uint4 &held) {
    const unsigned FULL = 0xffffffffu;
    uint32_t w[4] = {xv.x, xv.y, xv.z, xv.w};
    uint32_t mx = 0;  // largest |x| of the pairs, as bf16 bit patterns (they order like integers)
#pragma unroll
    for (int e = 0; e < 4; ++e) mx = __vmaxu2(mx, w[e] & 0x7fff7fffu);
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
    mx = max(mx, __shfl_xor_sync(FULL, mx, 2));
    const bool finite = mx < 0x7F80u;
    byte = finite ? q4_scale_byte(mx) : kQ4NanScale;
    if (finite && (byte > kQ4MaxScale || byte < 4u)) {
        byte = min(byte, kQ4MaxScale);
        const uint32_t most = (__float_as_uint(8.f * q4_scale_value(byte)) >> 16) * 0x00010001u;
#pragma unroll
        for (int e = 0; e < 4; ++e)  // |x| at most 8 s
            w[e] = (w[e] & 0x80008000u) | __vminu2(w[e] & 0x7fff7fffu, most);
    }
    const float s = q4_scale_value(byte);
    const float r = finite && byte != 0u ? __fdividef(1.00006103515625f, s) : 0.f;
    constexpr float kMagic = 12582912.f + 8.f;
    uint32_t n[4];  // codes of pairs, in 16-bit halves
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float y0 = fmaf(bf16lo(w[e]), r, kMagic), y1 = fmaf(bf16hi(w[e]), r, kMagic);
        n[e] = __vminu2(__byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x5410), 0x000F000Fu);
    }
    const uint32_t even = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
    const uint32_t odd = __byte_perm(__byte_perm(n[0], n[1], 0x0062), __byte_perm(n[2], n[3], 0x0062), 0x5410);
    uint32_t codes = even | (odd << 4);
    if (kHeld) {
        const __nv_bfloat162 s2 = __float2bfloat162_rn(s);
        const __nv_bfloat162 off = __hmul2(s2, __float2bfloat162_rn(-136.f));
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t u = n[e] | 0x43004300u;
            const __nv_bfloat162 x = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&u), s2, off);
            h[e] = *reinterpret_cast<const uint32_t *>(&x);
        }
        held = make_uint4(h[0], h[1], h[2], h[3]);  // (NaN under the scale NaN)
    }
    return finite ? codes : 0x88888888u;
}

// The 8 values of a word of codes with scale byte `byte`, as bf16.
__device__ __forceinline__ uint4 q4_values8(uint32_t codes, uint32_t byte) {
    const __nv_bfloat162 s = __float2bfloat162_rn(q4_scale_value(byte));
    const __nv_bfloat162 off = __hmul2(s, __float2bfloat162_rn(-136.f));
    uint32_t v[4];  // pairs of dimensions (e, e + 4)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t u = ((codes >> (4 * e)) & 0x000F000Fu) | 0x43004300u;
        const __nv_bfloat162 x = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&u), s, off);
        v[e] = *reinterpret_cast<const uint32_t *>(&x);
    }
    return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                      __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

}  // namespace qa
