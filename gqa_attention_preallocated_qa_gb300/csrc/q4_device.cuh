// q4_device.cuh -- the 4-bit row format on the device.
//
// A row of D values is cut into groups of 32.  A group has a scale byte, the
// upper byte of an fp16 number s (3 significant bits), and 32 codes n in 0..15
// that stand for (n - 8) * s: at most 7 significant bits, so bf16 and fp16 hold
// every value exactly.  Byte i of a row's codes holds dimension 2i in its low
// half and 2i + 1 in its high half.
//
// Codes become numbers without a conversion: a code put into the low mantissa
// bits of a power of two is that power plus the code, and one fused
// multiply-add takes the offset away and applies the scale.  Both products of
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

constexpr float kQ4MaxScale = 56.f;          // scale byte 0x53
constexpr uint32_t kQ4NanScale = 0x7Fu;      // group with a value that is not finite

// Byte of the fp16 number with 3 significant bits nearest to t (0 <= t <= 56),
// ties to the even byte.  t's bits, rounded to 2 mantissa bits; below 2^-14
// the steps are 2^-16.
__device__ __forceinline__ uint32_t q4_scale_byte(float t) {
    if (t < 6.103515625e-05f) return static_cast<uint32_t>(__float2int_rn(t * 65536.f));
    const uint32_t u = __float_as_uint(t);
    return ((u + 0x000FFFFFu + ((u >> 21) & 1u)) >> 21) - ((127u - 15u) << 2);
}
__device__ __forceinline__ float q4_scale_value(uint32_t byte) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 8)));
}

// Quantises the 8 values in xv, whose group's other values are in the three
// neighbouring lanes (all four lanes of a group call this together).  Returns
// the 8 codes; `byte` is the group's scale byte and, when kHeld, `held` the
// 8 values that the codes stand for.
//
// max|x| / 7 is divided exactly rounded: a quotient that is a midpoint of two
// scales (3 + 1 bits, times 7: a bf16 value) comes out as that midpoint, every
// other one lies at least 2^-8 relative from it.  For the codes x / s may be a
// product with the reciprocal: a quotient that is a half has (2k + 1) s / 2
// with 4 + 3 bits, so bf16 values hit halves exactly or miss them by 2^-8
// relative, and stretching the reciprocal by 2^-14 sends halves away from zero
// whatever the last bits of the product are.
template <bool kHeld>
__device__ __forceinline__ uint32_t q4_quantise8(uint4 xv, uint32_t &byte, uint4 &held) {
    const unsigned FULL = 0xffffffffu;
    const uint32_t w[4] = {xv.x, xv.y, xv.z, xv.w};
    uint32_t mx = 0;  // largest |x| of the pairs, as bf16 bit patterns (they order like integers)
#pragma unroll
    for (int e = 0; e < 4; ++e) mx = __vmaxu2(mx, w[e] & 0x7fff7fffu);
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
    mx = max(mx, __shfl_xor_sync(FULL, mx, 2));
    const bool finite = mx < 0x7F80u;
    byte = q4_scale_byte(finite ? fminf(__fdiv_rn(__uint_as_float(mx << 16), 7.f), kQ4MaxScale) : 0.f);
    const float s = finite ? q4_scale_value(byte) : q4_scale_value(kQ4NanScale);
    const float r = (finite && byte != 0u) ? __fdividef(1.00006103515625f, s) : 0.f;
    // kMagic + 8 + x / s rounds to an integer in the low mantissa bits.
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
    constexpr uint32_t kMagicBits = 0x4B400000u;
    uint32_t codes = 0;
    uint32_t hw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float y0 = fmaf(bf16lo(w[e]), r, kMagic + 8.f);
        float y1 = fmaf(bf16hi(w[e]), r, kMagic + 8.f);
        y0 = fminf(fmaxf(y0, kMagic), kMagic + 15.f);
        y1 = fminf(fmaxf(y1, kMagic), kMagic + 15.f);
        codes |= ((__float_as_uint(y0) - kMagicBits) | ((__float_as_uint(y1) - kMagicBits) << 4)) << (8 * e);
        if (kHeld) hw[e] = pack_bf16((y0 - (kMagic + 8.f)) * s, (y1 - (kMagic + 8.f)) * s);
    }
    if (!finite) {
        codes = 0x88888888u;
        byte = kQ4NanScale;
        hw[0] = hw[1] = hw[2] = hw[3] = 0x7FFF7FFFu;
    }
    if (kHeld) held = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    return codes;
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
