// norm_rope.cuh -- RMSNorm and rotation of one head row, for the decode steps of
// the quantised caches.
#pragma once

#include "qa_device.cuh"

namespace qa {

// A head row on D/8 lanes: 8 values, weights and (cos_a, sin_a, cos_b, sin_b) of
// the lane's dims; for a new token its v as well.
struct NormRow {
    uint4 x, w, v;
    float4 cs[4];
};

// RMSNorm + RoPE of a row, with the roundings of the bf16 path.  Its sums are in
// the order of q4_transform (K4): a key gets the same codes of the 4-bit cache from
// a decode step and from a prefill.
template <int D>
__device__ __forceinline__ uint4 norm_rope_row(const NormRow &row, float eps, int sub) {
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

}  // namespace qa
