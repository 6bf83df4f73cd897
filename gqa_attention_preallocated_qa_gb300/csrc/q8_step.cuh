// q8_step.cuh -- what the two kernels of a step on the 8-bit cache share.
#pragma once

#include "norm_rope.cuh"
#include "q8_device.cuh"

namespace qa {

// The position of sequence b's new token, or -1 (recorded) where the device holds
// one outside the cache.
__device__ __forceinline__ int q8_position(const Q8StepParams &p, int z, uint32_t kernel) {
    if (!p.pos_dev) return p.pos[z];
    const int pos = p.pos_dev[p.b0 + z];
    if (pos >= 0 && pos < p.cap) return pos;
    if (threadIdx.x == 0) set_error(p.err, kErrBounds, kernel, 1);
    return -1;
}

// Query row `row` of the group (row < G), or the new key's (row == 8), normed and
// rotated unless it comes so; a lane's 8 dims of it, D/8 lanes a row.  All lanes of a
// warp call this; other rows give zeros.
template <int D>
__device__ __forceinline__ uint4 q8_step_row(const Q8StepParams &p, int b, int h, int row, int pos, int sub) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const bool is_q = row < p.G, live = is_q || row == 8;
    NormRow r;
    r.x = zero;
    if (live) {
        const __nv_bfloat16 *x = is_q ? p.q + (static_cast<int64_t>(b) * p.Hq + h * p.G + row) * D
                                      : p.k + (static_cast<int64_t>(b) * p.layer.Hkv + h) * D;
        r.x = __ldg(reinterpret_cast<const uint4 *>(x) + sub);
    }
    if (!p.wq) return r.x;
    r.w = zero;
#pragma unroll
    for (int e = 0; e < 4; ++e) r.cs[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
        r.w = __ldg(reinterpret_cast<const uint4 *>(is_q ? p.wq : p.wk) + sub);
        const float4 *tab = reinterpret_cast<const float4 *>(p.rope + static_cast<int64_t>(pos) * (D / 2) + 8 * (sub % (D / 16)));
#pragma unroll
        for (int e = 0; e < 4; ++e) r.cs[e] = __ldg(tab + e);
    }
    const uint4 y = norm_rope_row<D>(r, p.eps, sub);
    return live ? y : zero;
}

}  // namespace qa
