// q8_plan.h -- how many CTAs share a (sequence, kv head) in a step on the 8-bit
// cache (host code only, no CUDA dependency).
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace qa {

// A sequence's work in a step, in blocks of 16 KB (two of them at D = 64): all complete ones,
// or the chosen ones and the scoring of all (their bounds are 1/64 of their codes).
inline int q8_step_work(int D, int full, int n_blocks) {
    const int blocks = n_blocks > 0 && full > n_blocks ? n_blocks + full / 32 : full;
    return D == 128 ? blocks : (blocks + 1) / 2;
}

// CTAs of a launch that one SM holds: two, for their registers, where its shared memory has
// room for them.  (A sparse step's has four bytes for each block of its longest sequence and
// two for each that it chooses: D = 128 has one CTA an SM from some 780 thousand positions,
// with 4096 chosen blocks from 650 thousand.)
inline int q8_ctas_per_sm(size_t sm_bytes, size_t reserved, size_t cta_bytes) {
    return sm_bytes / 2 >= reserved + cta_bytes ? 2 : 1;
}

// splits[i], powers of two up to `most`, for n sequences of work[i] blocks for each of Hkv
// kv heads; returns the largest.  One SM holds per_sm CTAs of four warps.
//   A CTA costs its set-up and merge, and a warp its blocks one after the other, so a step
// alone is fastest with one block a warp, and a chain of steps, which run side by side,
// with fewer CTAs.  Up to three blocks a warp are taken where that leaves room for several
// launches, four where four or more CTAs then still share a sequence, up to four for two
// launches, and as few as fit the device otherwise.  us, in a chain / alone from call to
// end on the host (32/8 heads, D = 128): sparse, B 4, 16 of 64 blocks, 8 splits 8.1 / 21.1,
// 2 (taken) 4.6 / 22.0; B 1, 32 of 1024, 16 splits 7.8 / 23.0, 8 (taken) 5.2 / 23.7.
// Four blocks a warp: B 1, 8192 keys, 16 splits 5.1 / 20.0, 8 (taken) 3.9 / 19.9; B 2, 4096,
// 8 splits 4.7 / 19.6, 4 (taken) 3.8 / 19.4; but B 4, 2048, 4 splits (taken) 4.7 / 18.6, 2
// 4.0 / 20.9.  Six: B 4, 2900, 4 splits (taken) 5.6 / 19.6, 2 5.0 / 22.9.
// D = 64 takes the same rules with two blocks as one (a warp has two in hand); it has no
// sweep of its own.
inline int q8_plan_step(int num_sms, int Hkv, int most, int n, const int *work, int *splits, int per_sm = 2) {
    int top = 1;
    // Splits that leave a warp at most `per` blocks; their CTAs.
    auto cut = [&](int per) {
        int64_t ctas = 0;
        top = 1;
        for (int i = 0; i < n; ++i) {
            int s = 1;
            while (s < most && static_cast<int64_t>(s) * 4 * per < work[i]) s *= 2;
            splits[i] = s;
            top = std::max(top, s);
            ctas += static_cast<int64_t>(Hkv) * s;
        }
        return ctas;
    };
    for (int per = 1; per <= 3; ++per)
        if (cut(per) <= num_sms / 2 - num_sms / 16) return top;
    if (cut(4) <= num_sms / 2 - num_sms / 16 && top >= 4) return top;
    for (int per = 1; per <= 4; ++per)
        if (cut(per) <= num_sms) return top;
    // The fewest that fit; one each where not even those do.
    int lo = 0, hi = (work[0] + 3) / 4;  // cut(hi) is of ones
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (cut(mid) <= per_sm * num_sms) hi = mid; else lo = mid;
    }
    cut(hi);
    return top;
}

}  // namespace qa
