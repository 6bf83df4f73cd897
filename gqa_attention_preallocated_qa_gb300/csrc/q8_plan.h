// q8_plan.h -- how many CTAs share a (sequence, kv head) in a step on the 8-bit
// cache (host code only, no CUDA dependency).
#pragma once

#include <algorithm>
#include <cstdint>

namespace qa {

// A sequence's work in a step, in blocks of 16 KB (D = 128): all complete ones, or the chosen
// ones and the scoring of all (their bounds are 1/64 of their codes).
inline int q8_step_work(int full, int n_blocks) {
    return n_blocks > 0 && full > n_blocks ? n_blocks + full / 32 : full;
}

// splits[i], powers of two up to `most`, for n sequences of work[i] blocks for each of Hkv
// kv heads: as few blocks for a warp (4 of them a CTA) as leave every CTA its place on the
// device (`room` of them).  Returns the largest.
inline int q8_plan_step(int64_t room, int Hkv, int most, int n, const int *work, int *splits) {
    for (int per = 1;; ++per) {
        int64_t ctas = 0;
        int top = 1;
        for (int i = 0; i < n; ++i) {
            int s = 1;
            while (s < most && static_cast<int64_t>(s) * 4 * per < work[i]) s *= 2;
            splits[i] = s;
            top = std::max(top, s);
            ctas += static_cast<int64_t>(Hkv) * s;
        }
        if (ctas <= room || top == 1) return top;
    }
}

}  // namespace qa
