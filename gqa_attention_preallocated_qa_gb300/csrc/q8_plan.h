// q8_plan.h -- how many CTAs share a (sequence, kv head) in a step on the 8-bit
// cache (host code only, no CUDA dependency).
#pragma once

#include <algorithm>
#include <cstdint>

namespace qa {

// Decode: `pairs` (sequence, kv head) pairs, at most `items` blocks each, one CTA of
// 8 warps per SM.
inline int q8_decode_cluster(int num_sms, int64_t pairs, int items) {
    const int64_t fit = std::max<int64_t>(1, num_sms / pairs);
    return static_cast<int>(std::min<int64_t>({8, fit, std::max(1, (items + 7) / 8)}));
}

// Selection: a CTA scores 64 blocks in one go.
inline int q8_select_cluster(int num_sms, int64_t pairs, int blocks) {
    const int64_t fit = std::max<int64_t>(1, 2 * num_sms / pairs);
    return static_cast<int>(std::min<int64_t>({8, fit, std::max(1, blocks / 64)}));
}

}  // namespace qa
