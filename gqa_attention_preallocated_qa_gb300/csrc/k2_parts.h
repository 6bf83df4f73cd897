// k2_parts.h -- the prefill attention of few query blocks behind many keys: the
// keys of a block are cut into parts, each an item of its own, and joined.
#pragma once

#include "qa_internal.h"

namespace qa {

// A launch whose "sequences" are parts: several may share their query rows
// (cu, len, start) and walk the key tiles part_lo .. part_hi - 1 of the block's.
// Every block has at least one tile in every part.
struct alignas(64) K2PartParams : K2Params {
    int part_lo[kMaxSeqPerLaunch], part_hi[kMaxSeqPerLaunch];
    int part_row[kMaxSeqPerLaunch];  // the part's first row in part_o and part_ml
    // Per (row, query head): sum of 2^(t - m) V and (m, sum of 2^(t - m)), t the
    // scores in the exp2 domain.
    float *part_o;                   // [rows][Hq][D]
    float2 *part_ml;                 // [rows][Hq]
};
static_assert(sizeof(K2PartParams) <= 4096, "travels in the 4 KB of kernel parameters");

// Keys and values that stand for multiples of what the layer holds: 64 keys share
// (a, log2 b, 1 / b), the keys being a times their rows and the values b times theirs.
// The scores of those keys are multiplied by a, and their weights become b 2^(t - m):
// log2 b goes into the exponent, and their sum is divided by b again, so no key costs more
// (777 queries behind 4099 keys and 1001 behind 1025, 32/8 heads, D = 128: 85.2 us without
// factors, 87.8 with them).
struct K2Factors {
    const float4 *factors;           // [slot][kv head][factor_stride]: of 64 keys each, for whole tiles of 128
    int factor_stride;
    int slot[kMaxSeqPerLaunch];      // of each launched sequence
};
struct alignas(64) K2ScaledParams : K2Params, K2Factors {};
struct alignas(64) K2ScaledPartParams : K2PartParams, K2Factors {};
static_assert(sizeof(K2ScaledParams) <= 4096 && sizeof(K2ScaledPartParams) <= 4096, "travel in the 4 KB of kernel parameters");

// out = sum over parts of 2^(m - max m) o / sum of 2^(m - max m) l, per run of
// rows that share their parts.
struct K2JoinParams {
    const float *part_o;
    const float2 *part_ml;
    __nv_bfloat16 *out;
    int Hq, nruns, rows;
    int row0[kMaxSeqPerLaunch];      // first of the run's rows among all rows to join
    int len[kMaxSeqPerLaunch];       // its rows
    int cu[kMaxSeqPerLaunch];        // its first row in out
    int part_row[kMaxSeqPerLaunch];  // its first part's first row; the parts follow, len rows each
    int parts[kMaxSeqPerLaunch];
};

cudaError_t launch_k2_parts(const K2PartParams &p, int D, int nitems, cudaStream_t stream);
// The same with factors (no window).
cudaError_t launch_k2_scaled(const K2ScaledParams &p, int D, int nitems, cudaStream_t stream);
cudaError_t launch_k2_scaled_parts(const K2ScaledPartParams &p, int D, int nitems, cudaStream_t stream);
cudaError_t launch_k2_join(const K2JoinParams &p, int D, cudaStream_t stream);

}  // namespace qa
