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
cudaError_t launch_k2_join(const K2JoinParams &p, int D, cudaStream_t stream);

}  // namespace qa
