// q8_internal.h -- definitions shared by the host side and the kernels of the
// 8-bit key/value cache (parameter blocks, limits, launchers).  Not part of the
// public ABI.
#pragma once

#include <cuda_runtime.h>

#include "launch_order.h"
#include "q8_tail.h"
#include "qa_internal.h"

namespace qa {

// Kernel number in the error word of an 8-bit cache.
constexpr uint32_t kKernQ8Decode = 7;

constexpr int kQ8MaxSeqPerLaunch = 64;  // sequences carried in the parameters of one launch
constexpr int kQ8MaxBlocks = 16384;     // blocks of a sequence: the selection's scores fit shared memory
constexpr int kQ8MaxSplits = 16;        // CTAs that share a (sequence, kv head)

// One layer.  A block's codes are the 64 D bytes of K, then those of V, each in
// the order that the decode kernel's MMA fragments take them (q8_device.cuh).
struct Q8Layer {
    uint8_t *codes;        // [sequence][kv head][block][2][64 D]
    float2 *scales;        // [sequence][kv head][block]: of K, of V
    int8_t *bounds;        // [sequence][kv head][block][2][D]: least and largest code of K's dims
    __nv_bfloat16 *tail;   // [sequence][kv head][buffer][2][64][D]
    Q8Tail *state;         // [sequence][kv head]
    int nblk, Hkv;         // blocks of a (sequence, kv head)
};

// Rows in packed [T][Hkv][D] tensors or in a layer laid out [slot][head][position][D]:
// base + off[z] + (position - start[z]) * tok + head * head, in elements.
struct Q8RowsParams {
    Q8Layer layer;
    __nv_bfloat16 *rows[2];              // of K and V (write: read only; read: either may be null)
    int64_t tok, head;
    int nseq, seq0;                      // seq0: cache slot of launched sequence 0
    // A read for prefill attention: the codes of the first ntok rows (whole blocks) as they
    // are, with the factors of their blocks and of the rest of the sequence's tiles of 128
    // here, [launched sequence][head][factor_stride]; null otherwise.
    float4 *factors;
    int factor_stride;
    int start[kQ8MaxSeqPerLaunch], ntok[kQ8MaxSeqPerLaunch];
    int item0[kQ8MaxSeqPerLaunch + 1];   // first work item (block) of each launched sequence
    int64_t off[kQ8MaxSeqPerLaunch];
};
static_assert(sizeof(Q8RowsParams) <= 4096, "travels in the 4 KB of kernel parameters");

// A launched sequence: the position of its new token, its place in the cache, and its
// first CTA; each kv head has 2^log_S of them.
struct alignas(16) Q8Seq {
    int pos, slot, cta0, log_S;
};

struct Q8StepParams {
    Q8Layer layer;
    const __nv_bfloat16 *q, *k, *v;      // [batch][Hq|Hkv][D]
    const __nv_bfloat16 *wq, *wk;        // [D], or null: q and k are normed and rotated
    __nv_bfloat16 *out;
    __nv_bfloat16 *k_held, *v_held;      // the new rows as the step attends to them (may be null)
    const float2 *rope;                  // [cap][D/2] (cos, sin)
    const int32_t *pos_dev;              // device positions, by slot (null: Q8Seq::pos)
    int32_t *blocks;                     // [batch][Hkv][n_blocks]: receives the chosen blocks (null: all are)
    uint32_t *err;
    int n_blocks;
    int n_scores;                        // blocks of the longest sequence that has to choose (0: none has)
    int Hq, G, cap;
    int nseq, ctas, cluster;             // sequences, CTAs with work, CTAs of a cluster (a multiple of every S)
    int per_seq;                         // CTAs of each sequence where all have the same number, else 0
    int early;                           // nothing that may still run writes this layer
    int fault;                           // test hook: the last CTA of the first kv head sends nothing (FaultPlan)
    uint64_t wait_ns;                    // limit of every bounded wait
    float eps, scale_log2;               // scale_log2: log2(e) / sqrt(D)
    Q8Seq seq[kQ8MaxSeqPerLaunch];       // by falling S
};
static_assert(sizeof(Q8StepParams) <= 4096, "travels in the 4 KB of kernel parameters");

// Work items of a write of positions start .. end - 1: its blocks, of which the
// last goes with the first one's item when it is not complete and another one.
QA_HD int q8_write_items(int start, int end) {
    const int first = start / kQ8Block, last = (end - 1) / kQ8Block;
    return last - first + 1 - (last > first && end % kQ8Block != 0 ? 1 : 0);
}
// Of a read: its blocks.  For prefill attention: those of all tiles of 128 below end.
QA_HD int q8_tile_items(int end) { return (end + 127) / 128 * 2; }
QA_HD int q8_read_items(int start, int end) { return (end - 1) / kQ8Block - start / kQ8Block + 1; }

// The rows of a prefill: k1 as for K1, its cache pointers and strides the workspace's.
struct Q8PrefillRowsParams {
    K1Params k1;
    Q8Layer layer;
    uint32_t *tickets;                   // [launched sequence][kv head], zero between launches
    int seq0;                            // cache slot of launched sequence 0
    int item0[kMaxSeqPerLaunch + 1];     // first block of each launched sequence
};
static_assert(sizeof(Q8PrefillRowsParams) <= 4096, "travels in the 4 KB of kernel parameters");

cudaError_t launch_q8_prefill_rows(const Q8PrefillRowsParams &p, int D, cudaStream_t stream);
cudaError_t launch_q8_write(const Q8RowsParams &p, int D, cudaStream_t stream);
cudaError_t launch_q8_read(const Q8RowsParams &p, int D, cudaStream_t stream);
size_t q8_step_smem(const Q8StepParams &p, int D);  // shared memory of a CTA, bytes
cudaError_t launch_q8_decode(const Q8StepParams &p, int D, cudaStream_t stream);

// Shared with the other caches' host sides.
bool supported_geometry(int n_q_heads, int n_kv_heads, int head_dim);
LaunchOrder &launch_order();
StreamRef stream_ref(cudaStream_t stream, int device);
void note_launch(StreamRef &at, cudaStream_t stream);
cudaError_t synchronise_device();

}  // namespace qa
