// q4_internal.h -- definitions shared by the host side and the kernels of the
// 4-bit key/value cache (parameter blocks, limits, launchers).  Not part of the
// public ABI.
#pragma once

#include <cuda_runtime.h>

#include "launch_order.h"
#include "q4_plan.h"
#include "qa_internal.h"

namespace qa {

// Kernel numbers in the error word of a 4-bit cache.
constexpr uint32_t kKernQ4Rows = 4, kKernQ4Decode = 5;

// Values of one row that share a scale.
constexpr int kQ4Group = 32;
// Rows of a (sequence, kv head) are padded to a multiple of this, so that the
// decode kernel's bulk copies of whole chunks stay inside the allocation and
// start on 16-byte boundaries.
constexpr int kQ4RowPad = 64;

// The row kernels (quantise, dequantise) work on tokens start[b] .. start[b] +
// ntok[b] - 1 of each launched sequence.  A row of 16-bit values is addressed
// by (sequence, token of the call, kv head): base + off[b] + token * tok +
// head * head_stride, in elements, which covers packed [T][Hkv][D] rows as well
// as a layer laid out [sequence][head][position][D].
struct Q4RowsParams {
    uint8_t *codes[2], *scales[2];       // layer base of K and V
    const __nv_bfloat16 *src[2];         // quantise: the rows of K and V
    __nv_bfloat16 *dst[2];               // the rows' values as the cache holds them (may be null)
    int64_t src_tok, src_head, dst_tok, dst_head;
    int64_t row_seq, row_head;           // cache strides in rows: sequence, head
    int nseq, Hkv, nblocks, kv_first, kv_count;  // kv_first/count: K (0) and V (1) served
    int unroll;                          // tokens per lane group of a block: 4 or 8
    int seq0;                            // cache slot of launched sequence 0
    int beside;                          // dequantise: starts beside the kernel before it, signals at once
    int start[kQ4MaxSeqPerLaunch], ntok[kQ4MaxSeqPerLaunch];
    int hidden[kQ4MaxSeqPerLaunch];      // dequantise: rows below this position come out as zeros
    int block0[kQ4MaxSeqPerLaunch + 1];  // first token block of each launched sequence
    int64_t src_off[kQ4MaxSeqPerLaunch], dst_off[kQ4MaxSeqPerLaunch];
};
static_assert(sizeof(Q4RowsParams) <= 4096, "travels in the 4 KB of kernel parameters");

// Tokens of one head that one warp quantises or dequantises: `unroll` per lane
// group, D/8 lanes each.
__host__ __device__ constexpr int q4_block_tokens(int D, int unroll) { return unroll * (32 / (D / 8)); }

// The transform of a prefill's rows (K1) with the keys and values quantised on
// the way: k1 as for K1, its cache pointers and strides those of the bf16
// workspace, which receives the values that the codes stand for.
struct Q4PrefillRowsParams {
    K1Params k1;
    uint8_t *codes[2], *scales[2];       // layer base of K and V
    int64_t row_seq, row_head;           // cache strides in rows
    int seq0;                            // cache slot of the first sequence
    int parts;                           // shares of a token (set at launch)
};
static_assert(sizeof(Q4PrefillRowsParams) <= 4096, "travels in the 4 KB of kernel parameters");


// A launched sequence: the slot of its first new token, its place in the cache,
// its new tokens and the first of their rows in q, k, v and out.
// Its CTAs are cta0 .. of a mixed launch, S for each kv head and head group; each
// of the S merges a run of E outputs (a multiple of 32); inv_S: ceil(2^32 / S), 0 for 1.
struct alignas(16) Q4Seq {
    int pos, slot, ntok, row0;
    int cta0, S, E;
    uint32_t inv_S;
};

struct Q4DecodeParams {
    uint8_t *kc, *ks, *vc, *vs;          // layer base: codes and scale bytes of K and V
    const __nv_bfloat16 *q, *k, *v;      // packed rows of the new tokens
    const __nv_bfloat16 *wq, *wk;        // [D]
    __nv_bfloat16 *out;
    __nv_bfloat16 *k_held, *v_held;      // the new rows as the cache holds them (may be null)
    const float2 *rope;                  // [cap][D/2] (cos, sin)
    const int32_t *pos_dev;              // device positions (null: pos[])
    uint32_t *err;
    int64_t row_seq, row_head;           // cache strides in rows
    int Hq, Hkv, G, HG, cap;
    int groups;                          // Hkv * HG
    int B, ctas, cluster;                // sequences, CTAs with work, CTAs of a cluster
    int mixed;                           // 0: every sequence has `cluster` splits, grid (cluster, groups, B)
    float eps, scale_log2;               // scale_log2: log2(e) / sqrt(D)
    int window;                          // attention window in keys (0: all earlier keys)
    int guard;                           // rows below each first new slot that a running launch may write
    int fault;                           // test hook: withhold the first stage of cluster 0 (FaultPlan)
    uint64_t wait_ns;                    // limit of every bounded wait
    int early;                           // 1: signal the next launch at once, 0: after the wait
    Q4Seq seq[kQ4MaxSeqPerLaunch];       // the launched sequences
    uint8_t seq_of[kQ4MaxSeqPerLaunch * kQ4MaxSplits];  // mixed: the sequence of `groups` CTAs at a time
};
static_assert(sizeof(Q4DecodeParams) <= 4096, "travels in the 4 KB of kernel parameters");

cudaError_t launch_q4_quantise(const Q4RowsParams &p, int D, cudaStream_t stream);
// False when a token of this geometry does not fit the kernel's stages: the
// rows then go through K1 and launch_q4_quantise.
bool q4_prefill_rows_fits(int Hq, int Hkv, int D);
cudaError_t launch_q4_prefill_rows(const Q4PrefillRowsParams &p, int D, cudaStream_t stream);
cudaError_t launch_q4_dequantise(const Q4RowsParams &p, int D, cudaStream_t stream);
// HPC heads x TPS tokens per CTA (TPS = 1, or 8 / HPC for launches of several tokens).
cudaError_t launch_q4_decode(const Q4DecodeParams &p, int D, int HPC, bool multi, cudaStream_t stream);
// How many clusters of S decode CTAs the current device holds at once, for S =
// 1..kQ4MaxSplits (entry 0 unused); asked for once per device, null on error.
const int *q4_cluster_capacities(int D, int HPC, bool multi);

// Shared with the bf16 cache's host side.
bool encode_kv_map(CUtensorMap *m, void *base, int D, int L, int Hkv, int cap, int box_rows);
bool encode_q_map(CUtensorMap *m, void *base, int D, int Hq, int T);
bool supported_geometry(int n_q_heads, int n_kv_heads, int head_dim);
LaunchOrder &launch_order();
// `stream` of `device` as the launch record takes it now: captured or not.
StreamRef stream_ref(cudaStream_t stream, int device);
void note_launch(StreamRef &at, cudaStream_t stream);
cudaError_t synchronise_device();
// Rotary table [capacity][D/2] of (cos, sin), in fp64, stored as fp32.
void fill_rope_table(float2 *tab, int capacity, int D, float theta);

}  // namespace qa
