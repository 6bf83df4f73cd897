// q8_tail.h -- which rows of a (sequence, kv head) of the 8-bit cache are kept in
// bf16, and what a write does to them.  Host and device; no CUDA dependency.
//
// A block of 64 positions gets its codes when its last row arrives, so the rows
// of a block that is not complete wait in bf16, in one of two buffers of 64 rows.
// The other one keeps the rows of the block before: a caller that steps back into
// it (speculative tokens that were not taken) finds them as they came.  Rows that
// are in neither buffer come back from the codes.
#pragma once

#ifdef __CUDACC__
#define QA_HD __host__ __device__ __forceinline__
#else
#define QA_HD inline
#endif

namespace qa {

constexpr int kQ8Block = 64;  // positions that share a scale

// Buffer i holds rows 0 .. rows[i] - 1 of block blk[i] (-1: nothing).  sealed: the
// block is complete, so that its codes, not these rows, are what the cache holds.
struct alignas(16) Q8Tail {
    int blk[2];
    short rows[2];
    short sealed[2];
};
static_assert(sizeof(Q8Tail) == 16, "read and written as one word");

// A write of positions start .. end - 1 (end > start).
struct Q8TailPlan {
    int from;       // buffer with rows 0 .. from_rows - 1 of the first block, -1: none
    int from_rows;  // at most the rows before start
    int dst;        // buffer that receives the rows of the last block, -1: none does
    Q8Tail next;
};

// keep: a block that the write completes leaves its rows in the buffer too (a decode
// step, which has them there; otherwise a complete block's rows go to the codes alone).
QA_HD Q8TailPlan q8_plan_tail(const Q8Tail &t, int start, int end, bool keep) {
    const int first = start / kQ8Block, before = start % kQ8Block;
    const int last = (end - 1) / kQ8Block;
    const int rest = end - last * kQ8Block;  // rows of the last block, 1 .. 64
    Q8TailPlan p;
    p.next = t;
    p.from = before > 0 && t.blk[0] == first ? 0 : before > 0 && t.blk[1] == first ? 1 : -1;
    p.from_rows = p.from < 0 ? 0 : t.rows[p.from] < before ? t.rows[p.from] : before;
    for (int i = 0; i < 2; ++i) {  // what the write overwrites is not kept
        if (t.blk[i] < first || t.blk[i] > last) continue;
        if (i == p.from && p.from_rows > 0) {
            p.next.rows[i] = static_cast<short>(p.from_rows);
            p.next.sealed[i] = last > first || rest == kQ8Block;
        } else {
            p.next.blk[i] = -1;
        }
    }
    p.dst = -1;
    if (rest < kQ8Block || keep) {
        if (last == first && p.from >= 0) {
            p.dst = p.from;
        } else {
            // An empty buffer, else one of a block further on (the caller stepped
            // back behind it), else that of the earlier block; never the first block's.
            const int *b = p.next.blk;
            p.dst = b[0] < 0 ? 0 : b[1] < 0 ? 1 : b[0] > last ? 0 : b[1] > last ? 1 : b[0] < b[1] ? 0 : 1;
            if (last > first && p.from >= 0 && b[p.from] >= 0) p.dst = 1 - p.from;
        }
        p.next.blk[p.dst] = last;
        p.next.rows[p.dst] = static_cast<short>(rest);
        p.next.sealed[p.dst] = rest == kQ8Block;
    }
    return p;
}

// The buffer that position `row` of block `blk` is read from, -1: the codes.
// raw: as the row came, if that is still there, though the block is complete.
QA_HD int q8_tail_of(const Q8Tail &t, int blk, int row, bool raw) {
    for (int i = 0; i < 2; ++i)
        if (t.blk[i] == blk && row < t.rows[i] && (raw || !t.sealed[i])) return i;
    return -1;
}

}  // namespace qa
