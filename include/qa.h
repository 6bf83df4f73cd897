/*
 * qa.h -- C ABI of the GB300 (sm_103a) attention hot path of a greedy
 * Qwen3-style decoder: per-head QK-RMSNorm + rotary embedding + KV-cache
 * append, causal grouped-query prefill attention (whole prompts or chunks
 * appended to what a layer holds; chunks of up to 8 tokens per sequence, such
 * as multi-token verify queries, run in the decode kernel's multi-token form)
 * and decode attention against a preallocated bf16 KV cache, with an optional
 * per-layer attention window.
 *
 * The arguments follow the pages' statement of the problem: a batch of
 * prompts with their lengths, one new token per sequence per decode step,
 * and a cache reset for every generate call (dryft-flash-infer agent guide,
 * sections "What is measured" and "Where the wins are"; the htn.dryft.ai
 * docs, "What to submit", for the Engine.generate contract of one token per
 * sequence per step, sequences kept in arrival order).  Following the
 * pegainfer PR #862 review ("add SM120 FlashInfer GDN prefill candidate",
 * summary and integration-boundary comments), the kernels sit behind a narrow
 * C ABI and an unsupported geometry or invalid argument fails validation with
 * a status code; there is no fallback path of any kind.
 *
 * Conventions for every entry point:
 *  - Tensors are bf16, contiguous, row-major, device pointers, 16-byte
 *    aligned.  The caller owns q, k, v, the norm weights and out; the library
 *    owns the cache, its lengths and its scratch until qa_cache_free.
 *  - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *    stream).  All device work is enqueued on it asynchronously; the call
 *    returns once it is enqueued.
 *  - Host-side validation runs before any launch; a call that returns an
 *    error status has enqueued nothing and changed no state.
 *  - Not thread-safe per cache: calls on one cache must come from one thread
 *    (or be serialised by the caller).
 */
#ifndef QA_H_
#define QA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QA_ABI_VERSION 7

typedef enum {
    QA_OK = 0,
    QA_ERR_INVALID_ARG = 1,        /* null pointer, out-of-range layer/batch/length */
    QA_ERR_UNSUPPORTED_SHAPE = 2,  /* head_dim not in {64,128}, Hq % Hkv != 0, group > 8 ... */
    QA_ERR_ALIGNMENT = 3,          /* a tensor pointer is not 16-byte aligned */
    QA_ERR_CAPACITY = 4,           /* a sequence would exceed the cache capacity (no eviction) */
    QA_ERR_STATE = 5,              /* the stream is being captured, and the call cannot be (qa_q4_prefill) */
    QA_ERR_CUDA = 6,               /* a CUDA runtime call failed (no device, launch error ...) */
    QA_ERR_DEVICE_TIMEOUT = 7,     /* a kernel gave up a bounded wait (reported by qa_get_device_error) */
    QA_ERR_DEVICE_BOUNDS = 8       /* a kernel saw a position outside the cache (qa_get_device_error) */
} qa_status;

/* Kernels counted by qa_stats (successful launches since qa_cache_alloc). */
enum {
    QA_KERNEL_NORM_ROPE_APPEND = 0, /* K1: fused QK-RMSNorm + RoPE + cache append (prefill rows) */
    QA_KERNEL_PREFILL_ATTN = 1,     /* K2: causal GQA flash attention, TMA + tcgen05 */
    QA_KERNEL_DECODE_ATTN = 2,      /* K3: fused norm/RoPE/append + split-KV decode + LSE merge
                                       (decode steps and short-chunk prefills) */
    QA_KERNEL_RESET = 3,            /* cache-length reset */
    QA_NUM_KERNELS = 4
};

/* Geometry of one cache: num_layers independent layer caches, each holding
 * max_batch sequences of up to `capacity` positions for n_kv_heads heads of
 * head_dim.  Supported: head_dim in {64, 128}; n_q_heads % n_kv_heads == 0
 * with group size n_q_heads / n_kv_heads in {1, 2, 4, 8}; capacity >= 1;
 * rope_theta > 0; rms_eps >= 0. */
typedef struct {
    int num_layers;
    int max_batch;
    int n_q_heads;
    int n_kv_heads;
    int head_dim;
    int capacity;
    float rope_theta;   /* rotary base; angle of pair i at position p is p * theta^(-2i/head_dim) */
    float rms_eps;      /* RMSNorm epsilon, added to the mean of squares */
} qa_config;

typedef struct qa_cache qa_cache; /* opaque */

/* Allocate a cache on the current CUDA device: K and V as bf16
 * [num_layers][max_batch][n_kv_heads][capacity][head_dim] (zero-filled),
 * int32 lengths [num_layers][max_batch] (all zero), an fp32 rotary table
 * [capacity][head_dim/2] of (cos, sin) built on the host in fp64,
 * per-sequence counters and an error word; the decode kernel's TMA tensor
 * maps (two per layer) are kept on the host.  Synchronous.
 * Errors: INVALID_ARG (cfg or out null, non-positive sizes),
 * UNSUPPORTED_SHAPE, CUDA (allocation failed; nothing is leaked). */
qa_status qa_cache_alloc(const qa_config *cfg, qa_cache **out);

/* Free everything qa_cache_alloc allocated.  Synchronises the device first.
 * NULL is accepted and ignored. */
qa_status qa_cache_free(qa_cache *cache);

/* Start a new generate call: every layer's lengths become 0 (device copy on
 * `stream`, host mirror immediately).  K/V memory is not cleared; no kernel
 * ever reads a slot at or beyond its sequence's length. */
qa_status qa_cache_reset(qa_cache *cache, void *stream);

/* Prefill one layer for `batch` prompts (sequence slots 0..batch-1), or the
 * next chunk of them: the L_b = prompt_lens[b] new tokens of sequence b take
 * positions P_b .. P_b + L_b - 1 after the P_b tokens the layer already holds
 * (P_b = 0 after a reset).
 * prompt_lens: HOST array [batch], each >= 0 with P_b + L_b <= capacity.
 * T = sum of L_b.  q: [T][Hq][D], k, v: [T][Hkv][D], packed in sequence order
 * (sequence b's tokens follow sequence b-1's).  q_norm_w, k_norm_w: [D].
 * out: [T][Hq][D]; it also serves as the staging buffer for the normed,
 * rotated queries, so it must not alias q, k or v.
 * Result: k' = RoPE(RMSNorm(k)) and v go to cache slots P_b..P_b+L_b-1, the
 * layer's lengths become P_b + L_b, and for the new token at position i
 * out[t][h] = sum_{j<=i} softmax_j(q'_t,h . K_j / sqrt(D)) V_j over sequence
 * b's cached keys 0..i, q' = RoPE(RMSNorm(q)), kv head h / (Hq/Hkv).
 * Work: when some L_b exceeds 8, K1 writes q' into out and k', v into the
 * cache, then K2 (one launch per 8 sequences) computes the attention.  K2
 * starts its set-up while K1 ends (programmatic dependent launch) and reads
 * or writes global memory only once the kernel before it has finished, so
 * the call is ordered after earlier work on the stream as a plain launch
 * would be.  When
 * every L_b is at most 8 (a verify step of speculative decoding, a short
 * append), the decode kernel's multi-token form does all of it in one launch
 * per 64 sequences that have new tokens (each streams its cache once for all
 * of its new tokens; counted as QA_KERNEL_DECODE_ATTN).  That form overlaps
 * the previous kernel on the stream like qa_decode_step, with the same
 * condition on q, k and v.
 * Errors: INVALID_ARG, ALIGNMENT, CAPACITY (P_b + L_b above capacity). */
qa_status qa_prefill(qa_cache *cache, int layer, int batch, const int32_t *prompt_lens,
                     const void *q, const void *k, const void *v,
                     const void *q_norm_w, const void *k_norm_w, void *out, void *stream);

/* One decode step of one layer: one new token for each of sequences
 * 0..batch-1, at position pos_b = current length of sequence b.
 * q: [batch][Hq][D], k, v: [batch][Hkv][D], weights [D], out: [batch][Hq][D].
 * One fused launch: RMSNorm + RoPE of q and k at pos_b, append of k' and v to
 * slot pos_b, attention of every q head over slots 0..pos_b (the new token
 * attends to itself) split over the key range (the splits of one sequence and
 * kv head form one thread-block cluster), log-sum-exp merge of the splits in
 * distributed shared memory, length += 1 (host copy and device lengths).
 * Positions come from the cache's host copy of the lengths and travel in the
 * launch parameters (one launch per 64 sequences).  Launches may overlap the
 * previous kernel on the stream (programmatic dependent launch): the step
 * reads q, k, v and the weights before that kernel has finished, so they must
 * not be written by the immediately preceding decode step or short chunk (its
 * out buffer in particular must not be this step's q, k or v).  A launch
 * lets the next one start at once, and each of its thread blocks waits for
 * the previous kernel before it exits; the library tracks, per stream, the
 * launches that can still be running when a new one starts (bounded by the
 * thread blocks the device holds at once) and makes the new launch read the
 * cache rows they append to its layer only after its wait.  Kernels of other
 * code enqueued between these calls on the same stream must not let their
 * successors start before they themselves have waited for their predecessor
 * (the usual use of programmatic dependent launch), and one that writes this
 * step's q, k, v or weights not before it has stored them: a kernel that signals
 * between its wait and its stores releases a step that reads what was there
 * before.  A kernel that never signals fulfils both.  For callers whose kernels
 * do not, see qa_set_early_reads.
 * Errors: INVALID_ARG, ALIGNMENT, CAPACITY (a sequence already holds
 * `capacity` tokens; nothing is evicted or wrapped), CUDA (a launch failed;
 * with more than 64 sequences the launches before it were enqueued and their
 * sequences have advanced, on the device and in the host copy). */
qa_status qa_decode_step(qa_cache *cache, int layer, int batch,
                         const void *q, const void *k, const void *v,
                         const void *q_norm_w, const void *k_norm_w, void *out, void *stream);

/* The same decode step with positions read from the DEVICE lengths, for
 * CUDA-graph capture: a captured step advances the lengths on the device at
 * every replay, so one graph serves every position.  (No counterpart in the
 * pages; it serves the NEXT item "CUDA-graph-captured multi-layer decode step".)
 * Arguments, layouts and ownership as qa_decode_step.  Differences:
 *  - the kernel reads lens[b] from the device: at once when no launch that may
 *    still be running writes this layer (the library's per-stream launch
 *    record says so; e.g. each layer of a captured multi-layer step), and
 *    then it overlaps the previous launch like qa_decode_step; otherwise after
 *    the previous kernel on the stream has finished.  The last kv-head group
 *    of each sequence sets lens[b] + 1 (a per-sequence counter, reset by
 *    qa_cache_reset);
 *  - the host copy of the lengths is not advanced (call qa_cache_sync_lengths
 *    before any call that uses it: qa_prefill, qa_decode_step, the split plan);
 *  - a sequence already at capacity is detected on the device: the step does
 *    nothing for that sequence and qa_get_device_error returns
 *    QA_ERR_DEVICE_BOUNDS;
 *  - the split count is planned for a full cache (capacity) under the cache's
 *    overlap setting (qa_cache_set_decode_overlap), so a captured step and the
 *    same step run eagerly give bit-identical results (any count is correct;
 *    it only sets the speed).
 * Capture requires that the first call on this device for this geometry ran
 * outside capture (it configures the kernel and caches the occupancy query).
 * Errors: INVALID_ARG, ALIGNMENT (host side); DEVICE_BOUNDS (device side). */
qa_status qa_decode_step_device_lengths(qa_cache *cache, int layer, int batch,
                                        const void *q, const void *k, const void *v,
                                        const void *q_norm_w, const void *k_norm_w, void *out,
                                        void *stream);

/* Sliding-window attention for one layer: from now on a token at position i
 * attends to keys max(0, i + 1 - window) .. i in qa_prefill and the decode
 * steps (the new token always included); window = 0 restores attention over
 * all earlier keys (the default).  The cache keeps every key (nothing is
 * evicted); the window only limits what is read.  (No counterpart in the
 * pages' kernels; it serves the NEXT item "sliding-window mask variant".)
 * Host-side only, takes effect for launches after the call.
 * Errors: INVALID_ARG (no such layer, window < 0). */
qa_status qa_cache_set_window(qa_cache *cache, int layer, int window);

/* How many consecutive decode-kernel launches (decode steps, short chunks)
 * the split plan lets run on the device at once.  A launch's split count S
 * is the largest (<= 16) for which `launches` launches' thread-block
 * clusters fit together, so that each launch streams its cache while the
 * next ones start (programmatic dependent launch).
 * Until this is called, each host-position launch chooses from the library's
 * record of the launches on its stream: 1 when nothing may still run beside
 * it (right after a prefill, a reset or a synchronisation through this
 * library), 2 when launches on its own layer may (a single-layer loop), and
 * up to 6 when only other layers' launches may (a loop over attention
 * layers), fewer while 6 would leave a launch a single split (on GB300 this
 * gave the best rate per step at batch 1 and 4 for caches of 512 to 16384
 * keys).  Kernels of other code are not in that record: a caller whose
 * decode launches are separated by other kernels (a model's projections
 * between the attention layers) gets the most splits per launch with 1.
 * Device-length steps always plan for that last case (or the number set
 * here), so a captured step and the same step run eagerly agree bit for bit.
 * Any value gives the same result up to the summation order of the split
 * merge.
 * Host-side only, takes effect for launches after the call.
 * Errors: INVALID_ARG (launches outside 1..8). */
qa_status qa_cache_set_decode_overlap(qa_cache *cache, int launches);

/* Whether the launches that overlap earlier kernels of their stream do so: decode
 * and sparse steps and short chunks on caches of any kind, process-wide.  on = 1 is
 * the default.  With 0 such a launch starts when everything before it on its stream
 * has finished, so it reads what that wrote, whenever it signalled; results are the
 * same, and a chain of steps loses their overlap.  Host-side only, takes effect for
 * launches after the call; a captured launch keeps what held at its capture.
 * Errors: INVALID_ARG (not 0 or 1). */
qa_status qa_set_early_reads(int on);

/* Copy one layer's device lengths into the host copy (synchronises `stream`),
 * after decode steps that advanced them on the device. */
qa_status qa_cache_sync_lengths(qa_cache *cache, int layer, void *stream);

/* ---- test and benchmark hooks ------------------------------------------ */

/* Device pointers of one layer's K, V ([max_batch][Hkv][capacity][D] bf16)
 * and lengths ([max_batch] int32), and the element strides of K/V for
 * (sequence, head, position, dim).  Any output pointer may be NULL. */
qa_status qa_cache_view(qa_cache *cache, int layer, void **k, void **v, int32_t **lens,
                        int64_t strides[4]);

/* Overwrite one layer's lengths (HOST array [max_batch], each in
 * [0, capacity]); synchronous with respect to `stream`.  Used to decode
 * against a cache filled through qa_cache_view. */
qa_status qa_cache_set_lengths(qa_cache *cache, int layer, const int32_t *lens_host,
                               void *stream);

/* Copy the host mirror of one layer's lengths into lens_host[max_batch]. */
qa_status qa_cache_lengths(qa_cache *cache, int layer, int32_t *lens_host);

/* Run only K1 of a prefill: like qa_prefill, but the normed, rotated queries
 * go to qprime_out [T][Hq][D] and no attention is computed. */
qa_status qa_prefill_transform(qa_cache *cache, int layer, int batch, const int32_t *prompt_lens,
                               const void *q, const void *k, const void *v,
                               const void *q_norm_w, const void *k_norm_w, void *qprime_out,
                               void *stream);

/* Run only the attention of a prefill (K2): for sequence b, the last
 * prompt_lens[b] positions the layer holds (appended earlier, e.g. by
 * qa_prefill_transform) attend causally to keys 0..own position (and the
 * layer's window), exactly as in qa_prefill.  qprime: [T][Hq][D] normed,
 * rotated queries of those tokens (qa_prefill_transform's output); out:
 * [T][Hq][D]; out may be qprime (in place, as qa_prefill does).  Always the
 * prefill kernel, whatever the lengths.  Splitting qa_prefill this way lets
 * each kernel be timed on its own.  The lengths are not changed.
 * Errors: INVALID_ARG (a prompt_lens[b] above what sequence b holds),
 * ALIGNMENT. */
qa_status qa_prefill_attend(qa_cache *cache, int layer, int batch, const int32_t *prompt_lens,
                            const void *qprime, void *out, void *stream);

/* Synchronise the device, read and clear the error word the kernels set when
 * a bounded wait expired or a position fell outside the cache.  Returns
 * QA_OK, QA_ERR_DEVICE_TIMEOUT or QA_ERR_DEVICE_BOUNDS; *detail (may be NULL)
 * receives the raw word: bits 0-7 kind, 8-15 kernel, 16-31 site. */
qa_status qa_get_device_error(qa_cache *cache, uint32_t *detail);

/* Failure-detection test hook.  Arms the next launch of `kernel`
 * (QA_KERNEL_PREFILL_ATTN, or QA_KERNEL_DECODE_ATTN: decode steps, short
 * chunks and qa_decode_step_noalloc, and those of a 4-bit or 8-bit cache), process-wide: in that launch one tile
 * copy is withheld (prefill: a V tile of the first thread block, or both
 * halves of it in the first CTA pair of the pair form; decode: the first cache
 * chunk of each block of the first sequence's first kv-head group that streams
 * any; a step on an 8-bit cache: what the last thread block of the first sequence's first
 * kv head sends to the others, if it has several), so a wait for it can never succeed, and every bounded
 * wait of the launch gives up after wait_us
 * microseconds (1 .. 2000000) instead of 2 s.  The waiting thread records
 * QA_ERR_DEVICE_TIMEOUT (kernel and site in the detail word) in the error
 * word that qa_get_device_error / qa_noalloc_get_device_error read, the block
 * waits (bounded) for its own copies in flight and for what its cluster peers
 * send it, frees its tensor memory and exits; that launch's outputs and the
 * cache slots it appends are undefined, everything else stays usable.
 * kernel = -1 disarms.  Nothing faults or hangs: every wait is bounded.
 * Errors: INVALID_ARG (another kernel index, wait_us out of range). */
qa_status qa_debug_arm_wait_timeout(int kernel, uint32_t wait_us);

/* Successful-launch counters per kernel (QA_KERNEL_*), proving which native
 * kernels ran (the launch-counter check of the pegainfer PR #862 review). */
qa_status qa_stats(qa_cache *cache, uint64_t launches[QA_NUM_KERNELS]);

/* Bytes of device memory the cache owns: K+V, and scratch (device lengths,
 * rotary table, error word). */
qa_status qa_memory_info(qa_cache *cache, uint64_t *kv_bytes, uint64_t *scratch_bytes);

/* Number of key-range splits qa_decode_step uses for the current lengths of
 * `layer` and `batch` sequences when it runs beside other layers' launches
 * (up to 6 launches unless set; see qa_cache_set_decode_overlap;
 * a pure host computation; a step launches one kernel per 64 sequences, and
 * this is the first one's count). */
int qa_decode_splits(qa_cache *cache, int layer, int batch);

/* ---- allocation-free decode step ----------------------------------------
 * The pages have no counterpart of this entry point.  It is for callers that
 * may not allocate device memory at all: engines that hand out every byte of
 * the GPU from their own arena and forbid any other allocation, and plug-ins
 * embedded in a host framework that owns the device allocator.  Such a caller
 * owns the cache memory and the lengths itself and passes them in.
 *
 * One decode step of one layer, computed by the same kernel body as
 * qa_decode_step: for each of sequences 0..batch-1 the new token's q and k are
 * RMS-normed and rotated at position positions[b], k' and v are written to
 * cache slot positions[b], and every query head attends over slots
 * 0..positions[b] (inclusive).
 *   cfg         geometry (num_layers is ignored; one layer is passed).
 *   positions   HOST int32 [batch]: current length of each sequence, which is
 *               the slot of its new token; each must be < capacity.  The
 *               caller advances its own lengths after the call.  The
 *               positions and their rotary values are copied into the
 *               launch's parameters at this call.
 *   k_cache, v_cache  DEVICE bf16 [max_batch][n_kv_heads][capacity][head_dim]
 *               of this layer, caller-owned, read and appended to.
 *   q, k, v, q_norm_w, k_norm_w, out: as in qa_decode_step.
 * Nothing is allocated: no cudaMalloc, cudaFree or allocating library call.
 * The kernel's only global scratch is its error word (the key-range splits
 * are merged in distributed shared memory), kept in a fixed 256-byte array in
 * the library's device code that every GPU loading the library holds until
 * the process exits.  The first call on a device looks up that array's
 * address (no allocation).
 * Every call shares the array: calls that may overlap on the GPU (different
 * streams without ordering) race on it.  The error word is zero at load and
 * is cleared only by qa_noalloc_get_device_error, so it keeps the first error
 * of any call since the last read.
 * Limits: batch <= 16 (the per-sequence positions and rotary values travel in
 * the kernel parameters), else QA_ERR_UNSUPPORTED_SHAPE.  Errors:
 * INVALID_ARG, UNSUPPORTED_SHAPE, ALIGNMENT, CAPACITY (a position >=
 * capacity), CUDA. */
qa_status qa_decode_step_noalloc(const qa_config *cfg, int batch, const int32_t *positions,
                                 void *k_cache, void *v_cache, const void *q, const void *k,
                                 const void *v, const void *q_norm_w, const void *k_norm_w,
                                 void *out, void *stream);

/* Read and clear the error word of qa_decode_step_noalloc on the current
 * device, after synchronising `stream` (the stream the steps ran on; calls on
 * other streams must have finished too).  Returns QA_OK,
 * QA_ERR_DEVICE_TIMEOUT or QA_ERR_DEVICE_BOUNDS; *detail (may be NULL)
 * receives the raw word (bits 0-7 kind, 8-15 kernel, 16-31 site).  Allocates
 * nothing: a 4-byte copy into host memory and a 4-byte memset.
 * Errors: CUDA. */
qa_status qa_noalloc_get_device_error(uint32_t *detail, void *stream);

/* ---- 4-bit cache ----------------------------------------------------------
 * A key/value cache whose rows are held in 4 bits a value and one scale byte
 * per 32 values: 4.25 bits instead of 16, so a decode step reads 3.76 times
 * fewer bytes.  (The pages have no counterpart.)
 *
 * Format.  A row (one position of one kv head) is cut into groups of 32
 * consecutive dimensions.  A group stands for the values (n - 8) * s, n its
 * codes in 0..15 and s the fp16 number whose upper byte is the group's scale
 * byte (5 exponent bits, 2 mantissa bits).  Quantising a row x, per group:
 * s is max|x| / 7 rounded to the nearest such number (ties to the even byte),
 * at most 56; n - 8 is x / s rounded to the nearest integer, halves away from
 * zero, held to -8..7; n = 8 where s = 0.  So magnitudes up to 392 keep the
 * full resolution, larger ones are held to 392 (448 below zero), and a group
 * whose largest magnitude is at most 7 * 2^-17 becomes zero (below 7 * 2^-14
 * the scale has fewer bits).  A group with a value that is not finite gets
 * scale byte 0x7f, which reads as NaN throughout.  Every value has at most 7
 * significant bits: bf16 holds it exactly, and a row that is read back is
 * exactly what attention saw.  Byte i of a row's codes holds dimension 2i in
 * its low four bits and 2i + 1 in its high four.
 *
 * The caller keeps the lengths: every call names the positions it is about
 * (HOST arrays, which travel in the launch parameters), so that a speculative
 * token is dropped by writing its position again.  A call reads only positions
 * below the ones it writes; rows that nothing wrote may hold anything.
 *
 * Conventions as above; a call on more than 64 sequences is several launches,
 * and an error of a later one leaves the earlier ones enqueued.  Calls may be
 * made with another device current; the
 * stream belongs to the cache's device.  qa_q4_append and qa_q4_read are
 * ordered on their stream like plain launches.  Decode steps, and in a prefill
 * the sequences of few tokens (qa_q4_prefill says which), overlap earlier
 * kernels of the stream like qa_decode_step, with the same conditions on other
 * code's kernels between the calls.  They read q, k, v and the weights before
 * an earlier decode step or prefill has finished: what such a call writes (out,
 * k_held, v_held) is no input of a later one unless another kernel or copy on
 * the stream that fulfils those conditions lies between them. */
typedef struct qa_q4_cache qa_q4_cache; /* opaque */

/* Kernels counted by qa_q4_stats. */
enum {
    QA_Q4_KERNEL_NORM_ROPE = 0,    /* K1, for geometries whose token does not fit K4's transform */
    QA_Q4_KERNEL_QUANTISE = 1,     /* K4: rows into the cache (a prefill's: with norm and rotation) */
    QA_Q4_KERNEL_DEQUANTISE = 2,   /* K4: rows out of the cache */
    QA_Q4_KERNEL_PREFILL_ATTN = 3, /* K2 on the workspace (and the join of its parts) */
    QA_Q4_KERNEL_DECODE = 4,       /* K5: decode steps and short chunks, 8 tokens a launch */
    QA_Q4_NUM_KERNELS = 5
};

/* Allocate a 4-bit cache on the current device, with the geometry that
 * qa_cache_alloc takes: codes [num_layers][max_batch][n_kv_heads][rows][D/2]
 * and scale bytes [...][rows][D/32] for K and for V (zero-filled; rows is the
 * capacity, rounded up to a multiple of 64), an error word, and the rotary
 * table (computed on the device; the caches of one device, rope_theta and
 * head_dim that are alive share one).  Synchronous.
 * What prefill attention needs beside them is allocated by the first
 * qa_q4_prefill that takes it, and kept: a bf16 workspace of K and V of
 * min(max_batch, 8) sequences of one layer, [slot][n_kv_heads][capacity][D],
 * and, at capacity 1024 or more, the fp32 sums of keys in parts (20 MB at D =
 * 128).  No other call allocates.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, CUDA. */
qa_status qa_q4_cache_alloc(const qa_config *cfg, qa_q4_cache **out);

/* Free it.  Synchronises the device first.  NULL is accepted and ignored. */
qa_status qa_q4_cache_free(qa_q4_cache *cache);

/* Attention window of one layer, as qa_cache_set_window. */
qa_status qa_q4_cache_set_window(qa_q4_cache *cache, int layer, int window);

/* Quantise rows as they are (keys already normed and rotated) into positions
 * start[b] .. start[b] + ntok[b] - 1 of sequences 0..batch-1.
 * k, v: [T][Hkv][D] packed in sequence order, T = sum of ntok.
 * k_held, v_held: both NULL, or [T][Hkv][D] that receive the values the cache
 * now holds (they may be k and v themselves).
 * Errors: INVALID_ARG, ALIGNMENT, CAPACITY. */
qa_status qa_q4_append(qa_q4_cache *cache, int layer, int batch, const int32_t *start,
                       const int32_t *ntok, const void *k, const void *v, void *k_held,
                       void *v_held, void *stream);

/* Read the same ranges back as bf16 rows [T][Hkv][D].  k_out or v_out may be
 * NULL (that tensor is not read), not both.
 * Errors: INVALID_ARG, ALIGNMENT, CAPACITY. */
qa_status qa_q4_read(qa_q4_cache *cache, int layer, int batch, const int32_t *start,
                     const int32_t *ntok, void *k_out, void *v_out, void *stream);

/* Whole prompts (start 0) or the next chunk of them: the ntok[b] new tokens of
 * sequence b take positions start[b] ..; the cache holds the earlier ones.
 * Tensors as qa_prefill: q [T][Hq][D], k, v [T][Hkv][D], weights [D], out
 * [T][Hq][D] (it stages the queries: no alias of q, k, v).
 * Result: RoPE(RMSNorm(k)) and v are quantised into their positions, and every
 * new token attends causally to what the cache then holds (its own rows as
 * held, too), within the layer's window.
 * Sequences with few new tokens (up to 16; up to 24 behind 512 cached
 * positions, at most a window of which count) take the decode kernel, 8 tokens
 * a launch, one launch per 64 sequences, with a decode step's condition on the
 * inputs.  The others take K4 and K2 through the cache's workspace, up to 8
 * sequences at a time: calls with such sequences on several streams wait for
 * each other, and they cannot be captured into a graph (QA_ERR_STATE).  In that
 * form a key or value that is not finite and that some new token of the call
 * sees can reach the others of its sequence, also those before it (as in
 * qa_prefill: the tensor cores multiply it by their weight of zero).  Otherwise
 * what a token does not see reaches none of its outputs, whatever it holds.
 * Errors: INVALID_ARG, ALIGNMENT, CAPACITY, STATE, CUDA. */
qa_status qa_q4_prefill(qa_q4_cache *cache, int layer, int batch, const int32_t *start,
                        const int32_t *ntok, const void *q, const void *k, const void *v,
                        const void *q_norm_w, const void *k_norm_w, void *out, void *stream);

/* One decode step: one new token for each of sequences 0..batch-1 at
 * positions[b] (HOST), which attends to positions 0..positions[b], within the
 * layer's window.  Tensors as qa_decode_step.
 * k_held, v_held: both NULL, or [batch][Hkv][D] that receive the new rows as
 * the cache holds them.  out, k_held and v_held must not alias q, k or v.
 * Errors: INVALID_ARG, ALIGNMENT, CAPACITY (a position at or above the
 * capacity), CUDA. */
qa_status qa_q4_decode_step(qa_q4_cache *cache, int layer, int batch, const int32_t *positions,
                            const void *q, const void *k, const void *v, const void *q_norm_w,
                            const void *k_norm_w, void *out, void *k_held, void *v_held,
                            void *stream);

/* The same with positions in DEVICE memory (int32 [batch]), read when the
 * previous kernel on the stream has finished: for graph capture, where the
 * caller advances them inside the graph.  A position outside 0..capacity-1
 * leaves its sequence alone and sets QA_ERR_DEVICE_BOUNDS
 * (qa_q4_get_device_error).  The split count is planned for a full cache.
 * Capture requires one earlier call of this shape outside capture. */
qa_status qa_q4_decode_step_device_positions(qa_q4_cache *cache, int layer, int batch,
                                             const int32_t *positions, const void *q, const void *k,
                                             const void *v, const void *q_norm_w,
                                             const void *k_norm_w, void *out, void *k_held,
                                             void *v_held, void *stream);

/* Device pointers of one layer's codes and scale bytes, and the strides of
 * (sequence, kv head, position) in rows: a row is D/2 bytes of codes and D/32
 * scale bytes.  Any output pointer may be NULL. */
qa_status qa_q4_cache_view(qa_q4_cache *cache, int layer, void **k_codes, void **k_scales,
                           void **v_codes, void **v_scales, int64_t strides[3]);

/* As qa_get_device_error. */
qa_status qa_q4_get_device_error(qa_q4_cache *cache, uint32_t *detail);

/* Successful launches per kernel (QA_Q4_KERNEL_*). */
qa_status qa_q4_stats(qa_q4_cache *cache, uint64_t launches[QA_Q4_NUM_KERNELS]);

/* Device bytes: codes and scale bytes, and the scratch that the cache comes to
 * use: error word and rotary table (which other caches may share), and the
 * workspace and the sums of parts, whether or not a call has taken them yet. */
qa_status qa_q4_memory_info(qa_q4_cache *cache, uint64_t *cache_bytes, uint64_t *scratch_bytes);

/* ---- 8-bit cache ----------------------------------------------------------
 * A key/value cache whose rows are held in 8 bits a value with one scale for each
 * block of 64 positions and kv head, and a decode step that attends to a few blocks
 * which a cheap score picks for its queries.  Against the 4-bit cache it holds 127
 * steps to each side instead of 7 and is 1.9 times smaller than bf16 instead of 3.76.
 * (The pages have no counterpart.)
 *
 * Format.  A block is 64 consecutive positions of one kv head, from a multiple of
 * 64.  When its last row is written the block is complete: its keys and its values
 * are each held as 64 x D integers n in -127..127 and one fp32 scale s, and stand for
 * n * s.  With a the largest magnitude in the block, s = a / 127 and n is x * (127 / a)
 * rounded to the nearest integer, halves to even; the two quotients and the product
 * are rounded to fp32.  A block with a < 2^-64 becomes zeros (s = 0), and one with a
 * value that is not finite reads as NaN throughout.
 * The rows of a block that is not complete are held in bf16 as they came, so what the
 * cache holds does not depend on how its rows were cut into calls.  A call sees the
 * rows that it brings itself in bf16, and complete blocks of earlier calls in 8 bits.
 *
 * The caller keeps the lengths: every call names the positions it is about, and a
 * speculative token is dropped by writing its position again.  Writing a position
 * of a block again begins that block anew from there: its earlier rows are needed as
 * they came.  The cache has them while the position lies in one of the last two blocks
 * of which it kept rows (the one being filled and the one before, as far as each was
 * not written as a whole at once); further back they are the block's values, rounded
 * to bf16.  A call reads only positions below the ones it writes; rows that nothing
 * wrote may hold anything.
 *
 * Conventions as above; a call on more than 64 sequences is several launches, and an
 * error of a later one leaves the earlier ones enqueued.  Calls may be made with
 * another device current; the stream belongs to the cache's device.  Outputs share no
 * byte with inputs or with each other (INVALID_ARG).
 * All calls but qa_q8_prefill may be captured into graphs, on one stream or on several
 * that wait for each other's events.  qa_q8_append, qa_q8_read and
 * qa_q8_prefill are ordered on their stream like plain launches.  Decode and sparse
 * steps overlap earlier kernels of the stream like qa_decode_step, with the same
 * conditions on other code's kernels between the calls: they read q, k, v and the weights
 * before the kernel in front of them has finished.  So a kernel that writes these does not
 * signal before it has stored them, and what a call of this library writes (out, k_held,
 * v_held, k_out, v_out) is no input of a later step unless another kernel or copy on the
 * stream that fulfils those conditions lies between them.  (With device positions, and
 * behind a call that writes the same layer, a step waits first.) */
typedef struct qa_q8_cache qa_q8_cache; /* opaque */

/* Kernels counted by qa_q8_stats. */
enum {
    QA_Q8_KERNEL_WRITE = 0,        /* K6: rows into the cache (a prefill's: with norm and rotation) */
    QA_Q8_KERNEL_READ = 1,         /* K6: rows out of the cache */
    QA_Q8_KERNEL_PREFILL_ATTN = 2, /* K2 on the workspace (and the join of its parts) */
    QA_Q8_KERNEL_DECODE = 3,       /* K7: decode steps */
    QA_Q8_KERNEL_SPARSE = 4,       /* K7: sparse steps */
    QA_Q8_NUM_KERNELS = 5
};

/* Allocate an 8-bit cache on the current device, with the geometry that
 * qa_cache_alloc takes, a capacity of at most 2^20 and at most 2^40 blocks in all: codes, scales, the least and
 * the largest code of each dimension of a block's keys, and per sequence and kv head
 * 2 x 64 rows of K and V in bf16 (zero-filled); an error word; and the rotary table
 * (shared as qa_q4_cache_alloc says).  Synchronous.
 * What prefill attention needs beside them is allocated by the first qa_q8_prefill,
 * and kept: the workspace that qa_q4_cache_alloc describes.  No other call allocates.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, CUDA. */
qa_status qa_q8_cache_alloc(const qa_config *cfg, qa_q8_cache **out);

/* Free it.  Synchronises the device first.  NULL is accepted and ignored. */
qa_status qa_q8_cache_free(qa_q8_cache *cache);

/* Write rows as they are (keys already normed and rotated) to positions start[b] ..
 * start[b] + ntok[b] - 1 of sequences 0..batch-1.
 * k, v: [T][Hkv][D] packed in sequence order, T = sum of ntok.
 * Errors: INVALID_ARG, ALIGNMENT, CAPACITY. */
qa_status qa_q8_append(qa_q8_cache *cache, int layer, int batch, const int32_t *start,
                       const int32_t *ntok, const void *k, const void *v, void *stream);

/* Read the same ranges as bf16 rows [T][Hkv][D]: n * s rounded to fp32 and then to
 * bf16 where the block is complete, else the row as it came.  k_out or v_out may be
 * NULL (that tensor is not read), not both.
 * Errors: INVALID_ARG, ALIGNMENT, CAPACITY. */
qa_status qa_q8_read(qa_q8_cache *cache, int layer, int batch, const int32_t *start,
                     const int32_t *ntok, void *k_out, void *v_out, void *stream);

/* Whole prompts (start 0) or the next chunk of them, with the arguments of
 * qa_q4_prefill: RoPE(RMSNorm(k)) and v are written to their positions, and every new
 * token attends causally to the earlier positions and to its own call's rows.  Rows
 * of earlier complete blocks enter the attention as n * s, not rounded to bf16.
 * All sequences go through the cache's workspace, up to 8 at a time: calls on several
 * streams wait for each other, and they cannot be captured into a graph (QA_ERR_STATE).
 * A key or value that is not finite and that some new token of the call sees can reach
 * the others of its sequence, also those before it (as in qa_prefill).  A single
 * new token is cheaper as a decode step.
 * Errors: INVALID_ARG, ALIGNMENT, CAPACITY, STATE, CUDA. */
qa_status qa_q8_prefill(qa_q8_cache *cache, int layer, int batch, const int32_t *start,
                        const int32_t *ntok, const void *q, const void *k, const void *v,
                        const void *q_norm_w, const void *k_norm_w, void *out, void *stream);

/* One decode step: one new token for each of sequences 0..batch-1 at positions[b]
 * (HOST), which attends to positions 0..positions[b].  Tensors as qa_decode_step.
 * q_norm_w and k_norm_w may both be NULL: q and k are then taken as they are (already
 * normed and rotated).
 * k_held, v_held: both NULL, or [batch][Hkv][D] that receive the new rows as the step
 * attends to them.
 * Weights of complete blocks are rounded to fp16: 2^-11 of a weight, or 2^-32 of the
 * largest where that is more.  A value's code carries an offset that is taken away again,
 * which costs 3.02 * 2^-17 of the block's largest value at most, in the block's share of
 * the weights.  A value that is not finite in a row held as it came makes its dimension of
 * the heads that see it infinite or NaN.
 * Errors: INVALID_ARG, ALIGNMENT, CAPACITY (a position at or above the capacity), CUDA. */
qa_status qa_q8_decode_step(qa_q8_cache *cache, int layer, int batch, const int32_t *positions,
                            const void *q, const void *k, const void *v, const void *q_norm_w,
                            const void *k_norm_w, void *out, void *k_held, void *v_held,
                            void *stream);

/* The same with positions in DEVICE memory (int32 [batch]), read when the previous
 * kernel on the stream has finished: for graph capture, where the caller advances
 * them inside the graph.  (So such steps do not overlap each other, unlike those with
 * host positions.)  A position outside 0..capacity-1 leaves its sequence alone and sets
 * QA_ERR_DEVICE_BOUNDS (qa_q8_get_device_error).  The split count is planned for a full
 * cache. */
qa_status qa_q8_decode_step_device_positions(qa_q8_cache *cache, int layer, int batch,
                                             const int32_t *positions, const void *q, const void *k,
                                             const void *v, const void *q_norm_w,
                                             const void *k_norm_w, void *out, void *k_held,
                                             void *v_held, void *stream);

/* A decode step whose token attends, for each kv head, to n_blocks of the complete
 * blocks before it and to the rows of the block that it is in itself (at positions
 * that are a multiple of 64 that is the new row alone).  The blocks are those of the
 * highest scores, the lower index first among equals.  With lo and hi the least and
 * the largest n of each dimension of the block's keys, s their scale, and c the queries
 * of the kv head's group as integers in -127..127 (one scale for the group, made like
 * n above), a block's score is
 *     s * sum over the group's heads and the dimensions of max(c lo, c hi),
 * the integer sum times s rounded to fp32.  The first and the last complete block, and
 * those with a key that is not finite, score infinity.  Queries that are not finite, or
 * all below 2^-64, have c = 0.
 * n_blocks: 1 .. ceil(capacity / 64).  blocks: int32 [batch][Hkv][n_blocks] in DEVICE memory, 4-byte
 * aligned; receives the chosen blocks in rising order, then -1 where there were fewer.
 * Everything else as qa_q8_decode_step. */
qa_status qa_q8_sparse_step(qa_q8_cache *cache, int layer, int batch, const int32_t *positions,
                            int n_blocks, const void *q, const void *k, const void *v,
                            const void *q_norm_w, const void *k_norm_w, void *out, int32_t *blocks,
                            void *k_held, void *v_held, void *stream);

/* The same with positions in DEVICE memory.  A sequence whose position is outside the
 * cache gets a list of -1. */
qa_status qa_q8_sparse_step_device_positions(qa_q8_cache *cache, int layer, int batch,
                                             const int32_t *positions, int n_blocks, const void *q,
                                             const void *k, const void *v, const void *q_norm_w,
                                             const void *k_norm_w, void *out, int32_t *blocks,
                                             void *k_held, void *v_held, void *stream);

/* As qa_get_device_error. */
qa_status qa_q8_get_device_error(qa_q8_cache *cache, uint32_t *detail);

/* Successful launches per kernel (QA_Q8_KERNEL_*). */
qa_status qa_q8_stats(qa_q8_cache *cache, uint64_t launches[QA_Q8_NUM_KERNELS]);

/* Device bytes, as qa_q4_memory_info. */
qa_status qa_q8_memory_info(qa_q8_cache *cache, uint64_t *cache_bytes, uint64_t *scratch_bytes);

/* Static description of a status code. */
const char *qa_status_str(qa_status status);

/* QA_ABI_VERSION of the loaded library. */
int qa_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QA_H_ */
