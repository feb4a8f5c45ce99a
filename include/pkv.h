/*
 * pkv.h -- paged KV cache append and packed varlen attention on one GB300.
 *
 * The problem (vllm-metal v0.4.0 release page, section "Replacing attention,
 * reusing the rest"): a serving step is flattened onto ONE packed query axis,
 * with cu_seqlens marking where each request's query tokens start; KV stays in
 * fixed-size pages located through per-request block tables; one attention
 * launch covers everything the scheduler packed into the step -- chunked
 * prefill chunks, decode tokens and speculative-verify windows.  The same page
 * ("What v0.4.0 adds", batched MTP) has verify windows ride in the packed
 * target batch, and ("Prefix caching on hybrid models") rows are written into
 * pools in place.
 *
 * Conventions shared by every call:
 *  - All tensors are dense and row-major; bf16 is IEEE bfloat16 bit patterns.
 *  - kv_pool:  bf16 [num_blocks][2][num_kv_heads][block_size][head_dim];
 *              index 1 of the second axis selects K (0) or V (1).  Each
 *              (block, K|V, head) slab is one contiguous block_size*head_dim run.
 *  - q, out:   bf16 [total_q][num_q_heads][head_dim], packed in sequence order.
 *  - k, v:     bf16 [num_tokens][num_kv_heads][head_dim] (this step's new tokens).
 *  - cu_q_lens [num_seqs+1] int32, cu_q_lens[0] = 0, non-decreasing;
 *    q_len(s) = cu_q_lens[s+1] - cu_q_lens[s].
 *  - context_lens [num_seqs] int32: keys of sequence s INCLUDING this step's
 *    new tokens (append first, then attend).  q_len(s) <= context_lens[s].
 *  - Causality: query i of sequence s sits at position ctx - q_len + i and sees
 *    keys 0 .. ctx - q_len + i.
 *  - GQA: query head hq reads KV head hq / (num_q_heads / num_kv_heads).
 *  - block_tables [num_seqs][max_blocks_per_seq] int32: logical block j of
 *    sequence s is physical block block_tables[s][j]; entries at or past
 *    ceil(ctx/block_size) are never read.  Several sequences may share blocks.
 *  - Supported: block_size 16, head_dim 64 or 128, num_q_heads a multiple of
 *    num_kv_heads with group size <= 16.  Anything else: PKV_ERR_UNSUPPORTED.
 *
 * Ownership and execution: the caller owns every buffer.  The library never
 * allocates device memory, keeps no per-call state between calls, and enqueues
 * work asynchronously on the caller's stream.  Device pointers must be
 * 16-byte aligned.
 *
 * Errors: host-detectable problems return a non-zero pkv_status before any
 * work is enqueued.  Problems only the device can see (a slot or block id
 * outside the pool, a plan that does not match the device metadata, a pipeline
 * wait that timed out) are written to *dev_status (int32, device memory; first
 * error wins; caller zeroes it and reads it after synchronising); the offending
 * token/block is skipped, nothing is read or written out of bounds, and no
 * kernel traps or asserts.  dev_status may be NULL to ignore them.
 */
#ifndef PKV_H_
#define PKV_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PKV_API __attribute__((visibility("default")))
#else
#define PKV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *pkv_stream;

typedef enum pkv_status {
  PKV_OK = 0,
  PKV_ERR_NULL = 1,          /* a required pointer is NULL */
  PKV_ERR_SHAPE = 2,         /* inconsistent sizes (cu_q_lens not monotone, ...) */
  PKV_ERR_RANGE = 3,         /* q_len > context_len, block id / slot out of range, ... */
  PKV_ERR_UNSUPPORTED = 4,   /* head_dim, block_size or group size not supported */
  PKV_ERR_WORKSPACE = 5,     /* plan or workspace buffer too small */
  PKV_ERR_CUDA = 6,          /* a CUDA runtime call failed (launch, attribute, ...) */
  PKV_ERR_DEVICE_CHECK = 7,  /* value written to *dev_status by a kernel */
  PKV_ERR_ALIGN = 8,         /* a device pointer is not 16-byte aligned */
  PKV_ERR_STATE = 9,         /* a call out of order (pkv_planner_post / pkv_planner_wait) */
  PKV_ERR_HOST_MEMORY = 10   /* host memory or a thread for the planner could not be had */
} pkv_status;

/* Device-side error codes written to *dev_status (first one wins). */
#define PKV_DEV_OK 0
#define PKV_DEV_BAD_SLOT 1       /* append: slot >= num_blocks*block_size (token skipped) */
#define PKV_DEV_BAD_BLOCK 2      /* attention: block id outside [0, num_blocks) (block skipped) */
#define PKV_DEV_TIMEOUT 3        /* a pipeline wait exceeded its bound (tile abandoned) */
#define PKV_DEV_PLAN_MISMATCH 4  /* device cu_q_lens/context_lens disagree with the plan */
#define PKV_DEV_BAD_POSITION 5   /* rotating append: position >= max_positions (token skipped) */
#define PKV_DEV_BAD_ROW 6        /* pages: a row index past the tables (that row left out) */
#define PKV_DEV_NO_BLOCKS 7      /* reserve: too few free blocks or table columns (nothing changed) */
#define PKV_DEV_BAD_COUNT 8      /* pages: a reference count that does not fit the tables */

typedef struct pkv_pool_desc {
  int32_t num_blocks;   /* physical blocks in kv_pool */
  int32_t block_size;   /* tokens per block; must be 16 */
  int32_t num_kv_heads; /* Hkv */
  int32_t head_dim;     /* D: 64 or 128 */
} pkv_pool_desc;

/* Summary of a step plan, written by pkv_plan_step. */
typedef struct pkv_plan_info {
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t total_q;
  int32_t num_decode_warps;  /* warps of the split-KV kernel; each streams an equal share of keys */
  int32_t num_decode_pieces; /* (row group, KV head, key range) pieces over all decode warps */
  int32_t num_merge_groups;  /* results combined from partials: decode (row group, KV head)
                                pairs whose keys span several pieces, then prefill sub-tiles
                                whose keys span several work items */
  int32_t num_partials;      /* decode partial-result slots (one per piece of a merge group) */
  int32_t num_prefill_tiles; /* tensor-core work items: a key range of two 128-token x 1-head
                                query tiles of one KV head */
  int32_t num_kernels;       /* kernel launches one pkv_paged_varlen_attention call makes */
  int32_t max_blocks_needed; /* max over sequences of ceil(context_len / block_size) */
  int32_t num_prefill_ctas;  /* persistent tensor-core CTAs (one per SM at most); each runs
                                an equal-cost range of the work items' key tiles */
  int32_t num_prefill_partials; /* prefill partial-result slots (128 rows each) */
  int32_t num_prefill_merges;   /* prefill merge groups (the last ones of num_merge_groups) */
  int32_t lookahead;            /* further decode steps the plan stays valid for (chained
                                   decode, pkv_plan_decode_chain); 0 for a single step */
  int32_t num_shared_ctas;      /* split-KV CTAs whose warp pairs each read blocks several row
                                   groups share once for two of them: a prefix several
                                   sequences share (needs host block tables), or a verify
                                   window wider than one row group */
  int32_t num_gather_rows;      /* query tokens listed by the tensor-core shared-prefix
                                   items (a prefix many query rows share is read once per
                                   128 rows on the tensor cores; needs host block tables) */
  int32_t merge_rows;           /* query rows of the largest decode merge group (its row
                                   group's tokens x the G heads of a KV head, <= 16; 0 when
                                   there is none): the merge launch covers that many rows
                                   of every decode group */
  int32_t num_shared_items;     /* shared-block items of those CTAs' warp pairs (each pair
                                   runs a chain of them, one after another) */
  int64_t kv_tokens;         /* sum of context_lens over sequences with q_len > 0 */
  int64_t decode_blocks;     /* (KV block, KV head) pairs the split-KV kernel attends, each
                                counted once: per sequence (however many row groups read
                                it), a prefix its shared-prefix CTAs read once per group,
                                a prefix gathered onto the tensor cores not at all */
  int64_t plan_bytes;        /* bytes of the plan buffer (host, then device copy) */
  int64_t workspace_bytes;   /* device workspace the attention call needs */
  int64_t gather_pairs;      /* (query row, key) pairs the tensor-core kernel computes for
                                gathered shared-prefix rows (row = token x query head) */
} pkv_plan_info;

/* Library version (major*10000 + minor*100 + patch). */
PKV_API int32_t pkv_version(void);

/* Human-readable name of a pkv_status or a PKV_DEV_* code. */
PKV_API const char *pkv_status_string(int32_t status);

/* Total kernel launches enqueued by this library since it was loaded. */
PKV_API int64_t pkv_kernel_launch_count(void);

/* Kernel ids for pkv_set_profile_events. */
#define PKV_KERNEL_APPEND 0
#define PKV_KERNEL_DECODE 1
#define PKV_KERNEL_MERGE 2
#define PKV_KERNEL_PREFILL 3
#define PKV_KERNEL_STATE 4
#define PKV_KERNEL_ROPE 5   /* pkv_rope_kv_append and pkv_rope_kv_append_fp8 */
#define PKV_KERNEL_STAGE 6  /* 8-bit attention: bf16 copies of the tensor-core sequences' blocks */
#define PKV_KERNEL_PAGES 7  /* every kernel of the fork, free, reserve and compact calls */
#define PKV_KERNEL_COPY 8   /* pkv_copy_blocks */
#define PKV_KERNEL_BEAM 9   /* pkv_beam_select: both kernels */
#define PKV_KERNEL_INDEX 10 /* pkv_update_block_index */
#define PKV_KERNEL_SELECT 11 /* pkv_select_blocks: both kernels */
#define PKV_KERNEL_SPARSE 12 /* pkv_paged_sparse_attention */

/*
 * Profiling hook (off by default).  After this call, every launch of kernel
 * `which` made FROM THE CALLING HOST THREAD is bracketed by
 * cudaEventRecord(start_event) / cudaEventRecord(stop_event) on the launch
 * stream, so the caller can time that kernel alone with its own events
 * (cudaEvent_t handles, created and owned by the caller).  When the launch
 * stream is being captured into a CUDA graph the records are made with
 * cudaEventRecordExternal, i.e. they become event-record nodes that fire on
 * every replay.  While any event is set, kernels launch without programmatic
 * dependent launch, so each one's interval holds that kernel alone.  Passing
 * NULL for both turns it off again.  Returns PKV_ERR_RANGE for an unknown
 * kernel id.
 */
PKV_API pkv_status pkv_set_profile_events(int32_t which, void *start_event, void *stop_event);

/*
 * KV append (the in-place row scatter of the "Prefix caching on hybrid
 * models" section, applied to the paged KV pool of "Replacing attention,
 * reusing the rest").
 *   For each token t < num_tokens with slot = slot_mapping[t]:
 *     slot < 0                        : padding, nothing written;
 *     0 <= slot < num_blocks*bs       : kv_pool[slot/bs][0][h][slot%bs][:] = k[t][h][:],
 *                                       kv_pool[slot/bs][1][h][slot%bs][:] = v[t][h][:]
 *                                       for every KV head h (raw 16-bit copies);
 *     slot >= num_blocks*bs           : token skipped, PKV_DEV_BAD_SLOT to *dev_status.
 *   k, v: device bf16 [num_tokens][Hkv][D]; slot_mapping: device int32 [num_tokens];
 *   kv_pool: device, layout above.  Two tokens with the same slot: unspecified
 *   which one lands.  num_tokens == 0 enqueues nothing and returns PKV_OK.
 */
PKV_API pkv_status pkv_paged_kv_append(const void *k, const void *v, const int32_t *slot_mapping,
                               int32_t num_tokens, void *kv_pool, const pkv_pool_desc *desc,
                               int32_t *dev_status, pkv_stream stream);

/* The position rotation of the two appends below. */
typedef struct pkv_rope {
  const float *cos_sin;     /* device fp32 [max_positions][rotary_dim]: of each position the
                               rotary_dim / 2 cosines, then the rotary_dim / 2 sines */
  const int32_t *positions; /* device int32 [num_tokens] */
  int32_t max_positions;
  int32_t rotary_dim;       /* elements of a head that are rotated, the first ones: a multiple
                               of 16, at most head_dim; the others pass through */
  int32_t interleaved;      /* 0: pairs (i, i + rotary_dim / 2); 1: pairs (2 i, 2 i + 1) */
} pkv_rope;

/*
 * KV append with the position rotation applied on the way (one kernel in place
 * of a rotation of q and k followed by pkv_paged_kv_append).
 *   For each token t < num_tokens at position p = positions[t], each head of q
 *   and k and each pair i < rotary_dim / 2 of its elements (a, b):
 *     a' = a cos[p][i] - b sin[p][i],   b' = b cos[p][i] + a sin[p][i],
 *   evaluated in fp32 (each product and sum rounded) and rounded once to bf16.
 *   q_out[t] gets the rotated q; with slot = slot_mapping[t] the pool gets the
 *   rotated k and v as pkv_paged_kv_append writes them:
 *     slot < 0                 : no k or v written (q is rotated all the same);
 *     slot >= num_blocks*bs    : k and v skipped, PKV_DEV_BAD_SLOT to *dev_status;
 *     p < 0                    : padding: nothing of the token is read or written,
 *                                and its slot may be anything;
 *     p >= max_positions       : the token skipped, PKV_DEV_BAD_POSITION (whatever
 *                                its slot).
 *   q: device bf16 [num_tokens][num_q_heads][D], k, v: [num_tokens][Hkv][D], the
 *   heads of a token contiguous, consecutive tokens q_stride, k_stride, v_stride
 *   elements apart (>= heads * D, a multiple of 8), so the three may be parts of
 *   one packed projection.  q_out: as q, with q_out_stride; it may be q itself
 *   with the same stride (rotation in place), and must not overlap the inputs
 *   otherwise.  num_q_heads = 0: k and v only (q, q_out ignored).
 *   Two tokens with the same slot: unspecified which one lands.  num_tokens == 0
 *   enqueues nothing.  Errors: PKV_ERR_UNSUPPORTED (rotary_dim), PKV_ERR_SHAPE
 *   (a negative count, a stride), PKV_ERR_NULL, PKV_ERR_ALIGN (16 bytes; 4 for
 *   positions and slot_mapping).
 *   The kernel lets its dependents launch only when it has finished, so
 *   pkv_paged_varlen_attention may follow it directly with q = q_out.
 */
PKV_API pkv_status pkv_rope_kv_append(const void *q, int64_t q_stride, const void *k,
                                      int64_t k_stride, const void *v, int64_t v_stride,
                                      const pkv_rope *rope, const int32_t *slot_mapping,
                                      int32_t num_tokens, int32_t num_q_heads, void *q_out,
                                      int64_t q_out_stride, void *kv_pool,
                                      const pkv_pool_desc *desc, int32_t *dev_status,
                                      pkv_stream stream);

/*
 * The 8-bit pool: kv_pool holds e4m3 values (8-bit floats, 4 exponent and 3
 * mantissa bits, largest 448) in the bf16 pool's layout, one byte a value, and
 * kv_scales, device fp32 [num_blocks][Hkv][2], the scale of the K (0) and V (1)
 * rows of each block and KV head: a stored c stands for c * scale.
 *
 * pkv_rope_kv_append_fp8 is pkv_rope_kv_append into such a pool (rope NULL: no
 * rotation; then num_q_heads must be 0).  For each block, KV head and K or V
 * that the step writes to, N being its new rows and `first` the smallest offset
 * among them:
 *   - rows below `first` are kept rows (the block is filled in order); when
 *     first is 0 the block is new, and its old scale and bytes do not matter;
 *   - the scale s stays when first > 0, s > 0 and 448 s >= max |N|; otherwise it
 *     becomes the smallest power of two s' >= 2^-64 with 448 s' >= max |N|
 *     (infinities and NaN are left out of the maximum) and each kept value c
 *     becomes c s / s'.  A stored s that is not positive and finite counts as 0:
 *     the rows kept under it become zeros;
 *   - the new rows are stored as x / scale.
 *   Both are evaluated in fp32 (exactly, when the scales are powers of two), rounded
 *   to nearest even and saturate at +-448; NaN stays NaN.  Rows
 *   past the new ones are left as they were.
 *   The new tokens of one block must lie within 16 consecutive tokens of the
 *   step (skipped tokens between them counted): a block is looked after by the
 *   thread block of its first one.  Tokens of one block further apart, like two tokens
 *   with the same slot, leave that block's values unspecified (where the kernel
 *   sees it, it skips the later token and reports PKV_DEV_BAD_SLOT).
 *   Other arguments, skipped tokens and errors as pkv_rope_kv_append; kv_scales
 *   must be 16-byte aligned.
 */
PKV_API pkv_status pkv_rope_kv_append_fp8(const void *q, int64_t q_stride, const void *k,
                                          int64_t k_stride, const void *v, int64_t v_stride,
                                          const pkv_rope *rope, const int32_t *slot_mapping,
                                          int32_t num_tokens, int32_t num_q_heads, void *q_out,
                                          int64_t q_out_stride, void *kv_pool, float *kv_scales,
                                          const pkv_pool_desc *desc, int32_t *dev_status,
                                          pkv_stream stream);

/*
 * Host step metadata (the per-threadgroup search over cu_seqlens that the
 * vllm-metal kernel performs, moved to the host where the scheduler already
 * holds the lengths).  Validates the lengths, splits each sequence's keys into
 * work tiles sized for num_sms SMs, assigns partial-result slots and sizes the
 * workspace.
 *   cu_q_lens, context_lens: HOST arrays (num_seqs+1 and num_seqs int32).
 *   num_sms: SMs of the target GPU; <= 0 asks the CUDA runtime for the SM count
 *   of the calling thread's current device (PKV_ERR_CUDA if there is none).
 *   plan: host buffer receiving plan_capacity bytes at most; may be NULL to
 *   query sizes only (info is always filled on success).
 * Returns PKV_ERR_WORKSPACE if plan is non-NULL and plan_capacity < info->plan_bytes,
 * PKV_ERR_HOST_MEMORY if the planner's own host scratch (reused per calling
 * thread, grown with the step) could not be allocated.
 * The plan buffer is opaque; upload it unchanged (e.g. cudaMemcpyAsync) before
 * the attention call that uses it.
 *
 * Compared with the plainest form of this call -- (cu_q_lens, context_lens,
 * num_seqs, num_q_heads, pool) -> plan -- three things are added, each because
 * the plan depends on it or the caller should own it: num_sms (the work is cut
 * into equal shares for that many SMs, so a plan is tied to a GPU size); a
 * caller-owned plan buffer with its capacity (the library allocates nothing,
 * host or device, and the caller picks pinned memory for an asynchronous
 * upload); and the pkv_plan_info summary, which the attention call takes in
 * place of parsing the device copy of the plan on the host.
 */
PKV_API pkv_status pkv_plan_step(const int32_t *cu_q_lens, const int32_t *context_lens, int32_t num_seqs,
                         int32_t num_q_heads, const pkv_pool_desc *desc, int32_t num_sms,
                         void *plan, int64_t plan_capacity, pkv_plan_info *info);

/*
 * Host planning on a worker thread.  A serving loop plans each step on the host
 * while it also queues that step's input copy and KV append (the append needs
 * no plan); with the planner on a thread of its own, the plan is computed while
 * the calling thread issues those calls instead of after them.  A pkv_planner
 * owns one thread and runs one pkv_plan_step_ex call at a time.
 *
 * pkv_planner_create: starts the thread.  After finishing a job the thread
 * polls for the next one for spin_us microseconds (so a loop whose steps follow
 * each other within that time hands a job over without a thread wake-up), then
 * sleeps until one is posted; spin_us <= 0 sleeps at once.  *out receives the
 * planner.  Errors: PKV_ERR_NULL (out NULL), PKV_ERR_RANGE (spin_us above
 * 1,000,000), PKV_ERR_HOST_MEMORY (the planner or its thread could not be
 * created).
 *
 * pkv_planner_destroy: finishes a posted job, stops and joins the thread and
 * frees the planner.  NULL is a no-op.  Not to be called concurrently with
 * another call on the same planner.
 *
 * pkv_planner_post: hands the thread one pkv_plan_step_ex call with these
 * arguments and returns at once.  Every pointer must stay valid, and the arrays
 * and *desc unchanged, until pkv_planner_wait has returned; the thread writes
 * plan and *info.  num_sms <= 0 is resolved here, on the calling thread's
 * current device (PKV_ERR_CUDA if there is none), not on the worker.
 * PKV_ERR_STATE if a job is already posted and not yet waited for; PKV_ERR_NULL
 * if planner is NULL.  The job's own errors come from pkv_planner_wait.  The
 * thread keeps its own planner scratch, as any calling thread does.
 *
 * pkv_planner_wait: waits (polling) until the posted job has finished and
 * returns its status, the value pkv_plan_step_ex would have returned; *info
 * and the plan buffer then hold its results.  PKV_ERR_STATE if no job is
 * posted; PKV_ERR_NULL if planner is NULL.
 *
 * post and wait on one planner are meant for one calling thread at a time.
 */
typedef struct pkv_planner pkv_planner;
PKV_API pkv_status pkv_planner_create(int32_t spin_us, pkv_planner **out);
PKV_API void pkv_planner_destroy(pkv_planner *planner);
PKV_API pkv_status pkv_planner_post(pkv_planner *planner, const int32_t *cu_q_lens,
                                    const int32_t *context_lens, int32_t num_seqs,
                                    int32_t num_q_heads, const pkv_pool_desc *desc,
                                    int32_t num_sms, int32_t steps, const int32_t *block_tables,
                                    int32_t max_blocks_per_seq, int32_t prefill_min_q, void *plan,
                                    int64_t plan_capacity, pkv_plan_info *info);
PKV_API pkv_status pkv_planner_wait(pkv_planner *planner);

/*
 * Bytes of device workspace the attention call needs for a plan (the same
 * value as info->workspace_bytes; 0 when the step needs none).  info NULL: 0.
 */
PKV_API size_t pkv_workspace_size(const pkv_plan_info *info);

/*
 * Stream-ordered copy of `bytes` bytes from src to dst on `stream`, for moving
 * a step's inputs and plan up and its output back without leaving this API:
 * host to device, device to host or device to device, the direction taken from
 * the pointers (unified addressing).  The call returns once the copy is queued;
 * it is asynchronous with respect to the host only when the host side is pinned
 * (page-locked) memory, and the caller keeps both buffers alive and unchanged
 * until the stream has passed the copy.  bytes == 0: nothing is queued.
 * Errors: PKV_ERR_RANGE (bytes < 0), PKV_ERR_NULL (a NULL pointer with
 * bytes > 0), PKV_ERR_CUDA (the runtime refused the copy).
 */
PKV_API pkv_status pkv_copy_async(void *dst, const void *src, int64_t bytes, pkv_stream stream);

/*
 * Plan for a chain of `steps` decode steps of the same batch (the vllm-metal
 * page's MLX engine, "Chained greedy decode": several decode steps built into
 * one graph and run with a single sync per chunk).  context_lens are those of
 * the first step; every later step adds each sequence's q_len tokens.  The one
 * plan serves all steps: it is sized for the last step's contexts, and each
 * step reads the current contexts from the device copy of context_lens, which
 * pkv_decode_advance moves on between steps.  Block tables must already hold
 * the blocks of the last step's contexts (info->max_blocks_needed counts them).
 * Sequences with q_len >= 64 (tensor-core prefill rows) are not supported here:
 * PKV_ERR_UNSUPPORTED.  steps < 1: PKV_ERR_RANGE.  Otherwise as pkv_plan_step;
 * info->lookahead = steps - 1.
 */
PKV_API pkv_status pkv_plan_decode_chain(const int32_t *cu_q_lens, const int32_t *context_lens,
                                         int32_t num_seqs, int32_t num_q_heads,
                                         const pkv_pool_desc *desc, int32_t num_sms, int32_t steps,
                                         void *plan, int64_t plan_capacity, pkv_plan_info *info);

/*
 * The general form of pkv_plan_step / pkv_plan_decode_chain: steps = 1 is a
 * single step, steps > 1 a decode chain.  block_tables, when not NULL, is a
 * HOST copy of the step's block tables ([num_seqs][max_blocks_per_seq] int32,
 * the same entries the device copy holds): the plan then also carries the
 * physical ids of the first blocks each split-KV warp reads, so its first copies
 * start without waiting for a block-table read, and sequences whose tables
 * start with the same physical blocks read those blocks once per work unit.
 * The attention kernel checks the carried ids against the device block tables;
 * on a disagreement it reports PKV_DEV_PLAN_MISMATCH and writes no result built
 * from the disagreeing blocks (those rows of out are left as they were).
 * prefill_min_q: sequences with at least this many query tokens run on the
 * tensor-core prefill kernel; 0 picks the default (64); a negative value keeps
 * every sequence on the split-KV kernel (both compute the same function).
 */
PKV_API pkv_status pkv_plan_step_ex(const int32_t *cu_q_lens, const int32_t *context_lens,
                                    int32_t num_seqs, int32_t num_q_heads,
                                    const pkv_pool_desc *desc, int32_t num_sms, int32_t steps,
                                    const int32_t *block_tables, int32_t max_blocks_per_seq,
                                    int32_t prefill_min_q, void *plan, int64_t plan_capacity,
                                    pkv_plan_info *info);

/*
 * Device-side move to the next step of a decode chain: for every sequence s
 * with q = cu_q_lens[s+1] - cu_q_lens[s] > 0, context_lens[s] += q and
 * slot_mapping[cu_q_lens[s] + i] = the pool slot of position
 * context_lens[s] - q + i (new value), i.e. block_tables[s][pos / block_size] *
 * block_size + pos % block_size, for i < q.  A position whose block lies
 * outside the table or the pool gets slot -1 (not written by the next append)
 * and PKV_DEV_BAD_BLOCK goes to *dev_status.  All arrays are device int32;
 * the kernel runs after the preceding attention call in stream order, so that
 * call read the old contexts.
 */
PKV_API pkv_status pkv_decode_advance(int32_t *context_lens, int32_t *slot_mapping,
                                      const int32_t *cu_q_lens, const int32_t *block_tables,
                                      int32_t max_blocks_per_seq, int32_t num_seqs,
                                      const pkv_pool_desc *desc, int32_t *dev_status,
                                      pkv_stream stream);

/*
 * Packed varlen attention over the paged KV pool ("Replacing attention,
 * reusing the rest": one launch sequence for prefill chunks, decode tokens and
 * verify windows):
 *   out[t][hq][:] = sum_p softmax_p(scale * q[t][hq] . K[p][hq/G]) V[p][hq/G]
 *   over the keys p visible to token t (causal rule above), K/V of position p
 *   read from kv_pool block block_tables[s][p/bs], offset p%bs.
 *   q, out: device bf16 (layout above).  cu_q_lens, context_lens, block_tables:
 *   DEVICE copies of the arrays the plan was built from.  plan_dev: device copy
 *   of the plan buffer; info: the host summary pkv_plan_step returned.
 *   workspace: device scratch of at least info->workspace_bytes (256-byte
 *   aligned; contents on entry do not matter).  Rows of sequences with
 *   q_len == 0 do not exist.  Accumulation is fp32; out is rounded once to bf16.
 *   Kernels are launched with programmatic stream serialisation: their launch
 *   overlaps the tail of the preceding kernel on the stream.  The first kernel
 *   of the call waits for that preceding kernel to complete
 *   (griddepcontrol.wait) before it reads kv_pool or the workspace; the plan,
 *   q, cu_q_lens, context_lens and block_tables are read before that wait.  A
 *   kernel that lets its dependents launch early
 *   (griddepcontrol.launch_dependents) and runs right before this call must
 *   therefore not write those five: this library's KV append writes only
 *   kv_pool; kernels that do not signal early are simply waited for.  Inside
 *   the call, when a step has both tensor-core and split-KV work, the
 *   tensor-core kernel lets the split-KV kernel launch only once its own wait
 *   has returned, so the split-KV kernel reads the pool without a further wait
 *   and starts on each SM the tensor-core kernel's persistent CTAs leave; it
 *   waits at its end instead, so every kernel of the call completes after the
 *   ones before it (the call as a whole is stream-ordered).
 */
PKV_API pkv_status pkv_paged_varlen_attention(const void *q, const int32_t *cu_q_lens,
                                      const int32_t *context_lens, const int32_t *block_tables,
                                      int32_t max_blocks_per_seq, const void *kv_pool,
                                      const pkv_pool_desc *desc, float scale,
                                      const pkv_plan_info *info, const void *plan_dev, void *out,
                                      void *workspace, int64_t workspace_bytes,
                                      int32_t *dev_status, pkv_stream stream);

/*
 * pkv_plan_step_ex with the work cut for the kernels of an 8-bit pool (more
 * split-KV warps an SM; beside a prefill they get SMs of their own).  The plan
 * serves a bf16 pool too, as any other plan serves an 8-bit pool: only the
 * division of the work differs, and with it the time.
 *
 * Workspace.  Over an 8-bit pool a tensor-core sequence takes bf16 copies of its
 * whole context, 8 ceil(context / 128) blocks of 64 Hkv D bytes (8 heads of 128:
 * 4 KB a key), sequences that share cached blocks one each; a gathered shared
 * prefix takes one for all its sequences.  This planner keeps the copies of a step
 * within 8 GiB beside those of its longest sequence: past that, the sequences with
 * the fewest query tokens a key run on the split-KV kernel (the same results, more
 * time).  A plan of the other planners has no such limit; pkv_plan_stage_fp8 says
 * what it needs.
 */
PKV_API pkv_status pkv_plan_step_fp8(const int32_t *cu_q_lens, const int32_t *context_lens,
                                     int32_t num_seqs, int32_t num_q_heads,
                                     const pkv_pool_desc *desc, int32_t num_sms, int32_t steps,
                                     const int32_t *block_tables, int32_t max_blocks_per_seq,
                                     int32_t prefill_min_q, void *plan, int64_t plan_capacity,
                                     pkv_plan_info *info);

/* pkv_planner_post for a pkv_plan_step_fp8 call (pkv_planner_wait returns its status). */
PKV_API pkv_status pkv_planner_post_fp8(pkv_planner *planner, const int32_t *cu_q_lens,
                                        const int32_t *context_lens, int32_t num_seqs,
                                        int32_t num_q_heads, const pkv_pool_desc *desc,
                                        int32_t num_sms, int32_t steps,
                                        const int32_t *block_tables, int32_t max_blocks_per_seq,
                                        int32_t prefill_min_q, void *plan, int64_t plan_capacity,
                                        pkv_plan_info *info);

/* What an 8-bit pool adds to a plan's summary, written by pkv_plan_stage_fp8. */
typedef struct pkv_fp8_info {
  int32_t staged_blocks;   /* bf16 copies of blocks the tensor-core kernel reads */
  int32_t max_rows;        /* query rows of the largest split-KV row group */
  int64_t workspace_bytes; /* workspace pkv_paged_varlen_attention_fp8 needs */
} pkv_fp8_info;

/*
 * What an 8-bit pool adds to a plan.  The split-KV kernel reads the 8-bit blocks
 * directly; the tensor-core kernel reads bf16 copies of the blocks its sequences
 * need, made in the workspace by the same attention call.
 *   plan, info: a finished HOST plan (pkv_plan_step and its relatives).
 *   stage_begin: HOST int32 [num_seqs + 1], written: sequence s's blocks 0, 1, ..
 *   get copies stage_begin[s], stage_begin[s] + 1, .. < stage_begin[s + 1] (none
 *   for a sequence the tensor cores do not read).
 * Upload stage_begin beside the plan.  When fp8->staged_blocks is 0 (no
 * tensor-core work) the attention call takes NULL for it.
 * Errors: PKV_ERR_NULL, PKV_ERR_SHAPE (info and plan disagree),
 * PKV_ERR_UNSUPPORTED (more copies than 32-bit row coordinates reach).
 */
PKV_API pkv_status pkv_plan_stage_fp8(const void *plan, const pkv_plan_info *info,
                                      int32_t *stage_begin, pkv_fp8_info *fp8);

/*
 * pkv_paged_varlen_attention over an 8-bit pool (layout above): the same step,
 * plan, rules and results, with K[p] = c_k scale_k and V[p] = c_v scale_v.
 * kv_scales: any positive normal values (not only powers of two).
 *   fp8, stage_begin: the summary pkv_plan_stage_fp8 wrote, and a DEVICE copy of
 *   its array.  workspace_bytes: at least fp8->workspace_bytes; a workspace serves one
 *   call at a time (calls that may overlap need one each).  A row group with
 *   more than fp8->max_rows rows, and tensor-core rows whose sequence stage_begin
 *   does not give all the copies they read, are reported (PKV_DEV_PLAN_MISMATCH)
 *   and not attended: their rows of out are left as they were.
 *   Rounding: on the split-KV kernel every stored value enters the products
 *   exactly (fp16); a key's weight w (1 for the row's largest) times its V scale
 *   is rounded to fp16 relative to the largest V scale v that the row group has
 *   read: by 2^-11 of itself where w scale >= 2^-28 v, by 2^-39 v below.  So V
 *   scales of one head within a factor 2^r of each other leave 2^-11 to every
 *   weight down to 2^(r - 28); a block whose V scale is 2^-28 of another's loses
 *   bits whatever its weight.  On the tensor-core kernel c * scale is rounded to
 *   bf16 (exact for power-of-two scales) and the weights to bf16, 2^-8.
 *   Accumulation is fp32; out is rounded once to bf16.
 *   Bytes of a block past its sequence's context are never used, whatever they
 *   hold, nor are the scales of a block that lies past it altogether (one that a
 *   chained plan's later steps will fill).  A NaN stored in a visible row reaches every row of out that sees it,
 *   and may reach rows of the same sequence's step that come before it.
 * Kernel order, early launches and errors as pkv_paged_varlen_attention (block
 * ids are read from the device tables); kv_scales is read after the wait for the
 * preceding kernel, as kv_pool is.
 */
PKV_API pkv_status pkv_paged_varlen_attention_fp8(
    const void *q, const int32_t *cu_q_lens, const int32_t *context_lens,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const void *kv_pool,
    const float *kv_scales, const pkv_pool_desc *desc, float scale, const pkv_plan_info *info,
    const void *plan_dev, const pkv_fp8_info *fp8, const int32_t *stage_begin, void *out,
    void *workspace, int64_t workspace_bytes, int32_t *dev_status, pkv_stream stream);

/*
 * State-row checkpoint (the vllm-metal v0.4.0 page, "Prefix caching on hybrid
 * models"): linear-attention layers keep a recurrent state per sequence that a
 * block table cannot address, so reusing a prefix means checkpointing that
 * state at block boundaries into state pools, and the rows are written in place
 * rather than by copying the pool.
 *   For each row i < num_rows with slot = dst_slots[i]:
 *     slot < 0               : nothing written;
 *     0 <= slot < num_slots  : pool[slot][0 .. row_bytes) = src[i][0 .. row_bytes)
 *                              (raw bytes);
 *     slot >= num_slots      : row skipped, PKV_DEV_BAD_SLOT to *dev_status.
 *   src: device [num_rows][row_bytes]; dst_slots: device int32 [num_rows];
 *   pool: device [num_slots][row_bytes].  row_bytes must be a positive multiple
 *   of 16 (else PKV_ERR_SHAPE) and src, pool 16-byte aligned (else
 *   PKV_ERR_ALIGN).  Bytes outside the written rows are untouched.  Two rows
 *   with the same slot: unspecified which one lands.  num_rows == 0 enqueues
 *   nothing and returns PKV_OK.
 */
PKV_API pkv_status pkv_state_checkpoint(const void *src, const int32_t *dst_slots,
                                        int32_t num_rows, void *pool, int64_t num_slots,
                                        int64_t row_bytes, int32_t *dev_status,
                                        pkv_stream stream);

/*
 * Pages of the cache: the block tables of the sequences a scheduler runs, and who
 * holds which block.  Conventions of the five calls below:
 *  - block_tables: device int32 [num_rows][max_blocks_per_seq], one row a sequence;
 *    row r's used entries are its first ceil(context_lens[r] / 16) (at most
 *    max_blocks_per_seq; a negative length counts as 0), the others are never read
 *    and are written only where a call says so.  An empty row has length 0.
 *  - ref_counts: device int32 [num_blocks]: how many used entries of all tables hold
 *    the block; 0: the block is free.  There is no other free list, and free blocks
 *    are always handed out from the lowest id up, so results do not depend on the
 *    order in which threads run.  A caller that holds a block outside the tables
 *    adds one to its count.
 *  - A used entry outside [0, num_blocks) is left out of the counts (copied as it is)
 *    and reported, PKV_DEV_BAD_BLOCK.  Counts that do not match the tables are
 *    reported where a call sees it, PKV_DEV_BAD_COUNT.
 *  - The kernels are launched with programmatic stream serialisation and wait for the
 *    preceding kernel before they touch anything; a call does not let its dependents
 *    launch before it has finished, and the lengths it wrote are visible to the whole GPU by
 *    then, so the appends, the selection and the sparse attention may follow directly.
 *    pkv_paged_varlen_attention, which reads the tables ahead of its wait too, follows an append.
 *
 * pkv_copy_blocks: whole blocks copied inside every array of `arrays` (each layer's
 * pool, the scales of 8-bit pools, block indexes: whatever is stored by block):
 *   for i < num_pairs (and i < *num_pairs_dev when that is not NULL):
 *     arrays[a].data row dst[i] = row src[i], raw bytes, row_bytes each.
 *   src, dst: device int32 [num_pairs]; a pair with a negative entry is skipped, one
 *   with an entry >= num_blocks too, PKV_DEV_BAD_BLOCK.  No dst may be another pair's
 *   src or dst (such blocks hold unspecified bytes).  num_pairs_dev: device int32.
 *   arrays: HOST array of num_arrays; data device, at least 4-byte aligned, row_bytes
 *   a positive multiple of 4 (16 of both for full speed).  One launch for every
 *   PKV_COPY_ARRAYS of them.  Nothing is enqueued for 0 pairs or arrays.
 */
#define PKV_COPY_ARRAYS 128
typedef struct pkv_block_array {
  void *data;        /* device, [num_blocks] rows */
  int64_t row_bytes;
} pkv_block_array;

PKV_API pkv_status pkv_copy_blocks(const pkv_block_array *arrays, int32_t num_arrays,
                                   int32_t num_blocks, const int32_t *src, const int32_t *dst,
                                   int32_t num_pairs, const int32_t *num_pairs_dev,
                                   int32_t *dev_status, pkv_stream stream);

/*
 * Fork: row i of new_tables (num_new rows) takes the used entries of row parents[i]
 * of block_tables (num_rows rows), and new_context_lens[i] its length.  The blocks
 * are shared, a partly filled last one too (pkv_reserve_blocks copies it when it is
 * to be written).  A negative parent gives an empty row; one >= num_rows too,
 * PKV_DEV_BAD_ROW.  Counts: with keep_parents = 1 every child adds one to each of its
 * blocks; with 0 the old rows end with the call (beam search's reordering: the new
 * tables take the old ones' place), which takes one off for each old row.  Both have
 * max_blocks_per_seq columns; the new arrays must not overlap the old ones.
 */
PKV_API pkv_status pkv_fork_sequences(const int32_t *parents, int32_t num_new,
                                      const int32_t *block_tables, const int32_t *context_lens,
                                      int32_t num_rows, int32_t max_blocks_per_seq,
                                      int32_t *ref_counts, int32_t num_blocks,
                                      int32_t keep_parents, int32_t *new_tables,
                                      int32_t *new_context_lens, int32_t *dev_status,
                                      pkv_stream stream);

/*
 * Free: each row listed in rows (device int32 [num_listed]; negative entries are
 * skipped, entries >= num_rows too, PKV_DEV_BAD_ROW) takes one off the counts of its
 * used entries and gets length 0; its entries stay as they are.  A row listed twice is
 * freed once.  A count that is 0 or less already stays and is reported.
 */
PKV_API pkv_status pkv_free_sequences(const int32_t *rows, int32_t num_listed,
                                      const int32_t *block_tables, int32_t *context_lens,
                                      int32_t num_rows, int32_t max_blocks_per_seq,
                                      int32_t *ref_counts, int32_t num_blocks,
                                      int32_t *dev_status, pkv_stream stream);

/*
 * Reserve: room for the new tokens of a step.  Row r gets n = cu_new[r + 1] -
 * cu_new[r] of them (0 where negative; device int32 [num_rows + 1]): its table the
 * blocks they need, context_lens[r] += n, and slot_mapping[cu_new[r] + i] the slot of
 * position context_lens[r] + i (old length), for the append.  Entries of slot_mapping
 * before cu_new[0] or from cu_new[num_rows] on (a step padded to num_tokens) get -1,
 * which the append skips; entries past num_tokens are not written.  num_rows == 0 enqueues
 * nothing: slot_mapping stays as it is, and a caller that appends all the same fills it with -1
 * (the Python call does).
 *   A partly filled last block that other rows hold too is not written to: the row
 *   takes a new block in its place, copy_src[r] and copy_dst[r] say which (-1 where
 *   there is none), for a pkv_copy_blocks before the append.  When every holder of such
 *   a block gets new tokens in this call, the last of those rows keeps it.  New blocks
 *   go to the rows in order, to each its copy first.
 *   When the free blocks or a table's columns do not suffice (PKV_DEV_NO_BLOCKS), a partly
 *   filled block is outside the pool (PKV_DEV_BAD_BLOCK) or its count is below the number of
 *   rows that write to it (PKV_DEV_BAD_COUNT), nothing changes, every slot and pair is -1
 *   and that is reported.
 *   workspace: device, 16-byte aligned, pkv_pages_workspace_size(num_rows, num_blocks)
 *   bytes, contents do not matter; one call at a time.  num_rows > 8192:
 *   PKV_ERR_UNSUPPORTED.
 */
PKV_API size_t pkv_pages_workspace_size(int32_t num_rows, int32_t num_blocks);
PKV_API pkv_status pkv_reserve_blocks(const int32_t *cu_new, int32_t *block_tables,
                                      int32_t *context_lens, int32_t num_rows,
                                      int32_t max_blocks_per_seq, int32_t *ref_counts,
                                      int32_t num_blocks, int32_t *slot_mapping,
                                      int32_t num_tokens, int32_t *copy_src, int32_t *copy_dst,
                                      void *workspace, int64_t workspace_bytes,
                                      int32_t *dev_status, pkv_stream stream);

/*
 * Compact: the blocks in use (count != 0) move to ids 0 .. L - 1, L being how many
 * there are.  The i-th block in use with id >= L goes to the i-th free id below L:
 * copy_src[i], copy_dst[i] (device int32 [num_pairs_max], -1 past the last pair;
 * num_pairs_max >= num_blocks / 2 holds every case, fewer: PKV_ERR_SHAPE), their number
 * to *num_pairs (device int32), for a pkv_copy_blocks.  new_tables gets the used entries
 * renamed, new_ref_counts the counts at the new ids.  new_tables may be block_tables and
 * new_ref_counts ref_counts (in place).  A used entry of a block whose count is 0 and whose
 * id is >= L keeps its id, PKV_DEV_BAD_COUNT.  A caller that holds blocks outside the tables
 * renames them by the pairs.  workspace as for pkv_reserve_blocks.
 */
PKV_API pkv_status pkv_compact_blocks(const int32_t *block_tables, const int32_t *context_lens,
                                      int32_t num_rows, int32_t max_blocks_per_seq,
                                      const int32_t *ref_counts, int32_t num_blocks,
                                      int32_t *new_tables, int32_t *new_ref_counts,
                                      int32_t *copy_src, int32_t *copy_dst,
                                      int32_t num_pairs_max, int32_t *num_pairs, void *workspace,
                                      int64_t workspace_bytes, int32_t *dev_status,
                                      pkv_stream stream);

/*
 * Beam search's selection.  For request b and its beam k (row r = b num_beams + k of
 * logits, vocab entries, row_stride elements apart) every token t is a candidate with
 *   score = cum_scores[r] + logits[r][t] - log(sum_u exp(logits[r][u]));
 * a beam with finished[r] != 0 (finished may be NULL: none) has one candidate,
 * pad_token with score cum_scores[r], and its logits are not read.  The num_select
 * best candidates of each request, by score, then beam, then token, go to scores
 * (fp32), tokens and parents (int32; r, the row index), [num_requests][num_select].
 *   Within a beam candidates are ranked by their logits, between beams by the score to
 *   39 bits or more (of a log-sum accumulated in 32).  Candidates whose score is not finite
 *   in fp32 (masked logits of -inf; every one of a beam whose logits hold NaN or +inf, or with a
 *   cum_scores that is not finite) are never selected; finite logits may have any size.  Where
 *   too few candidates remain, score -inf, token -1 and parent -1 fill the rest.  parents is
 *   what pkv_fork_sequences takes.
 *   logit_type: PKV_BF16, PKV_FP16 or PKV_FP32; logits aligned to their type.
 *   num_select <= 128, num_beams <= 1024, vocab >= 1.  workspace: device, 16-byte
 *   aligned, pkv_beam_workspace_size(...) bytes, contents do not matter; one call at a
 *   time.  scores, tokens and parents must not overlap the inputs.  The first kernel waits
 *   for the preceding one before it reads anything.
 */
#define PKV_BF16 0
#define PKV_FP16 1
#define PKV_FP32 2
PKV_API size_t pkv_beam_workspace_size(int32_t num_requests, int32_t num_beams, int32_t vocab,
                                       int32_t num_select);
PKV_API pkv_status pkv_beam_select(const void *logits, int32_t logit_type, int64_t row_stride,
                                   const float *cum_scores, const uint8_t *finished,
                                   int32_t num_requests, int32_t num_beams, int32_t vocab,
                                   int32_t num_select, int32_t pad_token, float *scores,
                                   int32_t *tokens, int32_t *parents, void *workspace,
                                   int64_t workspace_bytes, pkv_stream stream);

/*
 * Attention over selected blocks of a bf16 pool, for contexts too long to be read
 * whole at every step.  A block index holds, for each block and KV head, bounds of its
 * keys in 8 bits:
 *   index: device int8 [num_blocks][Hkv][2][D], index_scales: device fp32
 *   [num_blocks][Hkv].  With s the scale, the smallest power of two >= 2^-64 with
 *   |K| <= 127 s for every key of the block, lo = floor(min K / s) and
 *   hi = ceil(max K / s) by element: lo s <= K <= hi s.  (Keys' infinities and NaN
 *   count as 0.)
 *
 * pkv_update_block_index makes the rows of the blocks a step has written to, after
 * its append (and rotates nothing: it reads the keys back from the pool):
 *   slot_mapping as the append's: a block is taken to hold the rows up to its
 *   largest slot of the step; its bounds are made anew from those rows, so a slot
 *   written again after rejected tokens shrinks them again.  The tokens of one block must lie within
 *   16 consecutive ones of the step.  Negative slots are skipped, slots past the pool too,
 *   PKV_DEV_BAD_SLOT.
 */
PKV_API pkv_status pkv_update_block_index(const void *kv_pool, const pkv_pool_desc *desc,
                                          const int32_t *slot_mapping, int32_t num_tokens,
                                          int8_t *index, float *index_scales,
                                          int32_t *dev_status, pkv_stream stream);

/*
 * Selection, for each query token t (at position p of its sequence) and KV head h, of
 * num_select of its blocks 0 .. p / 16: all of them if there are no more; otherwise
 * the first sink_blocks, the last recent_blocks (that of p among them) and, of the
 * rest, those with the largest scores, ties to the lower block.
 *   Score: an upper bound, but for the rounding of q below, of the sum over the group's heads
 *   of q . k over the keys of the block.  With u the smallest power of two with |q| <= 2047 u
 *   in the group (infinities and NaN count as 0), P and N the sums over the heads of the
 *   positive and the negative elements of q / u, each rounded to an integer (to even):
 *     score = float(sum_d P[d] hi[d] + N[d] lo[d]) * index_scale,
 *   an integer rounded once to fp32 and scaled: the same number in any order.
 *   Every token reads its blocks' index rows for itself, so long chunks are for
 *   pkv_paged_varlen_attention: with 64 blocks of 32 / 8 heads, D = 128, selection and
 *   attention are faster up to some 64 tokens at 32768 keys and 400 at 131072.
 *   q: device bf16 [total_q][num_q_heads][D]; the group (num_q_heads / Hkv) is at most 16.
 *   cu_q_lens, context_lens, block_tables: DEVICE arrays as pkv_paged_varlen_attention
 *   takes them.  selected: device int32 [total_q][Hkv][num_select]: logical blocks,
 *   ascending, then -1.  1 <= recent_blocks, 0 <= sink_blocks, their sum <= num_select.
 *   max_blocks_per_seq > 2^30: PKV_ERR_UNSUPPORTED.
 *   A block id outside the pool has score -inf, PKV_DEV_BAD_BLOCK.  A token past cu_q_lens'
 *   last entry gets -1 throughout; so does every token of a sequence whose context is shorter
 *   than its window or has more blocks than the table columns, PKV_DEV_PLAN_MISMATCH.
 *   workspace: device, 16-byte aligned; any size from pkv_select_workspace_size(1, ...)
 *   on serves (fewer bytes than pkv_select_workspace_size(total_q, ...): the tokens in
 *   several passes); contents do not matter, one call at a time.
 *   cu_q_lens and context_lens may be read before the preceding kernel of the stream has
 *   completed (one that lets its dependents launch early must not write them; none of this
 *   library does); everything else is touched after it.
 */
PKV_API size_t pkv_select_workspace_size(int64_t total_q, int32_t num_kv_heads,
                                         int32_t max_blocks_per_seq);
PKV_API pkv_status pkv_select_blocks(const void *q, const int32_t *cu_q_lens,
                                     const int32_t *context_lens, const int32_t *block_tables,
                                     int32_t max_blocks_per_seq, int32_t num_seqs,
                                     int64_t total_q, int32_t num_q_heads, const int8_t *index,
                                     const float *index_scales, const pkv_pool_desc *desc,
                                     int32_t num_select, int32_t sink_blocks,
                                     int32_t recent_blocks, int32_t *selected, void *workspace,
                                     int64_t workspace_bytes, int32_t *dev_status,
                                     pkv_stream stream);

/*
 * Attention of each query token, group by group, over the keys of its selected blocks
 * that it sees:
 *   out[t][hq][:] = sum_p softmax_p(scale * q[t][hq] . K[p][h]) V[p][h],  h = hq / G,
 *   over the positions p <= the token's, p / 16 in selected[t][h].
 *   With every block of its context selected a token's result is that of
 *   pkv_paged_varlen_attention, but for the rounding of its weights.  selected: as
 *   pkv_select_blocks writes it, or a caller's own choice in any order (entries outside the
 *   token's blocks are skipped; one that is there twice counts twice).  A block id outside the
 *   pool is skipped, PKV_DEV_BAD_BLOCK.  A token that sees no key gets zeros; one past
 *   cu_q_lens' last entry is left as it was; so is every token of a sequence whose context is
 *   shorter than its window or has more blocks than the table columns, PKV_DEV_PLAN_MISMATCH.
 *   num_q_heads / Hkv <= 16.  Weights go into the product with V as two bf16 parts (2^-14 of a
 *   weight at most is lost), sums are fp32, out is rounded once to bf16.  Bytes of a visible
 *   block past the token's position do not reach its row.  out may be q itself, and must not
 *   overlap the inputs otherwise.  The lengths may be read before the preceding kernel has
 *   completed, everything else is touched after it.
 *   The next kernel may be launched while this one runs: out must not be the q of a
 *   pkv_paged_varlen_attention directly behind it (this call and the selection wait).
 */
PKV_API pkv_status pkv_paged_sparse_attention(const void *q, const int32_t *cu_q_lens,
                                              const int32_t *context_lens,
                                              const int32_t *block_tables,
                                              int32_t max_blocks_per_seq, int32_t num_seqs,
                                              int64_t total_q, int32_t num_q_heads,
                                              const int32_t *selected, int32_t num_select,
                                              const void *kv_pool, const pkv_pool_desc *desc,
                                              float scale, void *out, int32_t *dev_status,
                                              pkv_stream stream);

/*
 * Size of the fixed scratch array used by pkv_paged_varlen_attention_noalloc
 * (16 MiB).  Every GPU that loads this library holds these bytes until the
 * process exits.
 */
#define PKV_NOALLOC_SCRATCH_BYTES (16 * 1024 * 1024)

/*
 * pkv_paged_varlen_attention without a workspace argument, for callers that
 * cannot allocate device memory (no cudaMalloc available or allowed: a plugin
 * that is handed only the step's tensors, a path where an allocation could
 * block or fail, a runtime that pre-budgets all device memory).  The pages have
 * no counterpart to this call; it exists only for such callers.
 *
 * Same arguments, computation and results as pkv_paged_varlen_attention; the
 * caller still passes every input and the output.  The split-KV partial
 * results go to a fixed array in the library's device image
 * (PKV_NOALLOC_SCRATCH_BYTES), so this call allocates nothing: no cudaMalloc,
 * no cudaFree, no allocating library routine.
 *  - Returns PKV_ERR_WORKSPACE, before anything is enqueued, when the step
 *    needs more scratch than that (info->workspace_bytes >
 *    PKV_NOALLOC_SCRATCH_BYTES); plan such steps with more SMs' worth of
 *    smaller splits or use pkv_paged_varlen_attention.
 *  - The calling thread's current device must be the device of the buffers and
 *    the stream.  The first call made with a given device current looks up the
 *    array's device address on that device (cudaGetSymbolAddress, which may
 *    load the library's module there); make that first call before any stream
 *    capture.  The address is kept for the life of the loaded library: after
 *    cudaDeviceReset on a device, do not call this entry point on that device
 *    again in the same process (the kept address would be stale).
 *  - All calls on a device share the one array and it keeps the last call's
 *    contents.  Nothing in it needs to start at zero (every partial is written
 *    before it is read).  Calls whose work overlaps on the GPU (different
 *    streams, or different host threads, without ordering between them) race
 *    on the array and give wrong results: order them on one stream.
 */
PKV_API pkv_status pkv_paged_varlen_attention_noalloc(
    const void *q, const int32_t *cu_q_lens, const int32_t *context_lens,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const void *kv_pool,
    const pkv_pool_desc *desc, float scale, const pkv_plan_info *info, const void *plan_dev,
    void *out, int32_t *dev_status, pkv_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H_ */
