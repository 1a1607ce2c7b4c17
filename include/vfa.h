/*
 * vfa.h -- C ABI of libvfa: variable-length FlashAttention forward and paged
 * GQA decode for NVIDIA GB300 (sm_103a), with the operators around them
 * (query / key norm and rotation, a 4-bit paged cache, page operations, a
 * cache bounded by window and sinks or by eviction).
 *
 * Conventions shared by every entry point:
 *   - Every pointer argument named as a device buffer is a CUDA device
 *     address on the current device, allocated and owned by the caller.  The
 *     library never allocates, frees or retains caller memory, and keeps no
 *     pointer after a call returns.
 *   - Calls are asynchronous: they enqueue work on `stream` (NULL means the
 *     legacy default stream) and return.  Results are ready when the stream
 *     has reached that point.
 *   - Host-detected errors (null or misaligned pointers, unsupported sizes,
 *     a too-small workspace, a device that is not compute capability 10.3)
 *     return a non-zero vfa_status immediately and enqueue nothing.
 *     vfa_last_error() then describes the problem.
 *   - Data errors that only the device can see (cu_seqlens that are not a
 *     valid prefix sum, a block id outside the pool, a tile count above the
 *     tile capacity) never fault or trap: the kernels record a status code
 *     in a device status word, skip the offending work and leave its outputs
 *     untouched.  vfa_read_status() fetches that word.
 *   - bf16 means IEEE bfloat16 (1-8-7); f32 is IEEE binary32.
 */
#ifndef VFA_H
#define VFA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A CUDA stream handle (the same object as cudaStream_t / CUstream). */
typedef struct CUstream_st *vfa_stream_t;

typedef enum {
    VFA_OK = 0,
    VFA_ERR_INVALID_ARG = 1,   /* host: null/misaligned pointer, bad size        */
    VFA_ERR_UNSUPPORTED = 2,   /* host: a size this build does not implement     */
    VFA_ERR_ARCH = 3,          /* host: the current device is not sm_103         */
    VFA_ERR_CUDA = 4,          /* host: a CUDA runtime call failed               */
    VFA_ERR_BAD_SEQLENS = 5,   /* device: cu_seqlens not a valid prefix sum      */
    VFA_ERR_BAD_BLOCK = 6,     /* device: block id or tile count out of range    */
    VFA_ERR_TIMEOUT = 7,       /* device: a bounded wait inside a kernel expired */
    VFA_ERR_WORKSPACE = 8,     /* device: the work list does not fit the workspace */
    VFA_ERR_NO_PAGES = 9       /* device: fewer free pages than the call needs     */
} vfa_status;

/* Message for the last non-OK status returned on the calling host thread. */
const char *vfa_last_error(void);

/* Library version string, e.g. "vfa 0.1 sm_103a". */
const char *vfa_version(void);

/* ------------------------------------------------------------------------ */
/* Variable-length attention forward                                         */
/* ------------------------------------------------------------------------ */

/*
 * Workspace bytes vfa_varlen_fwd needs for these sizes (an upper bound that
 * holds for any cu_seqlens with these totals).  The first int32 of the
 * workspace is the call's device status word (see vfa_read_status).
 */
size_t vfa_varlen_fwd_workspace_bytes(int batch, int total_q, int total_k, int num_heads,
                                      int head_dim);

/*
 * Tile shape the forward uses for `head_dim`: q tile rows (*block_q), key
 * tile rows (*block_k), and whether one work item holds two q tiles
 * (*pair_tiles, 0 or 1).  The work list is built over these tiles.
 * Returns VFA_ERR_UNSUPPORTED for a head_dim this build does not implement.
 */
vfa_status vfa_varlen_fwd_tile_shape(int head_dim, int *block_q, int *block_k, int *pair_tiles);

/*
 * Exact softmax(scale * Q K^T, optional causal mask) V over packed
 * variable-length sequences, plus the per-(token, head) log-sum-exp.
 *
 * Defined by "Varlen Flash Attention Implementation Plan" (rustytorch),
 * Task 1 Step 1 (kernel preconditions, packed layout, masks, online-softmax
 * recurrence and the out / lse epilogue) and Task 2 Step 1 (the CPU
 * reference it must agree with).  The plan's kernel takes one block per
 * (global q tile, head); this library instead builds a per-sequence q-tile
 * work list on the device and covers every query row.
 *
 * q            device bf16 [total_q, num_heads, head_dim], packed row-major.
 * k, v         device bf16 [total_k, num_kv_heads, head_dim]; query head h
 *              reads kv head h / (num_heads / num_kv_heads) (grouped-query
 *              attention; num_kv_heads == num_heads is the plan's layout).
 * cu_seqlens_q device int32 [batch + 1]: 0, running sums of the q lengths;
 *              cu_seqlens_q[batch] == total_q.  Sequence b owns q rows
 *              [cu_seqlens_q[b], cu_seqlens_q[b+1]).
 * cu_seqlens_k device int32 [batch + 1], the same for keys/values.
 * total_q, total_k  the tensors' first extents (needed on the host to describe
 *              the tensors to the TMA engine).
 * max_seqlen_q an upper bound on every q length (checked on the device).
 * softmax_scale the factor applied to q.k before the softmax.
 * causal       0: no mask; 1: top-left causal mask in local positions --
 *              local key j is visible to local query i iff j <= i (the
 *              plan's kernel); 2: bottom-right -- j <= i + Lk_b - Lq_b, so the
 *              last query sees every key (a query block at the end of a longer
 *              key sequence) and rows with i + Lk_b - Lq_b < 0 see none.
 *              Other values: VFA_ERR_INVALID_ARG.
 * window_left  < 0: no window.  >= 0 (needs causal 1 or 2, else
 *              VFA_ERR_INVALID_ARG): a sliding window -- local key j is
 *              visible to local query i only if j >= i + off - window_left
 *              as well (off = 0 top-left, Lk_b - Lq_b bottom-right), so each
 *              query sees at most window_left + 1 keys ending at its
 *              diagonal.  The pages name sliding-window masks among the
 *              varlen variants without defining one; this is the reading
 *              taken.
 * out          device bf16 [total_q, num_heads, head_dim]: out = sum_j p_j v_j /
 *              sum_j p_j, rounded to nearest even; 0 for a query with no
 *              visible key.
 * lse          device f32 [total_q, num_heads]: natural-log sum of
 *              exp(scale * q.k_j) over visible keys; -FLT_MAX when there is
 *              none.
 * workspace    device scratch of at least vfa_varlen_fwd_workspace_bytes()
 *              bytes, 256-byte aligned; reused across calls; calls that share
 *              one workspace must be stream-ordered.
 *
 * Supported: head_dim in {64, 128, 256}; num_heads >= 1, a multiple of
 * num_kv_heads >= 1; batch >= 1; q, k,
 * v, out 16-byte aligned.  Sequences of length 0 are allowed (no rows, or no
 * keys).  Device-detected: cu_seqlens not starting at 0, decreasing, not
 * ending at total_q / total_k, or a q length above max_seqlen_q
 * -> VFA_ERR_BAD_SEQLENS, nothing written to out / lse.
 */
vfa_status vfa_varlen_fwd(const void *q, const void *k, const void *v,
                          const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                          int total_q, int total_k, int max_seqlen_q, int batch,
                          int num_heads, int num_kv_heads, int head_dim, float softmax_scale,
                          int causal, int window_left, void *out, float *lse, void *workspace,
                          size_t workspace_bytes, vfa_stream_t stream);

/*
 * vfa_varlen_fwd with sinks: where a window hides keys, the first sink_tokens
 * keys of each sequence stay visible.  Local key j is visible to local query
 * i iff j <= i + off and (j >= i + off - window_left or j < sink_tokens), off
 * as in vfa_varlen_fwd.  Only the key tiles of the sinks and of the window are
 * read.
 *
 * sink_tokens  >= 0 (else VFA_ERR_INVALID_ARG), any number: 0, or no window
 *              (window_left < 0), is vfa_varlen_fwd.
 * Other arguments, results, workspace and errors as in vfa_varlen_fwd.  k and
 * v are finite: a hidden key's weight is zero, but the product with it is
 * formed for the other rows' sake.
 */
vfa_status vfa_varlen_fwd_sinks(const void *q, const void *k, const void *v,
                                const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                int total_q, int total_k, int max_seqlen_q, int batch,
                                int num_heads, int num_kv_heads, int head_dim,
                                float softmax_scale, int causal, int window_left,
                                int sink_tokens, void *out, float *lse, void *workspace,
                                size_t workspace_bytes, vfa_stream_t stream);

/*
 * vfa_varlen_fwd with q and k given as FP8 E4M3 codes (1 byte each: 1 sign,
 * 4 exponent bits with bias 7, 3 mantissa bits, no infinities), each tensor
 * with one descale factor: element value = descale * code.  v stays bf16.
 * The plan names FP8 kernel configuration types without content; this is
 * the reading taken.  S = q.k is formed by the tensor core's FP8 product
 * (exact products, fp32 accumulation) and scaled by softmax_scale *
 * descale_q * descale_k; everything after S is as in vfa_varlen_fwd.
 *
 * q_fp8        device uint8 [total_q, num_heads, head_dim] E4M3 codes.
 * k_fp8        device uint8 [total_k, num_kv_heads, head_dim] E4M3 codes.
 * descale_q, descale_k  finite, > 0 (else VFA_ERR_INVALID_ARG).
 * Other arguments, outputs, workspace and errors as in vfa_varlen_fwd;
 * head_dim 64, 128 or 256 (else VFA_ERR_UNSUPPORTED).
 */
vfa_status vfa_varlen_fwd_fp8(const void *q_fp8, const void *k_fp8, const void *v,
                              const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                              int total_q, int total_k, int max_seqlen_q, int batch,
                              int num_heads, int num_kv_heads, int head_dim, float softmax_scale,
                              float descale_q, float descale_k, int causal, int window_left,
                              void *out, float *lse, void *workspace, size_t workspace_bytes,
                              vfa_stream_t stream);

/*
 * vfa_varlen_fwd without a caller workspace.  The pages have no counterpart:
 * this entry point exists for callers that cannot allocate device memory --
 * code on a real-time or callback thread that must not enter the allocator,
 * runtimes that give kernels a fixed memory plan and forbid other
 * allocations, plugins that only receive their inputs' and outputs' pointers.
 *
 * Same arguments, results and device checks as vfa_varlen_fwd, minus the
 * workspace: the scratch (status word, work list, scheduler records) lives
 * in one 1 MiB array inside the library, which every GPU that loads the
 * library keeps reserved until the process exits.  It allocates nothing and
 * frees nothing.
 *
 * device_status  nullable device int32 [1]: receives the call's status word
 *                (VFA_OK or VFA_ERR_BAD_SEQLENS ...), copied on `stream`.
 *
 * Limits and rules:
 *   - a problem whose vfa_varlen_fwd_workspace_bytes() exceeds 1 MiB returns
 *     VFA_ERR_UNSUPPORTED and enqueues nothing.  That size is exactly
 *     round256(round256(256 + 32 * num_heads * (total_q / 128 + batch))
 *     + 56 * (batch + 1)) bytes (integer division; round256 rounds up to a
 *     multiple of 256): the status word and counters, 32 bytes per work
 *     item, then 14 int32 of scheduler records per sequence;
 *   - the first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) and remembers it together with the current CUDA
 *     context; a call under another context (after cudaDeviceReset, or a
 *     thread with a context of its own) looks it up again.  Make such first
 *     calls before any stream capture;
 *   - all calls share the one array: calls whose work can overlap on the GPU
 *     (different streams without ordering) race and give undefined results.
 *     Each call rewrites every scratch word it reads, so stream-ordered calls
 *     are independent.
 */
vfa_status vfa_varlen_fwd_noalloc(const void *q, const void *k, const void *v,
                                  const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                  int total_q, int total_k, int max_seqlen_q, int batch,
                                  int num_heads, int num_kv_heads, int head_dim,
                                  float softmax_scale, int causal, int window_left, void *out,
                                  float *lse, int32_t *device_status, vfa_stream_t stream);

/*
 * The device tile scheduler alone (the first kernel vfa_varlen_fwd runs),
 * writing into caller buffers so the work list can be inspected.
 *
 * A tile is q tile i (local rows [i*block_q, min(Lq_b, (i+1)*block_q))) of
 * sequence b and head h; it visits the key tiles [first, end) that hold a
 * key its rows may see, and its cost is end - first.  Without a window
 * first = 0 and end = ceil(Lk_b / block_k), or with a causal mask
 * ceil(clamp(min(Lq_b, (i+1)*block_q) + off, 0, Lk_b) / block_k), off = 0 for
 * causal == 1 and Lk_b - Lq_b for causal == 2; a window (window_left >= 0,
 * as in vfa_varlen_fwd) gives first = floor(max(0, i*block_q + off -
 * window_left) / block_k); a tile that sees no key has first = end = 0.
 * The tiles of one (b, h) stay together; groups are ordered by their
 * largest cost, then total cost (descending), then (b, h); inside a group
 * by cost descending, then i (with a window: by i descending).  With
 * pair_tiles != 0 two consecutive tiles of a group form one item (what
 * vfa_varlen_fwd uses for head_dim <= 128); otherwise each tile is one
 * item.  Each item is eight int32: (b, i_a, h, end_a, i_b, end_b, first_a,
 * first_b), with i_b = -1 and end_b = first_b = 0 when the second slot is
 * empty.  Sequences with Lq_b == 0 give no items.
 *
 * block_k must be a power of two and block_q a multiple of block_k
 * (VFA_ERR_UNSUPPORTED otherwise); vfa_varlen_fwd_tile_shape() only returns
 * such shapes.
 *
 * items        device int32 [items_capacity, 8] (output).
 * n_items      device int32 [1] (output): number of items written.
 * status       device int32 [1] (output): VFA_OK or a device-detected code.
 * scratch      device scratch of vfa_varlen_fwd_workspace_bytes() bytes,
 *              8-byte aligned.
 */
vfa_status vfa_varlen_schedule(const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                               int total_q, int total_k, int max_seqlen_q, int batch,
                               int num_heads, int block_q, int block_k, int causal,
                               int window_left, int pair_tiles, int32_t *items,
                               int items_capacity,
                               int32_t *n_items, int32_t *status, void *scratch,
                               size_t scratch_bytes, vfa_stream_t stream);

/*
 * Gradients of vfa_varlen_fwd: dq, dk, dv for an upstream gradient dout.
 *
 * The pages name a varlen backward without defining it; this computes the
 * exact derivative of the forward's definition (same masks, head grouping
 * and window): with P = exp(scale * q.k - lse) over a row's visible keys,
 * dP = dout . v, Delta = sum_d dout * out and dS = P * (dP - Delta):
 *   dv[j] = sum_i P_ij dout_i,  dk[j] = scale * sum_i dS_ij q_i,
 *   dq[i] = scale * sum_j dS_ij k_j,
 * with dk, dv of a kv head summed over its query heads.  P and dS are
 * rounded to bf16 for the products (fp32 accumulation), as the forward's P.
 *
 * q, out, dout  device bf16 [total_q, num_heads, head_dim] (out and lse are
 *               the forward's results for these q, k, v).
 * k, v          device bf16 [total_k, num_kv_heads, head_dim].
 * lse           device f32 [total_q, num_heads], natural log (-FLT_MAX for
 *               rows without visible keys, which get dq = 0; an infinity is
 *               taken as well).
 * cu_seqlens_q/k, total_q/k, batch, num_heads, num_kv_heads, softmax_scale,
 * causal, window_left: as in vfa_varlen_fwd (softmax_scale must be > 0).
 * dq            device bf16 [total_q, num_heads, head_dim] (output).
 * dk, dv        device bf16 [total_k, num_kv_heads, head_dim] (output; keys
 *               no query sees get 0).
 * workspace     device scratch of vfa_varlen_bwd_workspace_bytes() bytes,
 *               256-byte aligned (status word, per-sequence key-tile and
 *               q-tile starts, Delta = rowsum(dout * out)); calls sharing it
 *               must be stream-ordered.  Its first int32 is the device status word
 *               (read with vfa_read_status): VFA_ERR_BAD_SEQLENS for invalid
 *               cu_seqlens (nothing written), VFA_ERR_TIMEOUT if a bounded
 *               wait expired.
 *
 * Supported: head_dim 64, 128 or 256 (others: VFA_ERR_UNSUPPORTED); 16-byte
 * aligned tensors.  No gradient is accumulated with atomics: dk and dv are
 * summed per key tile and dq per query tile in a fixed order, so the three
 * are bit-identical from run to run.
 */
size_t vfa_varlen_bwd_workspace_bytes(int batch, int total_q, int num_heads, int head_dim);

vfa_status vfa_varlen_bwd(const void *q, const void *k, const void *v, const void *out,
                          const void *dout, const float *lse, const int32_t *cu_seqlens_q,
                          const int32_t *cu_seqlens_k, int total_q, int total_k, int batch,
                          int num_heads, int num_kv_heads, int head_dim, float softmax_scale,
                          int causal, int window_left, void *dq, void *dk, void *dv,
                          void *workspace, size_t workspace_bytes, vfa_stream_t stream);

/*
 * Gradients of vfa_varlen_fwd_sinks: vfa_varlen_bwd under its mask.  A sink
 * gets a gradient from every query that sees it; the steps of the sinks' key
 * tiles are cut into chunks that run side by side and are added in a fixed
 * order, so results are bit-identical from run to run.
 *
 * workspace    vfa_varlen_bwd_sinks_workspace_bytes() bytes for at least
 *              these sizes and sink_tokens (at most 40 MB more than
 *              vfa_varlen_bwd's); without a window vfa_varlen_bwd's suffice.
 */
size_t vfa_varlen_bwd_sinks_workspace_bytes(int batch, int total_q, int num_heads, int head_dim,
                                            int sink_tokens);

vfa_status vfa_varlen_bwd_sinks(const void *q, const void *k, const void *v, const void *out,
                                const void *dout, const float *lse, const int32_t *cu_seqlens_q,
                                const int32_t *cu_seqlens_k, int total_q, int total_k, int batch,
                                int num_heads, int num_kv_heads, int head_dim,
                                float softmax_scale, int causal, int window_left,
                                int sink_tokens, void *dq, void *dk, void *dv, void *workspace,
                                size_t workspace_bytes, vfa_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Paged GQA decode                                                          */
/* ------------------------------------------------------------------------ */

/*
 * AttnState::new of "attention_ref.rs" (spark_storage): m = -inf, l = 0,
 * o = 0.
 *
 * m, l   device f32 [num_seqs, num_q_heads]; o device f32 [num_seqs,
 *        num_q_heads, head_dim].  device_status (nullable) device int32 [1] is
 *        set to VFA_OK.
 */
vfa_status vfa_paged_decode_init(float *m, float *l, float *o, int num_seqs, int num_q_heads,
                                 int head_dim, int32_t *device_status, vfa_stream_t stream);

/*
 * One tile update, step_tile_ref of "attention_ref.rs": for every sequence s
 * and q head qh (kv head kh = qh / (num_q_heads / num_kv_heads)) the state
 * (m, l, o) absorbs every one of the block_size tokens of every block id
 * tile_blocks[s, 0:tile_block_counts[s]]; logits are (q . k) / sqrt(head_dim).
 * After any sequence of steps the state satisfies m = max logit, l = sum
 * exp(logit - m), o = sum exp(logit - m) v over all tokens absorbed so far
 * (m is in natural-log units).  Each KV block is read once per kv head group.
 *
 * Two arguments extend the page's step (which always takes whole blocks and
 * 1/sqrt(head_dim)) for contexts that end inside their last block and for
 * other scales: with tile_token_counts the step absorbs only the first
 * tile_token_counts[s] tokens of sequence s's listed blocks, in list order
 * (blocks holding none of them are not read); softmax_scale > 0 replaces
 * 1/sqrt(head_dim).
 *
 * q                 device bf16 [num_seqs, num_q_heads, head_dim].
 * k_pool, v_pool    device bf16 [num_blocks, block_size, num_kv_heads, head_dim].
 * tile_blocks       device int32 [num_seqs, tile_capacity]: physical block ids.
 * tile_block_counts device int32 [num_seqs]: entries used per row (0 = no-op).
 * tile_token_counts nullable device int32 [num_seqs]: tokens to absorb, in
 *                   [0, tile_block_counts[s] * block_size] (0 = no-op); NULL
 *                   = every token of every listed block.
 * softmax_scale     logit scale; <= 0 means 1/sqrt(head_dim); NaN or inf is
 *                   VFA_ERR_INVALID_ARG.
 * m, l, o           the state (in/out), as in vfa_paged_decode_init.
 * device_status     nullable device int32 [1]: a count outside
 *                   [0, tile_capacity], a token count outside its range or a
 *                   block id outside [0, num_blocks) stores VFA_ERR_BAD_BLOCK
 *                   here (first error wins) and that sequence's state is left
 *                   unchanged for this step.
 *
 * Supported: head_dim in {64, 128, 256}; block_size == 16;
 * num_q_heads / num_kv_heads in {1, 2, 4, 8}; num_blocks <= 2^26.
 */
vfa_status vfa_paged_decode_step(const void *q, const void *k_pool, const void *v_pool,
                                 int num_blocks, const int32_t *tile_blocks,
                                 const int32_t *tile_block_counts,
                                 const int32_t *tile_token_counts, int tile_capacity,
                                 int num_seqs, int num_q_heads, int num_kv_heads,
                                 int head_dim, int block_size, float softmax_scale, float *m,
                                 float *l, float *o, int32_t *device_status,
                                 vfa_stream_t stream);

/*
 * vfa_paged_decode_step with each (sequence, kv head) tile cut into
 * num_splits contiguous runs of its blocks, one CTA per run, so a batch of
 * few sequences with long tiles still spreads over every SM.  The result
 * is the same state update: "attention_ref.rs" (file header) requires a
 * tile's fragmentation to give the single-shot result, and the runs are
 * merged with the same rule the step applies across tiles (m = max of the
 * parts, l and o rescaled by exp(m_part - m) and summed).
 *
 * Each run's CTA writes its partial (m, l, o) to `workspace` and takes a
 * ticket (one atomic add); the last CTA of a (sequence, kv head) merges
 * every run with the incoming state, writes (m, l, o) and sets the ticket
 * back to zero.  No CTA waits for another.
 *
 * Arguments, results and device checks as in vfa_paged_decode_step, plus:
 * num_splits     runs per tile, 1 ..  1024 (1 = vfa_paged_decode_step;
 *                vfa_paged_decode_split_count suggests one); runs past a
 *                tile's last block are empty.
 * workspace      device scratch of vfa_paged_decode_split_workspace_bytes()
 *                bytes, 256-byte aligned, ignored when num_splits == 1.  It
 *                must hold zeros before its first use (e.g. cleared when
 *                allocated); every call leaves it that way.  Calls sharing
 *                one workspace must be stream-ordered.
 */
vfa_status vfa_paged_decode_step_split(const void *q, const void *k_pool, const void *v_pool,
                                       int num_blocks, const int32_t *tile_blocks,
                                       const int32_t *tile_block_counts,
                                       const int32_t *tile_token_counts, int tile_capacity,
                                       int num_seqs, int num_q_heads, int num_kv_heads,
                                       int head_dim, int block_size, float softmax_scale,
                                       float *m, float *l, float *o, int32_t *device_status,
                                       int num_splits, void *workspace, size_t workspace_bytes,
                                       vfa_stream_t stream);

/*
 * Workspace bytes of vfa_paged_decode_step_split: one ticket per (sequence,
 * kv head) and (head_dim + 2) floats per (sequence, q head, run).  0 for
 * unsupported sizes.
 */
size_t vfa_paged_decode_split_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                              int head_dim, int num_splits);

/*
 * A run count for vfa_paged_decode_step_split on the current device: about
 * four CTAs per SM over num_seqs * num_kv_heads rows, with runs of at least
 * eight blocks of a tile_capacity-block tile.
 */
vfa_status vfa_paged_decode_split_count(int num_seqs, int num_kv_heads, int tile_capacity,
                                        int *num_splits);

/*
 * finalize_ref of "attention_ref.rs": out = bf16(o * (l > 0 ? 1 / l : 0)),
 * round to nearest even.  l: device f32 [num_seqs, num_q_heads]; o: device
 * f32 [num_seqs, num_q_heads, head_dim]; out: device bf16, same shape as o.
 */
vfa_status vfa_paged_decode_finalize(const float *l, const float *o, int num_seqs,
                                     int num_q_heads, int head_dim, void *out,
                                     vfa_stream_t stream);

/*
 * Attention of one new token per sequence over a paged bf16 cache, in one
 * launch: no state, whole contexts, with a window and sinks.  With n =
 * token_counts[s] the query is the token at position n - 1, which the cache
 * holds already:
 *   out[s, h] = sum_j p_j v_j / sum_j p_j, p_j = exp(softmax_scale q.k_j),
 * over the tokens j < n with j >= n - 1 - window_left or j < sink_tokens,
 * query head h on kv head h / (num_q_heads / num_kv_heads), and lse = the
 * natural log of sum_j p_j.  token_counts[s] == 0 gives out = 0 and lse =
 * -FLT_MAX.  Only pages that hold such tokens are read, and what their other
 * slots hold does not matter.  The batch's pages are spread over the SMs,
 * whatever the lengths.
 *
 * q, out       device bf16 [num_seqs, num_q_heads, head_dim].
 * k_pool, v_pool  device bf16 [num_blocks, 16, num_kv_heads, head_dim].
 * tables       device int32 [num_seqs, capacity]: physical page of each
 *              logical one.
 * token_counts device int32 [num_seqs], in [0, capacity * 16].
 * window_left  < 0: no window (sink_tokens then changes nothing).
 * sink_tokens  >= 0.
 * softmax_scale  <= 0 means 1/sqrt(head_dim); NaN or inf is
 *              VFA_ERR_INVALID_ARG.
 * lse          nullable device f32 [num_seqs, num_q_heads].
 * key_weights  nullable device f32 [num_seqs, num_kv_heads, capacity * 16]:
 *              the accumulated weight of each slot of a row's pages.  With
 *              it, key_weights_out (may be key_weights) gets, at every visible
 *              token, key_weights + the sum of p_j / sum_j p_j over the kv
 *              head's query heads; other slots are left as they were.
 * workspace    device scratch of vfa_paged_decode_workspace_bytes() bytes,
 *              256-byte aligned, with the capacity (0: without key_weights).
 *              It must hold zeros before its first use; every call leaves what
 *              has to be zero that way.  It serves every call with the same
 *              heads and head_dim that asks for no more bytes, with and
 *              without key_weights.  Calls sharing it must be stream-ordered.
 * Device-detected: a token count out of range or a page id outside [0,
 * num_blocks) among those it reads stores VFA_ERR_BAD_BLOCK in device_status
 * (nullable device int32 [1], the first error is kept) and leaves that
 * sequence's out, lse and key_weights_out as they were.
 * Supported: head_dim 64, 128 or 256; pages of 16 tokens; any num_q_heads that
 * is a multiple of num_kv_heads; num_seqs * (capacity + 64) <= 2^30 and
 * capacity, num_blocks <= 2^26.
 */
size_t vfa_paged_decode_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                        int capacity);

vfa_status vfa_paged_decode(const void *q, const void *k_pool, const void *v_pool, int num_blocks,
                            const int32_t *tables, int capacity, const int32_t *token_counts,
                            int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                            int window_left, int sink_tokens, float softmax_scale, void *out,
                            float *lse, const float *key_weights, float *key_weights_out,
                            int32_t *device_status, void *workspace, size_t workspace_bytes,
                            vfa_stream_t stream);

/*
 * Test hook for the block-table gather of vfa_paged_decode_step: runs the
 * same device address computation and writes, for every sequence s, listed
 * block b < count_s, token t and kv head kh, the K and V rows it reads into
 * k_out / v_out (device bf16 [num_seqs, tile_capacity, block_size,
 * num_kv_heads, head_dim]); unlisted slots are left untouched.  Errors as in
 * vfa_paged_decode_step.
 */
vfa_status vfa_debug_paged_gather(const void *k_pool, const void *v_pool, int num_blocks,
                                  const int32_t *tile_blocks, const int32_t *tile_block_counts,
                                  int tile_capacity, int num_seqs, int num_kv_heads,
                                  int head_dim, int block_size, void *k_out, void *v_out,
                                  int32_t *device_status, vfa_stream_t stream);

/*
 * Test hook for the bounded waits of every kernel in this library (no
 * counterpart on the pages): one CTA waits on a barrier that nothing
 * arrives on, gives up after the same limit as the pipeline waits (1 s),
 * stores VFA_ERR_TIMEOUT in device_status (first error wins) and exits; the
 * context stays usable.  device_status: device int32 [1], not NULL.
 */
vfa_status vfa_debug_bounded_wait(int32_t *device_status, vfa_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Query / key norm and position rotation                                    */
/* ------------------------------------------------------------------------ */

/*
 * RMS norm of every query and key head and the rotation of its position, in
 * one pass: what stands between a projection and vfa_varlen_fwd or a cache.
 * Per (token, head) vector x of head_dim elements with weight w:
 *   n = x * (mean(x^2) + eps)^-1/2 * w          (weight NULL: n = x)
 *   y_a = n_a cos(phi_i) - n_b sin(phi_i)
 *   y_b = n_b cos(phi_i) + n_a sin(phi_i)       for pair i < rotary_dim / 2
 *   y_d = n_d                                   for d >= rotary_dim
 * with (a, b) = (i, i + rotary_dim / 2), or (2i, 2i + 1) if interleaved, and
 * phi_i = 2 pi * turns_i * positions[axis_i, token].  fp32 arithmetic,
 * rounded once to bf16.
 *
 * q, k         device bf16 [tokens, heads, head_dim]; heads and dims are
 *              contiguous, tokens q_stride / k_stride elements apart (views of
 *              a joint projection's output are taken as they are).
 * q_out, k_out the results, same shape, strides q_out_stride / k_out_stride;
 *              may be q and k themselves (same pointer and stride), must not
 *              overlap them otherwise.
 * positions    device int32 [num_axes, tokens]: each token's position on each
 *              axis (one for text; time, height and width for video).  Any
 *              int32 value.
 * table        device uint64 [rotary_dim / 2][2]: turns per position in units
 *              of 2^-64 turn (round(inv_freq / (2 pi) * 2^64)), and the axis.
 *              The angle is position * turns modulo 2^64, exact for every
 *              position.  An axis >= num_axes reads the last one.
 * q_weight, k_weight  device f32 [head_dim], each nullable (no norm).
 * eps          finite, >= 0.
 *
 * Supported: head_dim 64, 128 or 256; at most 65535 heads; rotary_dim a multiple of 16 in
 * [0, head_dim] (0: positions and table are not read); pointers of bf16
 * tensors 16-byte aligned and strides multiples of 8, at least heads *
 * head_dim.  With tokens == 0 nothing is enqueued and tensors may be NULL.
 */
vfa_status vfa_qk_norm_rope_fwd(const void *q, const void *k, int64_t q_stride, int64_t k_stride,
                                const int32_t *positions, int num_axes, const uint64_t *table,
                                int rotary_dim, int interleaved, const float *q_weight,
                                const float *k_weight, float eps, int tokens, int num_q_heads,
                                int num_kv_heads, int head_dim, void *q_out, void *k_out,
                                int64_t q_out_stride, int64_t k_out_stride, vfa_stream_t stream);

/*
 * Gradients of vfa_qk_norm_rope_fwd: with g the rotation of the upstream
 * gradient by the opposite angles, r the inverse root mean square and
 * u = g * w,
 *   dweight = sum over tokens and heads of g * x * r
 *   dx = r * (u - x * r^2 * mean(u * x))        (weight NULL: dx = g)
 * q and k are the forward's inputs (not read where their weight is NULL, but
 * not NULL).  dq_out and dk_out are the upstream gradients, dq and dk the
 * results; all have strides as in the forward.  dq and dk may be dq_out and
 * dk_out themselves.  dq_weight, dk_weight: device f32 [head_dim], required
 * where the weight is given, ignored where it is NULL; set (not added to).
 * The sums run in a fixed order: results are bit-identical from run to run
 * on one device.
 *
 * workspace    device scratch of vfa_qk_norm_rope_bwd_workspace_bytes()
 *              bytes, 16-byte aligned; may be NULL where both weights are.
 *              Calls sharing it must be stream-ordered.
 */
size_t vfa_qk_norm_rope_bwd_workspace_bytes(int head_dim);

vfa_status vfa_qk_norm_rope_bwd(const void *q, const void *k, int64_t q_stride, int64_t k_stride,
                                const void *dq_out, const void *dk_out, int64_t dq_out_stride,
                                int64_t dk_out_stride, const int32_t *positions, int num_axes,
                                const uint64_t *table, int rotary_dim, int interleaved,
                                const float *q_weight, const float *k_weight, float eps,
                                int tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                void *dq, void *dk, int64_t dq_stride, int64_t dk_stride,
                                float *dq_weight, float *dk_weight, void *workspace,
                                size_t workspace_bytes, vfa_stream_t stream);

/* ------------------------------------------------------------------------ */
/* A paged cache held in 4 bits                                              */
/* ------------------------------------------------------------------------ */

/*
 * Format.  A pool is uint8 [num_blocks, num_kv_heads, 18 * head_dim]: pages of
 * 16 tokens, K and V of one kv head side by side.  A value is
 *   descale * scale * code
 * with code in E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) and one E4M3 scale
 * per 16 consecutive dims of a token.  descale_k and descale_v hold for the
 * whole pool and are powers of two in [2^-64, 2^64] (VFA_ERR_INVALID_ARG
 * otherwise): every value then has at most six significant bits and is exact
 * in bf16.  Bytes of a page's head, t = token in the page, d = dim, D =
 * head_dim, W = min(16, D / 8), c = d / W (integer divisions):
 *   K codes   t D/2 + d/2, low nibble for even d
 *   V codes   8 D + ((t/8) (D/(8 W)) + c/8) 32 W + ((c%8) 4 + (t/2)%4) W +
 *             (t%2) W/2 + (d%W)/2, low nibble for even d
 *   K scales  16 D + t D/16 + d/16
 *   V scales  17 D + ((d/16) 4 + (t/2)%4) 4 + t%2 + 2 (t/8)
 * No byte holds parts of two tokens.
 *
 * tables       device int32 [num_seqs, capacity]: physical page of each
 *              logical page (as tile_blocks of vfa_paged_decode_step; one
 *              table serves both kinds of pool).
 * device_status  nullable device int32 [1]; the first error is kept, so clear
 *              it before use.
 * Supported: head_dim 64, 128 or 256; at most 65535 kv heads; num_blocks <=
 * 2^26; pool, k, v 16-byte aligned.
 */
size_t vfa_kv4_block_bytes(int num_kv_heads, int head_dim);

/*
 * Writes packed tokens into the cache: token i of sequence s (packed row
 * cu_seqlens[s] + i) becomes position start_positions[s] + i of its table row.
 * Per group of 16 dims scale = E4M3(max |x / descale| / 6) and code =
 * E2M1(x / descale / scale), both to nearest even and saturating; a group
 * whose scale rounds to zero stores zeros.  Inputs are finite.
 *
 * k, v         device bf16 [total, num_kv_heads, head_dim], tokens k_stride /
 *              v_stride elements apart (multiples of 8).
 * cu_seqlens   device int32 [num_seqs + 1], from 0, not decreasing, ending at
 *              or below total: rows past the end are padding, whatever they hold.
 * Nothing but the written tokens' bytes changes.  Two tokens of one call
 * must not go to one slot (two rows writing a page they share): what that
 * slot then holds is unspecified.
 * Device-detected: cu_seqlens that are no prefix sum (VFA_ERR_BAD_SEQLENS),
 * positions or page ids out of range (VFA_ERR_BAD_BLOCK); the tokens they
 * leave without a place are skipped.
 */
vfa_status vfa_kv4_write(const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                         int total, void *pool, int num_blocks, const int32_t *tables,
                         int capacity, const int32_t *cu_seqlens, const int32_t *start_positions,
                         int num_seqs, int num_kv_heads, int head_dim, float descale_k,
                         float descale_v, int32_t *device_status, vfa_stream_t stream);

/*
 * Reads tokens back as bf16 (exact): the reverse of vfa_kv4_write with the
 * same arguments, k and v written.  With start_positions 0 and cu_seqlens the
 * context lengths, k and v are the packed keys and values vfa_varlen_fwd takes
 * for a prompt that continues them (causal = 2).  Rows without a place in the
 * cache (padding, errors) are left as they were.
 */
vfa_status vfa_kv4_gather(void *k, void *v, int64_t k_stride, int64_t v_stride, int total,
                          const void *pool, int num_blocks, const int32_t *tables, int capacity,
                          const int32_t *cu_seqlens, const int32_t *start_positions, int num_seqs,
                          int num_kv_heads, int head_dim, float descale_k, float descale_v,
                          int32_t *device_status, vfa_stream_t stream);

/*
 * Attention of one query token per sequence over the cache:
 *   out[s, h] = sum_j p_j v_j / sum_j p_j, p_j = exp(softmax_scale q.k_j),
 * over the first token_counts[s] tokens of the sequence's pages, query head h
 * on kv head h / (num_q_heads / num_kv_heads), and lse = the natural log of
 * sum_j p_j.  token_counts[s] == 0 gives out = 0 and lse = -FLT_MAX.  What a
 * page holds past the last token does not matter.  One launch; the work of
 * the batch is spread over the SMs by page, whatever the lengths.
 *
 * q, out       device bf16 [num_seqs, num_q_heads, head_dim].
 * token_counts device int32 [num_seqs], in [0, capacity * 16].
 * softmax_scale  <= 0 means 1/sqrt(head_dim); NaN or inf is
 *              VFA_ERR_INVALID_ARG.
 * lse          nullable device f32 [num_seqs, num_q_heads].
 * workspace    device scratch of vfa_kv4_decode_workspace_bytes() bytes,
 *              256-byte aligned: partial states, then tickets.  It must hold
 *              zeros before its first use; every call leaves the tickets zero.
 *              A workspace made for num_seqs sequences serves any smaller
 *              number with the same heads and head_dim.  Calls sharing it
 *              must be stream-ordered.
 * Device-detected: a token count out of range or a listed page id outside
 * [0, num_blocks) stores VFA_ERR_BAD_BLOCK and leaves that sequence's out and
 * lse rows (of the kv heads that saw it) as they were.
 * Supported: any num_q_heads that is a multiple of num_kv_heads;
 * num_seqs * (capacity + 64) <= 2^30.
 */
size_t vfa_kv4_decode_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                      int head_dim);

vfa_status vfa_kv4_decode(const void *q, const void *pool, int num_blocks, const int32_t *tables,
                          int capacity, const int32_t *token_counts, int num_seqs,
                          int num_q_heads, int num_kv_heads, int head_dim, float descale_k,
                          float descale_v, float softmax_scale, void *out, float *lse,
                          int32_t *device_status, void *workspace, size_t workspace_bytes,
                          vfa_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Pages of a cache                                                          */
/* ------------------------------------------------------------------------ */

/*
 * Which pages of a pool the sequences hold, kept on the device:
 *   refcounts     int32 [num_blocks]: rows that list the page, 0 = free;
 *   tables        int32 [num_seqs, capacity]: physical page of each logical one;
 *   token_counts  int32 [num_seqs]: tokens; the first ceil(tokens /
 *                 block_size) entries of a row are live.
 * One such state serves any number of pools (K and V of every layer, bf16 or
 * 4-bit): pools is a host array of num_pools device addresses (16-byte
 * aligned, num_blocks pages each) and page_bytes a host array of their page
 * sizes (multiples of 16, at most 2^31 - 4096); at most 256 pools, and 0 is
 * allowed.  Nothing is read back to the host, so the calls can be captured in
 * a graph.  num_blocks and the entries of one call are at most 2^26; an empty
 * list (no forks, no rows, no copies) enqueues nothing and may be NULL.
 *
 * New pages are the free pages with the lowest ids, handed out in the order
 * stated, so the results depend on the inputs alone.
 *
 * workspace     device scratch of vfa_pages_workspace_bytes() bytes (for at
 *               least this num_blocks, num_seqs and num_forks; no initial
 *               value needed), 16-byte aligned.  Calls sharing it must be
 *               stream-ordered.
 * device_status nullable device int32 [1]; the first error is kept.
 */
size_t vfa_pages_workspace_bytes(int num_blocks, int num_seqs, int num_forks);

/*
 * token_counts[s] += add_tokens[s], with new pages (refcount 1) for the rows
 * that need them, in the order of (s, logical page).  VFA_ERR_NO_PAGES (too
 * few free pages) or VFA_ERR_BAD_BLOCK (a negative addition, a row past its
 * capacity): nothing changes.
 */
vfa_status vfa_pages_extend(int32_t *refcounts, int num_blocks, int32_t *tables, int capacity,
                            int32_t *token_counts, int num_seqs, const int32_t *add_tokens,
                            int block_size, void *workspace, size_t workspace_bytes,
                            int32_t *device_status, vfa_stream_t stream);

/*
 * Row children[i] becomes a copy of row parents[i], i < num_forks: full pages
 * are shared (their refcounts grow), a partly filled last page is copied in
 * every pool to a new page of the child's own (in the order of i), so both
 * rows can be extended and written.  A negative parent skips the entry.  Every
 * child must have token_counts 0 and be listed once; a parent may be listed
 * any number of times.  VFA_ERR_NO_PAGES, or VFA_ERR_BAD_BLOCK for rows out of
 * range, a child in use or listed twice, a bad count or last page: nothing
 * changes.  A full page that is out of range or not in use is listed in the
 * child as it is, not counted, and recorded as VFA_ERR_BAD_BLOCK.
 */
vfa_status vfa_pages_fork(int32_t *refcounts, int num_blocks, int32_t *tables, int capacity,
                          int32_t *token_counts, int num_seqs, const int32_t *parents,
                          const int32_t *children, int num_forks, void *const *pools,
                          const int *page_bytes, int num_pools, int block_size, void *workspace,
                          size_t workspace_bytes, int32_t *device_status, vfa_stream_t stream);

/*
 * Rows seqs[i], i < n, give up their pages: refcounts fall by one per live
 * entry and token_counts become 0.  A row listed twice is freed once; a
 * negative entry is skipped.  Table entries keep their old values.  A row out
 * of range, a bad page id or a refcount that is 0 already is recorded as
 * VFA_ERR_BAD_BLOCK and skipped.
 */
vfa_status vfa_pages_free(int32_t *refcounts, int num_blocks, const int32_t *tables, int capacity,
                          int32_t *token_counts, int num_seqs, const int32_t *seqs, int n,
                          int block_size, int32_t *device_status, vfa_stream_t stream);

/*
 * Moves the used pages into [0, U), U = their number: those at or above U go,
 * in ascending order, to the free pages below U, in ascending order, in every
 * pool.  num_used (device int32 [1]) receives U.  The moved tables and
 * refcounts go to tables_out (live entries only; the others are left as they
 * were) and refcounts_out, which may be tables and refcounts themselves.  A
 * live entry that is out of range or not in use is kept and recorded as
 * VFA_ERR_BAD_BLOCK; a row with a bad count is skipped.
 */
vfa_status vfa_pages_compact(const int32_t *refcounts, int num_blocks, const int32_t *tables,
                             int capacity, const int32_t *token_counts, int num_seqs,
                             void *const *pools, const int *page_bytes, int num_pools,
                             int block_size, int32_t *refcounts_out, int32_t *tables_out,
                             int32_t *num_used, void *workspace, size_t workspace_bytes,
                             int32_t *device_status, vfa_stream_t stream);

/*
 * Page src[i] of every pool is copied over page dst[i], i < n (device int32
 * [n] each).  A negative src skips the entry; other ids out of range are
 * recorded as VFA_ERR_BAD_BLOCK and skipped.  A page may be the source of any
 * number of copies, but the target of one only and not a source as well.
 */
vfa_status vfa_pages_copy(void *const *pools, const int *page_bytes, int num_pools,
                          const int32_t *src, const int32_t *dst, int n, int num_blocks,
                          int32_t *device_status, vfa_stream_t stream);

/*
 * Rows give up their last tokens: token_counts_out[s] = new_counts[s] where 0
 * <= new_counts[s] < token_counts[s], and the pages behind the last token left
 * lose a reference.  A negative or equal new count leaves a row as it is.  A
 * new count above the old one, a bad old count, or a last page that would be
 * cut in two and that another row lists as well (its refcount before the call
 * is above 1) leaves the row as it is and is recorded as VFA_ERR_BAD_BLOCK; bad
 * page ids and refcounts that are 0 already are recorded and skipped.  Table
 * entries keep their old values.
 *
 * refcounts_out, token_counts_out  may be refcounts and token_counts.
 * workspace     device scratch of 8 * num_seqs bytes, 16-byte aligned.
 */
vfa_status vfa_pages_truncate(const int32_t *refcounts, int num_blocks, const int32_t *tables,
                              int capacity, const int32_t *token_counts, int num_seqs,
                              const int32_t *new_counts, int block_size, int32_t *refcounts_out,
                              int32_t *token_counts_out, void *workspace, size_t workspace_bytes,
                              int32_t *device_status, vfa_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Eviction by attention weight                                              */
/* ------------------------------------------------------------------------ */

/*
 * The accumulated attention weight of packed keys, for a prompt:
 *   key_weights_out[b, hk, j] = key_weights[b, hk, j] + the sum over the query
 *   heads of kv head hk and the queries i of sequence b that see key j of
 *   exp(softmax_scale q_i.k_j - lse_i)
 * with lse from vfa_varlen_fwd (or _sinks) under the same mask.  Key j of
 * sequence b is slot j of its row, as in vfa_paged_decode, which adds later
 * queries to the same sums.
 *
 * q, k, lse, cu_seqlens_q/k, totals, max_seqlen_q, heads, head_dim,
 * softmax_scale, causal, window_left, sink_tokens: as in vfa_varlen_fwd_sinks.
 * key_weights, key_weights_out  device f32 [batch, num_kv_heads, row_stride],
 *              may be the same; entries past a sequence's keys are left as they
 *              were.  row_stride is at least the longest key length.
 * workspace    device scratch of vfa_varlen_key_weights_workspace_bytes()
 *              bytes (at most 20 MB or 1 KB per key, and 8 bytes per key and
 *              head), 256-byte aligned; one made for some sizes serves smaller
 *              ones with as many heads.  Its first int32 is the device status
 *              word: VFA_ERR_BAD_SEQLENS (bad cu_seqlens, a q length above
 *              max_seqlen_q, more keys than row_stride; nothing is written) or
 *              VFA_ERR_TIMEOUT.  Calls sharing it must be stream-ordered.
 * The sums run in a fixed order: results are bit-identical from run to run.
 */
size_t vfa_varlen_key_weights_workspace_bytes(int batch, int total_q, int total_k, int max_seqlen_q,
                                              int num_heads);

vfa_status vfa_varlen_key_weights(const void *q, const void *k, const float *lse,
                                  const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                  int total_q, int total_k, int max_seqlen_q, int batch,
                                  int num_heads, int num_kv_heads, int head_dim,
                                  float softmax_scale, int causal, int window_left,
                                  int sink_tokens, const float *key_weights,
                                  float *key_weights_out, int64_t row_stride, void *workspace,
                                  size_t workspace_bytes, vfa_stream_t stream);

/*
 * Tokens of little weight leave a paged bf16 cache (one layer's pools).  Of
 * the n = token_counts[s] tokens of a row b = min(n, budgets[s]) stay (a
 * negative budget: all), for every kv head its own:
 *   - those with positions below s0 = min(sink_tokens, b),
 *   - those with the last min(recent_tokens, b - s0) positions,
 *   - of the others those with the largest key_weights, ties by the lowest slot
 *     (weights in the order of floats, any NaN the largest).
 * Kept tokens at slots >= b move, in ascending order, to the free slots below
 * b, in ascending order; the other slots of the pools stay as they are.
 * key_weights_out and positions_out get the values of the slots below b, and
 * key_weights_out zeros for the slots in [b, n), which tokens to come will take.
 * kept[s] = b; token_counts and the pages stay as they are, so that every layer
 * is called with the same ones, each with its own weights, positions and
 * history; vfa_pages_truncate with kept comes last.  Attention over the kept
 * tokens needs no order; a window over slots has no meaning after an eviction.
 *
 * key_weights  device f32 [num_seqs, num_kv_heads, capacity * 16].
 * positions    device int32, the same shape: which token of its sequence a slot
 *              holds, for slots below history[s][0]; slots past it were
 *              appended since and hold the tokens slot + history[s][1].
 * history      device int32 [num_seqs, 2], zeros for a new sequence (as its
 *              key_weights): becomes (b, history[s][1] + n - b).
 * key_weights_out, positions_out, history_out  may be the inputs.
 * refcounts    device int32 [num_blocks], as in the page operations: a row that
 *              loses tokens must be alone on the pages that hold its first b
 *              slots (refcount 1), since they are written.
 * kept         device int32 [num_seqs].
 * workspace    device scratch of vfa_cache_evict_workspace_bytes() bytes,
 *              256-byte aligned, no initial value.  Calls sharing it must be
 *              stream-ordered.
 * Device-detected: a bad count, history or page id, or a page shared as above,
 * stores VFA_ERR_BAD_BLOCK in device_status (nullable; the first error is kept):
 * the row's slots, key_weights_out and positions_out stay as they were, kept[s]
 * is n and history_out[s] is history[s].  Stored positions that are not one per
 * token may name more than b tokens that stay: the lowest slots of them do.
 * Supported: head_dim 64, 128 or 256; pages of 16 tokens; capacity and num_blocks <=
 * 2^26.
 */
size_t vfa_cache_evict_workspace_bytes(int num_seqs, int num_kv_heads, int capacity);

vfa_status vfa_cache_evict(void *k_pool, void *v_pool, const int32_t *refcounts, int num_blocks,
                           const int32_t *tables, int capacity, const int32_t *token_counts,
                           const int32_t *budgets, int num_seqs, int num_kv_heads, int head_dim,
                           const float *key_weights, const int32_t *positions,
                           const int32_t *history, int sink_tokens, int recent_tokens,
                           float *key_weights_out, int32_t *positions_out, int32_t *history_out,
                           int32_t *kept, void *workspace, size_t workspace_bytes,
                           int32_t *device_status, vfa_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Status                                                                    */
/* ------------------------------------------------------------------------ */

/*
 * Waits for `stream`, then copies the device int32 at `device_status_word`
 * (the first word of a vfa_varlen_fwd workspace, or a decode device_status)
 * to *host_status.
 */
vfa_status vfa_read_status(const void *device_status_word, vfa_stream_t stream,
                           int32_t *host_status);

#ifdef __cplusplus
}
#endif

#endif /* VFA_H */
