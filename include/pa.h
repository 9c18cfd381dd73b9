/*
 * pa.h -- C ABI of libpa: paged varlen attention for GB300 (sm_103a).
 *
 * One iteration-level (continuous) batch mixes decode rows (qo_len = 1) and
 * chunked-prefill rows (qo_len > 1, causal, starting at an offset).  Every
 * row reads its keys and values through a block table of fixed 16-token
 * pages; pages holding a shared prefix are referenced by many block tables
 * and stored once.
 *
 * Sources for the semantics (page titles and sections):
 *   - "Inference optimisation" (AI-infra book ch. 8), §8.1.1: prefill stores
 *     the keys and values of each layer; decode reads the whole context.
 *   - same, §8.3.1 and Fig. 8-10: fixed-size blocks, per-request block table
 *     from logical to physical block, logical order recovered through it.
 *   - same, §8.3.2 and Fig. 8-13: shared prefix blocks referenced by several
 *     block tables, stored once.
 *   - same, §8.2.3 and Fig. 8-8/8-9: a chunk of c new tokens after h old ones;
 *     new token j (0-based) attends to h + j + 1 keys.
 *   - "vLLM, SGLang and continuous batching", section "PagedAttention":
 *     16-token blocks, block table, attention kernel reads K/V through it.
 *   - "Disaggregated prefill and decode": qo_len / kv_len per request
 *     (decode sends qo_len = 1), and the HND page layout (head before token
 *     inside a page, so one head's page is contiguous).
 *
 * Conventions shared by every call:
 *   - All tensors are device memory owned by the caller.  No call allocates
 *     device memory: scratch space is the caller's `workspace`, except for
 *     pa_attention_varlen_noalloc, whose scratch is one fixed array that the
 *     library holds in each device's memory while it is loaded.
 *   - All launches are asynchronous on `stream` (a cudaStream_t; NULL is the
 *     legacy default stream).  A call that returns PA_OK has only enqueued
 *     work.
 *   - Arguments are validated on the host first; on any error nothing is
 *     launched and the status says why (pa_last_error_message() has detail).
 *   - bf16 means IEEE bfloat16 (torch.bfloat16).  Row-major, densely packed.
 *   - KV pool layout (HND): k_cache and v_cache are each
 *     [num_blocks, num_kv_heads, block_size, head_dim] bf16, so one
 *     (block, kv head) slab is block_size * head_dim * 2 bytes, contiguous.
 *     Base pointers must be 16-byte aligned.
 *   - Supported shapes: head_dim = 128, block_size = 16,
 *     num_q_heads = 4 * num_kv_heads (GQA groups of 4 consecutive query
 *     heads per kv head: q head h reads kv head h / 4), num_kv_heads <= 256.
 *     Others give PA_ERR_UNSUPPORTED.
 *   - Decode rows are planned in launches of up to 1024 rows; the rows of
 *     one launch may hold at most 1,048,576 / num_kv_heads key pages of 16
 *     tokens in all (131,072 pages, 2,097,152 tokens, with 8 kv heads: 1024
 *     CTA segments of at most 1024 pages, shared by the kv heads).  Beyond
 *     that the attention calls give PA_ERR_UNSUPPORTED; pa_plan_decode_grid
 *     answers the same on the host alone.
 *   - Kernels never trap.  A block id or slot outside the pool found on the
 *     device is skipped (its keys are masked out / its write is dropped) and
 *     recorded in the error word at the start of the workspace; read it with
 *     pa_get_device_error() after synchronising the stream.
 *   - Every wait inside a kernel is bounded in time; a wait that gives up
 *     records PA_ERR_DEVICE_TIMEOUT in the error word and the kernel returns.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* pa_stream_t; /* the same handle as cudaStream_t */

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,         /* null pointer, bad size, inconsistent metadata */
  PA_ERR_UNSUPPORTED = 2,         /* shape outside what the kernels implement */
  PA_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes below the *_workspace_size() query */
  PA_ERR_CUDA = 4,                /* a CUDA runtime call or launch failed */
  PA_ERR_DEVICE_INDEX = 5,        /* (error word) block id or slot outside the pool */
  PA_ERR_DEVICE_TIMEOUT = 6,      /* (error word) a bounded in-kernel wait gave up */
  PA_ERR_DEVICE_NO_BLOCKS = 7     /* (error word) pa_step_tables: the ring of free blocks ran out */
} pa_status;

#define PA_ABI_VERSION 1
#define PA_HEAD_DIM 128
#define PA_BLOCK_SIZE 16
#define PA_GQA_GROUP 4
#define PA_ERROR_WORD_BYTES 256   /* the workspace's first bytes hold the device error word */
#define PA_MAX_SEQ_LEN (1 << 20)  /* longest supported sequence (tokens) */

int32_t pa_abi_version(void);
const char* pa_status_string(int32_t status);
/* Detail of the last host-side error on the calling thread ("" if none). */
const char* pa_last_error_message(void);

/*
 * pa_kv_append -- write this step's new keys and values into their slots
 * ("Inference optimisation", AI-infra book ch. 8, §8.1.1: the keys and values
 * of every layer are kept for later tokens; §8.3.1 and Fig. 8-10: a token's
 * slot is a (physical block, offset) pair, and a sequence that grows takes a
 * new block from the free pool; "vLLM, SGLang and continuous batching",
 * section "PagedAttention": 16-token blocks).
 *   For new token i with slot = slot_mapping[i] >= 0, block = slot / 16 and
 *   offset = slot % 16, and every kv head h:
 *     k_cache[block, h, offset, :] = k_new[i, h, :]   (v likewise)
 *   Bytes are copied exactly.  slot < 0 means "no write" (padding).  Slots
 *   must be distinct; with duplicates the surviving row is unspecified.
 * k_new, v_new   [n_tokens, num_kv_heads, head_dim] bf16, 16-byte aligned.
 * slot_mapping   [n_tokens] int64, device.
 * k_cache, v_cache  the HND pools, modified in place.
 * workspace      device, >= PA_ERROR_WORD_BYTES bytes; only the error word is
 *                used.  A slot >= num_blocks * 16 is skipped and recorded as
 *                PA_ERR_DEVICE_INDEX.
 * n_tokens = 0 is valid and launches nothing.
 */
pa_status pa_kv_append(const void* k_new, const void* v_new, const int64_t* slot_mapping, int64_t n_tokens,
                       void* k_cache, void* v_cache, int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                       int32_t head_dim, void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * q8_0 KV pages ("Inference optimisation", AI-infra book ch. 8, §8.4.2 and
 * Fig. 8-23: every 32 values share one 2-byte scale next to their 8-bit
 * codes, 34 bytes instead of 64).  A q8_0 pool is
 * [num_blocks, num_kv_heads, PA_Q8_SLAB_BYTES] bytes: one (block, kv head)
 * slab holds block_size x head_dim int8 codes (token t, dim d at
 * t * head_dim + d), then block_size x head_dim / 32 little-endian binary16
 * scales (token t, group g = d / 32 at byte block_size * head_dim +
 * 2 * (t * head_dim / 32 + g)).  Per group: d = max|x| / 127 in binary32,
 * stored as binary16 rounded to nearest even; code = rint(x / d16) in
 * binary32 with d16 the stored scale, clamped to [-127, 127]; all codes 0
 * when d16 is 0.  A code stands for code * d16.  Inputs must be finite.
 */
#define PA_Q8_SLAB_BYTES (PA_BLOCK_SIZE * PA_HEAD_DIM + PA_BLOCK_SIZE * (PA_HEAD_DIM / 32) * 2) /* 2176 */

/*
 * pa_kv_append_q8 -- pa_kv_append into q8_0 pools: each (token, kv head)
 * row of k_new / v_new is quantized in groups of 32 as described above and
 * stored with its scales in the slot's page.  Same arguments, validation and
 * error word as pa_kv_append; k_cache and v_cache are q8_0 pools
 * (16-byte aligned).
 */
pa_status pa_kv_append_q8(const void* k_new, const void* v_new, const int64_t* slot_mapping, int64_t n_tokens,
                          void* k_cache, void* v_cache, int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                          int32_t head_dim, void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_attention_varlen_q8 -- pa_attention_varlen over q8_0 pools, for decode
 * rows: every K and V element is its code times its group's scale, the rest
 * of the definition is unchanged (fp32 arithmetic, bf16 out, natural-log
 * lse).  Rows with qo_len > 1 give PA_ERR_UNSUPPORTED; rows with qo_len = 0
 * are skipped.  Workspace as pa_attention_varlen
 * (pa_attention_workspace_size).  Reading 34 instead of 64 bytes per 32
 * values shortens the HBM-bound decode when the saved read time exceeds
 * the added dequantization (the pages' Delta T = Delta D / beta - T_c).
 */
pa_status pa_attention_varlen_q8(const void* q, const void* k_cache, const void* v_cache, int64_t num_blocks,
                                 const int32_t* block_tables, int32_t max_blocks_per_req, const int32_t* seq_lens,
                                 const int32_t* qo_indptr, const int32_t* seq_lens_host,
                                 const int32_t* qo_indptr_host, int32_t num_reqs, int32_t total_q,
                                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                 float sm_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                 pa_stream_t stream);

/*
 * q4 KV pages: 4-bit codes with a bf16 scale and offset for every 32 values
 * (20 bytes instead of 64).  The pages' grouping of q8_0 ("Inference
 * optimisation", AI-infra book ch. 8, §8.4.2 and Fig. 8-23) carried to four
 * bits, with an offset, since sixteen levels around zero waste half of them on
 * a channel that lies to one side.  A q4 pool is
 * [num_blocks, num_kv_heads, PA_Q4_SLAB_BYTES] bytes; one (block, kv head)
 * slab holds
 *   codes   1024 bytes: token t's dims 32 g .. 32 g + 31 (group g) are the 16
 *           bytes at 64 t + 16 (g ^ ((t >> 1) & 3)); of their little-endian
 *           32-bit word w, dim 32 g + 8 w + 2 i is bits 4 i .. 4 i + 3 and dim
 *           32 g + 8 w + 2 i + 1 bits 16 + 4 i .. 16 + 4 i + 3 (i = 0 .. 3);
 *   scales  256 bytes: at 1024 + 16 t + 4 g the bf16 D, then the bf16 Z of
 *           token t's group g.
 * A code c stands for the bf16 nearest (ties to even) to Z + D (1 + c / 16);
 * every call below computes with these bf16 values.  Quantising a group, in
 * binary32 operations rounded to nearest even: lo, hi = its least and greatest
 * value, D = bf16(16 ((hi - lo) / 15)), Z = bf16(lo - D), code = 16 ((x - Z) /
 * D) - 16 rounded to the nearest integer (ties to even) and clamped to
 * [0, 15]; all codes 0 when D is 0 (a group of equal values is kept exactly).
 * Inputs must be finite and at most 2^125 in magnitude (a greater x - Z may
 * overflow, which costs its code up to a step); a group with infinities or NaN
 * gets unspecified bytes (no other group is touched).
 */
#define PA_Q4_SLAB_BYTES (PA_BLOCK_SIZE * PA_HEAD_DIM / 2 + PA_BLOCK_SIZE * (PA_HEAD_DIM / 32) * 4) /* 1280 */

/*
 * pa_kv_append_q4 -- pa_kv_append into q4 pools: each (token, kv head) row of
 * k_new / v_new is quantized in groups of 32 as described above and stored
 * with its scales in the slot's page.  Same arguments, validation and error
 * word as pa_kv_append; k_cache and v_cache are q4 pools (16-byte aligned).
 * With duplicate slots the stored row may mix the rows written to it.
 * n_tokens * num_kv_heads must be below 2^31 (PA_ERR_UNSUPPORTED).
 */
pa_status pa_kv_append_q4(const void* k_new, const void* v_new, const int64_t* slot_mapping, int64_t n_tokens,
                          void* k_cache, void* v_cache, int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                          int32_t head_dim, void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_kv_read_q4 -- read cached rows of q4 pools back as bf16, by slot: the
 * values that pa_attention_varlen_q4 computes with, bit for bit (to move a
 * prefix to another worker, or into a bf16 pool through pa_kv_append).
 *   For row i with slot = slot_mapping[i], block = slot / 16 and offset =
 *   slot % 16, and every kv head h:
 *     k_out[i, h, :] = the values of k_cache[block, h], token offset  (v
 *     likewise).
 *   slot < 0 (padding) gives a row of zeros; so does a slot >= num_blocks *
 *   16, which is also recorded as PA_ERR_DEVICE_INDEX.  A slot may be named
 *   any number of times.
 * slot_mapping   [n_tokens] int64, device.
 * k_cache, v_cache  q4 pools, 16-byte aligned, read only.
 * k_out, v_out   [n_tokens, num_kv_heads, head_dim] bf16, 16-byte aligned;
 *                must not overlap each other or the pools.
 * workspace      device, >= PA_ERROR_WORD_BYTES bytes; only the error word is
 *                used.
 * n_tokens = 0 is valid and launches nothing.
 * Errors: PA_ERR_INVALID_ARG (n_tokens < 0, null or misaligned pointers),
 *   PA_ERR_UNSUPPORTED (shape, or n_tokens * num_kv_heads >= 2^31),
 *   PA_ERR_WORKSPACE_TOO_SMALL, PA_ERR_CUDA.
 */
pa_status pa_kv_read_q4(const int64_t* slot_mapping, int64_t n_tokens, const void* k_cache, const void* v_cache,
                        int64_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim, void* k_out,
                        void* v_out, void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_attention_varlen_q4 -- pa_attention_varlen over q4 pools, for decode,
 * chunked-prefill and verify rows alike: every K and V element is the bf16
 * value its code stands for, the rest of the definition, the arguments, the
 * workspace (pa_attention_workspace_size) and the errors are unchanged.
 * A workspace that only q4 calls use needs no zero-filling (apart from the
 * error word), and may come from calls of other sizes; the partial results
 * that a call leaves in it are no zeros for the other entry points' counters.
 * Weights are rounded to bf16 before they meet V in rows of several queries;
 * in rows of one they carry 16 bits, unless ceil(seq_len / 16) * num_kv_heads
 * exceeds a million.  Scores of rows with many queries must stay below 2^30 in
 * magnitude.  A (query, head) with a NaN among its scores has NaN in its out row
 * and its lse, and changes no other.
 */
pa_status pa_attention_varlen_q4(const void* q, const void* k_cache, const void* v_cache, int64_t num_blocks,
                                 const int32_t* block_tables, int32_t max_blocks_per_req, const int32_t* seq_lens,
                                 const int32_t* qo_indptr, const int32_t* seq_lens_host,
                                 const int32_t* qo_indptr_host, int32_t num_reqs, int32_t total_q,
                                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                 float sm_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                 pa_stream_t stream);

/*
 * pa_copy_blocks -- copy-on-write block copy ("Inference optimisation",
 * AI-infra book ch. 8, §8.3.2 and Fig. 8-15: before a branch writes into a
 * block it shares with another request, it gets its own copy of that block,
 * and the filled read-only blocks stay shared).
 *   For pair i, the whole block src_blocks[i] -- every kv head and token
 *   slot, of k_cache and of v_cache -- is copied into block dst_blocks[i].
 * src_blocks, dst_blocks  [n_pairs] int32, device.  The dst ids must be
 *                distinct and none may also be a src id of the call;
 *                otherwise which copy lands is undefined (no fault).
 * k_cache, v_cache  HND pools as for pa_kv_append, modified in place.
 * workspace      device, >= PA_ERROR_WORD_BYTES bytes; a pair naming a block
 *                outside [0, num_blocks) is skipped and PA_ERR_DEVICE_INDEX
 *                is recorded in its error word.
 * Errors: PA_ERR_INVALID_ARG (n_pairs < 0, null or misaligned pointers),
 *   PA_ERR_UNSUPPORTED (shape), PA_ERR_WORKSPACE_TOO_SMALL, PA_ERR_CUDA.
 */
pa_status pa_copy_blocks(const int32_t* src_blocks, const int32_t* dst_blocks, int64_t n_pairs, void* k_cache,
                         void* v_cache, int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                         int32_t head_dim, void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_attention_workspace_size -- bytes of device workspace that
 * pa_attention_varlen needs for a batch with at most these sizes.  The
 * workspace holds the error word and the split-KV partial results.
 */
size_t pa_attention_workspace_size(int32_t num_reqs, int32_t total_q, int32_t num_q_heads, int32_t head_dim,
                                   int32_t max_seq_len);

/*
 * pa_attention_varlen -- causal GQA softmax attention over a paged KV cache
 * for a varlen batch ("Inference optimisation", AI-infra book ch. 8: §8.1.1,
 * decode attends each new token to the whole cached context; §8.2.3, the
 * N_pair equation and Fig. 8-8/8-9, a chunk of c tokens after h cached ones,
 * token j seeing h + j + 1 keys; §8.3.1 and Fig. 8-10, keys found through the
 * block table; "Continuous batching architecture", iteration-level batches
 * mixing decode rows and prefill chunks; "Disaggregated prefill and decode",
 * per-request qo_len / kv_len).
 *   Request r has qo_len = qo_indptr[r+1] - qo_indptr[r] query tokens, rows
 *   qo_indptr[r] .. qo_indptr[r+1]-1 of q, and seq_len = seq_lens[r] keys
 *   (the KV length after this step's append, so 0 <= qo_len <= seq_len).
 *   Query j of request r sits at position p = seq_len - qo_len + j and, for
 *   every q head h with kv head g = h / 4:
 *     s_t  = sm_scale * <q[row, h, :], K_g[t, :]>      for t = 0 .. p
 *     out[row, h, :] = sum_t exp(s_t - m) V_g[t, :] / sum_t exp(s_t - m)
 *     lse[row, h]    = m + ln(sum_t exp(s_t - m)),  m = max_t s_t
 *   where K_g[t, :] = k_cache[block_tables[r, t / 16], g, t % 16, :].
 *   Decode rows (qo_len = 1) use the persistent split-KV decode kernel: the
 *   (row, kv head) key ranges are laid end to end and cut into one equal
 *   segment per CTA, and ranges cut between CTAs are merged by log-sum-exp
 *   inside the same kernel.  Rows with qo_len > 1 use the tensor-core
 *   prefill kernel; rows with qo_len = 0 are skipped.  Arithmetic is fp32 on
 *   bf16 data; out is rounded to bf16.  The launch plan is made on the host
 *   from seq_lens_host / qo_indptr_host and travels in the kernel
 *   parameters, so a CUDA graph captured around this call replays the plan
 *   of the lengths it was captured with (for graphs replayed with new
 *   lengths, decode-only batches use pa_decode_step, which plans on the
 *   device).
 * q              [total_q, num_q_heads, head_dim] bf16, 16-byte aligned.
 * block_tables   [num_reqs, max_blocks_per_req] int32, device.  Entries past
 *                ceil(seq_len / 16) are never read.
 * seq_lens       [num_reqs] int32, device.
 * qo_indptr      [num_reqs + 1] int32, device; qo_indptr[0] = 0, non-decreasing,
 *                qo_indptr[num_reqs] = total_q.
 * seq_lens_host, qo_indptr_host  host copies of the same two arrays; the
 *                launch plan (which rows decode, how many KV splits) is made
 *                from them on the host.  They must equal the device arrays.
 * out            [total_q, num_q_heads, head_dim] bf16, 16-byte aligned.
 * lse            [total_q, num_q_heads] float32 (natural log), or NULL.
 * workspace      device, >= pa_attention_workspace_size(num_reqs, total_q,
 *                num_q_heads, head_dim, max over r of seq_lens) bytes,
 *                256-byte aligned, ZERO-FILLED before its first use.  It
 *                holds the error word, per-(request, kv head) counters of
 *                finished key ranges and the partial results of key ranges
 *                cut between CTAs; every call leaves the counters at zero,
 *                so a workspace is reused without clearing by calls with the same
 *                num_reqs and num_kv_heads; where these change, the counters of one
 *                batch lie where another kept its partial results: zero it between
 *                them, or keep a workspace for each.  Calls sharing a workspace must
 *                not run concurrently.  After a PA_ERR_DEVICE_* error, zero it again.
 *                The error word is not cleared by this call (see
 *                pa_clear_device_error).
 */
pa_status pa_attention_varlen(const void* q, const void* k_cache, const void* v_cache, int64_t num_blocks,
                              const int32_t* block_tables, int32_t max_blocks_per_req, const int32_t* seq_lens,
                              const int32_t* qo_indptr, const int32_t* seq_lens_host, const int32_t* qo_indptr_host,
                              int32_t num_reqs, int32_t total_q, int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t head_dim, int32_t block_size, float sm_scale, void* out, float* lse,
                              void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * Decode step for CUDA graphs ("Inference optimisation", AI-infra book ch. 8,
 * §8.2.4: graphs captured in advance for a few row counts, inputs padded up
 * to the next captured size; "Continuous batching architecture", section
 * "CUDA graphs": one recorded launch sequence replayed for batches whose
 * padded shape matches, which removes the per-step CPU launch work).
 *
 * pa_decode_step -- the KV append and the attention of a decode-only batch
 * in one kernel launch whose launch shape depends only on the scalars
 * (num_reqs, num_kv_heads, max_seq_len) and the device's SM count, and which
 * reads no array on the host.  A launch captured in a CUDA graph is therefore valid for every
 * batch within those scalars: between replays the caller rewrites q, k_new,
 * v_new, block_tables and seq_lens in place.
 *   Row r (0 <= r < num_reqs) is one decode request with L = seq_lens[r]
 *   keys after this step (L >= 1), its new token at position L - 1 and
 *   query q[r].  The call writes k_new[r, h, :] / v_new[r, h, :] into
 *   k_cache / v_cache at the slot of position L - 1 (block
 *   block_tables[r, (L-1) / 16], offset (L-1) % 16; no slot_mapping is
 *   taken) and computes, for every q head, the attention of
 *   pa_attention_varlen with qo_len = 1 over the L keys, the new token
 *   included (out bf16, lse natural log).
 *   Rows with L = 0 are padding: nothing is written to the cache, their out
 *   rows are zero and lse is -inf.  Padding a batch to a captured size
 *   means L = 0 for the extra rows (KV lengths need no padding: the kernel
 *   reads the exact lengths).
 *   A row with L < 0, L > max_seq_len or more than max_blocks_per_req pages
 *   is treated as padding and recorded as PA_ERR_DEVICE_INDEX; a block id
 *   outside the pool is masked and recorded as in pa_attention_varlen.
 *   Requirement (copy-on-write, §8.3.2): the block receiving a row's new
 *   token is read by no other row of the call.  The appending CTA uses the
 *   new K/V directly, so the result equals pa_kv_append followed by
 *   pa_attention_varlen whenever that holds.
 * q              [num_reqs, num_q_heads, head_dim] bf16, 16-byte aligned.
 * k_new, v_new   [num_reqs, num_kv_heads, head_dim] bf16, 16-byte aligned.
 * k_cache, v_cache  HND bf16 pools, modified in place (the new tokens).
 * block_tables   [num_reqs, max_blocks_per_req] int32, device.
 * seq_lens       [num_reqs] int32, device only.
 * num_reqs       rows of the padded batch, 0 .. 1024 (see pa_decode_step_bucket).
 * max_seq_len    largest L any replay will use, 1 .. PA_MAX_SEQ_LEN.
 * out, lse       as pa_attention_varlen with total_q = num_reqs.
 * workspace      device, >= pa_decode_step_workspace_size(num_reqs,
 *                num_q_heads, head_dim, max_seq_len) bytes, 256-byte aligned,
 *                zero-filled before first use, left reusable by every call.
 *                Calls sharing a workspace must not run concurrently.
 * Errors: PA_ERR_INVALID_ARG (null or misaligned pointers, max_seq_len
 *   outside its range), PA_ERR_UNSUPPORTED (shape, num_reqs > 1024, or
 *   num_reqs x max_seq_len too large for one launch),
 *   PA_ERR_WORKSPACE_TOO_SMALL, PA_ERR_CUDA.  num_reqs = 0 launches nothing.
 */
pa_status pa_decode_step(const void* q, const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                         int64_t num_blocks, const int32_t* block_tables, int32_t max_blocks_per_req,
                         const int32_t* seq_lens, int32_t num_reqs, int32_t max_seq_len, int32_t num_q_heads,
                         int32_t num_kv_heads, int32_t head_dim, int32_t block_size, float sm_scale, void* out,
                         float* lse, void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_decode_step_workspace_size -- bytes of workspace pa_decode_step needs
 * for these scalars on the current device; 0 when no launch exists for them (num_reqs outside
 * 0 .. 1024, max_seq_len outside 1 .. PA_MAX_SEQ_LEN, num_q_heads < 4, or
 * num_reqs x max_seq_len too large).
 */
size_t pa_decode_step_workspace_size(int32_t num_reqs, int32_t num_q_heads, int32_t head_dim, int32_t max_seq_len);

/*
 * pa_decode_step_bucket -- the padded row count for a batch of num_reqs
 * decode rows: the smallest power of two >= num_reqs (1 for 0), so that a
 * handful of captured graphs cover 1 .. 1024 rows with less than 2x rows of
 * padding (padding rows cost no key reads).  -1 outside 0 .. 1024.
 */
int32_t pa_decode_step_bucket(int32_t num_reqs);

/*
 * pa_shared_prefix_workspace_size -- bytes of device workspace that
 * pa_attention_varlen_shared_prefix needs for a batch with at most these
 * sizes: the pa_attention_workspace_size() layout followed by the prefix
 * partial ([total_q, num_q_heads, head_dim + 1] fp32) and the key-chunk
 * partials it is merged from.  shared_prefix_pages = 0 gives
 * pa_attention_workspace_size().  Returns 0 for negative arguments.
 */
size_t pa_shared_prefix_workspace_size(int32_t num_reqs, int32_t total_q, int32_t num_q_heads, int32_t head_dim,
                                       int32_t max_seq_len, int32_t shared_prefix_pages);

/*
 * pa_attention_varlen_shared_prefix -- pa_attention_varlen for a batch whose
 * requests all begin with the same shared_prefix_pages pages (the shared
 * prefix blocks of "Inference optimisation" ch. 8, §8.3.2 and Fig. 8-13,
 * referenced by every block table and stored once).
 *   Same computation, arguments and results as pa_attention_varlen (up to
 *   fp32 rounding order), with the work split by key range:
 *     1. one tensor-core pass attends every query token of the batch to the
 *        prefix keys [0, 16 * shared_prefix_pages), reading each prefix page
 *        once per kv head for all rows together (no mask is needed: every
 *        query comes after the prefix); key chunks of it run on separate CTAs
 *        and are merged by log-sum-exp;
 *     2. the decode and prefill kernels attend each row to its own keys
 *        after the prefix and fold the prefix partial into their result by
 *        log-sum-exp before rounding to bf16.
 *   With fewer than two requests that have queries, or shared_prefix_pages
 *   = 0, the call runs exactly as pa_attention_varlen.
 * shared_prefix_pages  0 <= P <= max_blocks_per_req.  The caller asserts
 *                that entries 0 .. P-1 of every block-table row hold the same
 *                block ids (the pass reads them from the first request that
 *                has queries; rows that differ get that request's prefix).
 *                Every request with qo_len > 0 must have
 *                seq_len - qo_len >= 16 * P (the prefix is cached before this
 *                step's queries), else PA_ERR_INVALID_ARG.
 * workspace      >= pa_shared_prefix_workspace_size(num_reqs, total_q,
 *                num_q_heads, head_dim, max seq_len, P) bytes, 256-byte
 *                aligned, zero-filled before its first use, as for
 *                pa_attention_varlen (its counters are left at zero too).
 * Errors: as pa_attention_varlen.
 */
pa_status pa_attention_varlen_shared_prefix(
    const void* q, const void* k_cache, const void* v_cache, int64_t num_blocks, const int32_t* block_tables,
    int32_t max_blocks_per_req, const int32_t* seq_lens, const int32_t* qo_indptr, const int32_t* seq_lens_host,
    const int32_t* qo_indptr_host, int32_t num_reqs, int32_t total_q, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int32_t shared_prefix_pages, float sm_scale, void* out, float* lse,
    void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_attention_varlen_noalloc -- pa_attention_varlen for callers that cannot
 * allocate device memory.  The pages describe no counterpart of this call;
 * it exists for callers that cannot obtain a workspace: a real-time serving
 * loop that must not enter the allocator between steps, a host framework
 * whose device memory is all handed out to its own pool, or a plugin that is
 * handed only its input and output pointers.
 *   Same computation, arguments and results as pa_attention_varlen, except
 *   that there is no workspace argument: the scratch is a fixed array of
 *   PA_NOALLOC_SCRATCH_BYTES (24 MiB) inside the library, present on every
 *   GPU that loads the library until the process exits.  A batch whose
 *   pa_attention_workspace_size() exceeds it is rejected with
 *   PA_ERR_UNSUPPORTED (and a message in pa_last_error_message()).
 *   No device memory is allocated or freed by this call.
 * device_error   nullable device int32; if given, receives the call's device
 *                error word (PA_OK or PA_ERR_DEVICE_*) on `stream`.  With
 *                NULL the device error word of the call is not reported
 *                anywhere (the next call clears it).
 * num_reqs       0 .. 65535 as for pa_attention_varlen (PA_ERR_INVALID_ARG
 *                outside, checked before seq_lens_host is read).
 * Set-up: the first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress, with that device current) and caches it; make that
 *   first call before any stream capture.
 * Sharing: every call on a device uses the same array and leaves its contents
 *   there; each call clears its error word and counters on `stream` first.
 *   Calls that overlap on the GPU race on the array, so issue them in order
 *   (e.g. on one stream).
 */
#define PA_NOALLOC_SCRATCH_BYTES (24u << 20)
pa_status pa_attention_varlen_noalloc(const void* q, const void* k_cache, const void* v_cache, int64_t num_blocks,
                                      const int32_t* block_tables, int32_t max_blocks_per_req,
                                      const int32_t* seq_lens, const int32_t* qo_indptr,
                                      const int32_t* seq_lens_host, const int32_t* qo_indptr_host, int32_t num_reqs,
                                      int32_t total_q, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                      int32_t block_size, float sm_scale, void* out, float* lse,
                                      int32_t* device_error, pa_stream_t stream);

/*
 * pa_step_tables -- a step's block tables, slots, positions and offsets, made on
 * the device from the requests' lengths ("Inference optimisation", AI-infra book
 * ch. 8, §8.3.1 and Fig. 8-10: a sequence that grows takes a new block from the
 * free pool, its table maps logical to physical blocks), so that a decode loop
 * needs no host between its steps.
 *   Request r has c = cached_lens[r] tokens in the cache and brings n =
 *   new_tokens[r] (0: it waits; negative: it has ended).
 *   qo_indptr       the exclusive sums of n (0 for n < 0), and their total.
 *   seq_lens[r]     c + n; 0 for a request that has ended.
 *   Pages ceil(c / 16) .. ceil((c + n) / 16) - 1 of r are granted: their ids are
 *   taken from the head of the ring of free blocks, in the order of requests and
 *   pages, and written into block_tables[r].
 *   Token j of r is row i = qo_indptr[r] + j of the step: positions[i] = c + j,
 *   slot_mapping[i] = 16 block_tables[r, (c + j) / 16] + (c + j) % 16.  Rows from
 *   the total to n_tokens are padding: slot -1, position 0.
 *   Pages given back go to the ring's tail, in the order of requests and pages,
 *   and are not granted before the next call.  Their table entries stay as they
 *   are.  A page whose entry is outside the pool has no block, and nothing is given
 *   back for it.  Of a request that has ended: all that it holds, except its first
 *   shared_pages.  With window > 0, of a request with n > 0: pages j >= keep with
 *   16 (j + 1) <= c - window + 1, which no query of this or a later step of
 *   pa_attention_varlen_window sees, where keep = max(ceil(sink_tokens / 16),
 *   shared_pages); first_page_out[r] is then the first page behind keep that it
 *   still holds (first_page[r] where nothing was given back, 0 for a request
 *   that has ended).
 * new_tokens, cached_lens  [num_reqs] int32, device.
 *                 Lengths grow: cached_lens[r] is what seq_lens[r] was after the
 *                 call before (0 for a new request).  Where it is less (drafts that
 *                 were refused) the call knows nothing of the pages behind it: if
 *                 ceil(cached_lens[r] / 16) is less too, the caller first puts the
 *                 blocks of the pages from there to ceil(seq_lens[r] / 16) - 1 back,
 *                 each id to place (head + count) modulo num_blocks of free_ring,
 *                 and adds one to count; else they are lost to the pool.
 * first_page      [num_reqs] int32, device, or NULL for zeros: what the call
 *                 before left in first_page_out (0 for a new request).
 * block_tables    [num_reqs, max_blocks_per_req] int32, device, modified in place:
 *                 only the entries of granted pages are written.
 * free_ring       [num_blocks] int32, device, modified in place: the ids of the
 *                 pool's free blocks, in a ring (places behind them: anything).
 * free_state      [2] int32, device: the ring's head (0 .. num_blocks - 1) and the
 *                 number of ids in it.
 * window, sink_tokens, shared_pages  >= 0.  window = 0: nothing is given back
 *                 but by ended requests (and sink_tokens is ignored).  The first
 *                 shared_pages pages of every request are never given back (a
 *                 prefix that others use too).  Other pages must belong to one
 *                 request each.
 * n_tokens        rows of slot_mapping and positions.
 * seq_lens [num_reqs], qo_indptr [num_reqs + 1], positions [n_tokens] int32,
 * slot_mapping [n_tokens] int64, free_state_out [2], first_page_out [num_reqs]
 *                 int32 (or NULL when first_page is NULL and window is 0), device.
 *                 seq_lens may be cached_lens, free_state_out free_state and
 *                 first_page_out first_page: then a captured launch steps on at
 *                 every replay.  Otherwise outputs must not overlap anything, and
 *                 a call repeated on the same inputs gives the same again.
 * workspace       device, >= PA_ERROR_WORD_BYTES bytes, 256-byte aligned, zero-filled
 *                 before its first use: the error word, and a count that every call
 *                 leaves at zero.  Calls sharing it must not run concurrently.
 * Found on the device and recorded in the error word:
 *   PA_ERR_DEVICE_INDEX: a row with c outside [0, PA_MAX_SEQ_LEN], or with more
 *   than PA_MAX_SEQ_LEN tokens or max_blocks_per_req pages after the step, is
 *   taken as one that waits (with seq_len 0 if c itself is out of these bounds).
 *   If the new tokens of all rows exceed n_tokens, or free_state is out of its
 *   range, or more pages would come back than the ring has places for, all rows
 *   wait, and no page is granted or given back.  An id in the ring outside the
 *   pool is granted as -1.
 *   PA_ERR_DEVICE_NO_BLOCKS: the ring has fewer ids than pages are needed: the
 *   pages it could not grant get the table entry -1, their tokens the slot -1, in
 *   later steps too (each records it again).  What these tokens would have written
 *   is lost to their request: end it (the blocks that it has come back) and begin it
 *   anew.  No other request is touched.
 * Errors: PA_ERR_INVALID_ARG (num_reqs outside [0, 65535], n_tokens < 0,
 *   num_blocks outside [1, 2^31 - 1], a negative window, sink_tokens or
 *   shared_pages, max_blocks_per_req < 1, null or misaligned pointers),
 *   PA_ERR_WORKSPACE_TOO_SMALL, PA_ERR_CUDA.
 */
pa_status pa_step_tables(const int32_t* new_tokens, const int32_t* cached_lens, const int32_t* first_page,
                         int32_t num_reqs, int32_t* block_tables, int32_t max_blocks_per_req, int32_t* free_ring,
                         int64_t num_blocks, const int32_t* free_state, int32_t window, int32_t sink_tokens,
                         int32_t shared_pages, int32_t n_tokens, int32_t* seq_lens, int32_t* qo_indptr,
                         int64_t* slot_mapping, int32_t* positions, int32_t* free_state_out, int32_t* first_page_out,
                         void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_rope_turns -- the rotation speeds of pa_qk_norm_rope, computed on the host:
 * turns[i] = the fraction of a turn that pair i advances per position, inv_freq[i]
 * / (2 pi) modulo 1, in units of 2^-64, off by 2^-52 of the speed (a quotient in
 * binary64) or 2^-54 of a turn, whichever is more.  A position times this, modulo
 * 2^64, is the pair's angle, off by as much times the position: 2^-34 of a turn at
 * position 2^20 for a speed of one radian, where an angle in binary32 would be off
 * by up to a sixteenth of a radian.
 * inv_freq, turns  [n] host arrays.  Errors: PA_ERR_INVALID_ARG (n outside
 * [0, 64], null pointers, a speed that is not finite).
 */
pa_status pa_rope_turns(const double* inv_freq, int32_t n, uint64_t* turns);

/*
 * pa_qk_norm_rope -- queries and keys of a layer, normalised for each head and
 * rotated by their positions, in one pass (what a model does between the product
 * that makes q, k and v and pa_kv_append).
 *   For token i, head h and x = q[i, h, :] (k likewise):
 *     y = x / sqrt(mean(x^2) + eps) * weight      (y = x with a NULL weight)
 *     a, b = y[j], y[j + rotary_dim / 2]           (y[2 j], y[2 j + 1] if interleaved)
 *     a', b' = a cos t - b sin t, b cos t + a sin t,   j = 0 .. rotary_dim / 2 - 1
 *   with the angle t = positions[i] * inv_freq[j] (see pa_rope_turns); dims from
 *   rotary_dim on are not rotated.  Arithmetic is binary32 throughout and each
 *   result is rounded once to bf16.
 * q, k           bf16, device, 16-byte aligned: token i's heads are contiguous,
 *                [num_heads, head_dim] from element i * stride on; strides are in
 *                elements, multiples of 8, at least num_heads * head_dim (a column
 *                block of a fused product's rows has the stride of the whole row).
 * positions      [n_tokens] int32, device (a negative one rotates backwards).
 * q_weight, k_weight  [head_dim] float32, device, 16-byte aligned, or NULL.
 * turns          [rotary_dim / 2] uint64, device, 8-byte aligned: pa_rope_turns.
 * rotary_dim     0 .. head_dim, a multiple of 16 (0: no rotation; turns and
 *                positions may then be NULL).
 * interleaved    0 or 1.
 * q_out, k_out   [n_tokens, num_heads, head_dim] bf16, 16-byte aligned.  q_out may
 *                be q where q_stride is num_q_heads * head_dim (k_out likewise);
 *                otherwise outputs must not overlap inputs.
 * Errors: PA_ERR_INVALID_ARG (n_tokens < 0, strides, rotary_dim, interleaved, eps
 *   negative or not finite, null or misaligned pointers), PA_ERR_UNSUPPORTED
 *   (shape, or n_tokens x heads of 2^31 or more), PA_ERR_CUDA.
 * n_tokens = 0 is valid and launches nothing.
 */
pa_status pa_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const int32_t* positions,
                          int64_t n_tokens, const float* q_weight, const float* k_weight, float eps,
                          const uint64_t* turns, int32_t rotary_dim, int32_t interleaved, int32_t num_q_heads,
                          int32_t num_kv_heads, int32_t head_dim, void* q_out, void* k_out, pa_stream_t stream);

/*
 * pa_qk_norm_rope_append -- pa_qk_norm_rope whose keys, and the values v beside
 * them, go straight to their slots of the HND pools, as pa_kv_append would have
 * put them there: one pass from the layer's product to the cache.
 * v              as k, with a stride of its own; copied exactly.
 * slot_mapping   [n_tokens] int64, device; negative: nothing is written to the
 *                pools (the token's q_out row is).  Slots must be distinct.
 * k_cache, v_cache  HND pools, 16-byte aligned, modified in place.
 * workspace      device, >= PA_ERROR_WORD_BYTES bytes; only the error word is
 *                used.  A slot >= num_blocks * 16 is skipped and recorded as
 *                PA_ERR_DEVICE_INDEX.
 * Errors: as pa_qk_norm_rope and pa_kv_append.
 */
pa_status pa_qk_norm_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping,
                                 int64_t n_tokens, const float* q_weight, const float* k_weight, float eps,
                                 const uint64_t* turns, int32_t rotary_dim, int32_t interleaved, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim, int32_t block_size, void* q_out, void* k_cache,
                                 void* v_cache, int64_t num_blocks, void* workspace, size_t workspace_bytes,
                                 pa_stream_t stream);

/*
 * pa_window_workspace_size -- bytes of device workspace that
 * pa_attention_varlen_window and pa_decode_window need for a batch with at most
 * these sizes (0 for negative arguments).
 */
size_t pa_window_workspace_size(int32_t num_reqs, int32_t total_q, int32_t num_q_heads, int32_t head_dim,
                                int32_t window, int32_t sink_tokens);

/*
 * pa_attention_varlen_window -- pa_attention_varlen with a sliding window and
 * first tokens that stay visible: the query at position p sees the keys
 *     t <= p  with  t < sink_tokens  or  t > p - window
 *   (its own and the window - 1 before it, and the first sink_tokens), the rest of
 *   the definition, the arguments and the errors are pa_attention_varlen's, over
 *   bf16 pools.  A window of seq_len or more is pa_attention_varlen.
 *   Table entries of pages that hold no key which a query of the row's request
 *   sees are never read: with pa_step_tables they are given back.  Keys and
 *   values that no query of the request sees (slots behind its last token, tokens
 *   behind its window) may hold anything, infinities and NaN included.  Infinities
 *   and NaN in values that some queries of a request see reach these and no others
 *   (outputs that are not finite are computed a second time, which takes long).
 *   Weights are rounded to bf16 before they meet V in rows of more than two
 *   queries; in rows of one or two they carry 16 bits.  A (query, head) with a NaN
 *   among its scores has NaN in its out row and its lse, and changes no other.
 * window         >= 1.
 * sink_tokens    >= 0.
 * workspace      >= pa_window_workspace_size(num_reqs, total_q, num_q_heads,
 *                head_dim, window, sink_tokens) bytes, 256-byte aligned, zero-filled
 *                before its first use; as pa_attention_varlen otherwise.  Calls and
 *                graphs of any sizes may share one that is large enough for each:
 *                beside the error word nothing depends on what it held.  It may be
 *                pa_attention_varlen's for the same num_reqs and heads, whose counters
 *                stay as they are; for other batches the partial results that a call
 *                leaves are no zeros for that call's counters.
 * Errors: as pa_attention_varlen; PA_ERR_INVALID_ARG for window < 1 or
 *   sink_tokens < 0.
 */
pa_status pa_attention_varlen_window(const void* q, const void* k_cache, const void* v_cache, int64_t num_blocks,
                                     const int32_t* block_tables, int32_t max_blocks_per_req, const int32_t* seq_lens,
                                     const int32_t* qo_indptr, const int32_t* seq_lens_host,
                                     const int32_t* qo_indptr_host, int32_t num_reqs, int32_t total_q,
                                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                     float sm_scale, int32_t window, int32_t sink_tokens, void* out, float* lse,
                                     void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_decode_window -- pa_attention_varlen_window for a padded decode-only batch,
 * planned on the device ("Inference optimisation", AI-infra book ch. 8, §8.2.4:
 * graphs captured for a few padded shapes): the launch depends on the scalars
 * alone, so that one captured in a CUDA graph serves every batch within them, and
 * with pa_step_tables and pa_qk_norm_rope_append before it a decode layer runs
 * without the host.
 *   Row r is one request with query q[r], whose seq_lens[r] keys (its own token
 *   among them) are in the cache.  seq_lens[r] = 0: padding; its out row is zero
 *   and its lse -inf.  A row with seq_lens[r] outside [0, PA_MAX_SEQ_LEN] or more
 *   than max_blocks_per_req pages is taken as padding and recorded as
 *   PA_ERR_DEVICE_INDEX.
 * q, out         [num_reqs, num_q_heads, head_dim] bf16; lse [num_reqs,
 *                num_q_heads] float32 or NULL.
 * workspace      >= pa_window_workspace_size(num_reqs, num_reqs, ...).
 * Errors: as pa_attention_varlen_window; num_reqs is 0 .. 65535 (PA_ERR_INVALID_ARG
 *   otherwise).
 */
pa_status pa_decode_window(const void* q, const void* k_cache, const void* v_cache, int64_t num_blocks,
                           const int32_t* block_tables, int32_t max_blocks_per_req, const int32_t* seq_lens,
                           int32_t num_reqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                           int32_t block_size, float sm_scale, int32_t window, int32_t sink_tokens, void* out,
                           float* lse, void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_merge_lse -- combine two partial attentions of the same queries over
 * disjoint key sets A and B.  The pages do not define this operation; it is
 * part of this library's interface so that a caller can split one request's
 * keys (across calls or devices) and combine the results.  It is the
 * log-sum-exp identity of softmax over a union of key sets:
 *   M = max(lse_a, lse_b), w_a = exp(lse_a - M), w_b = exp(lse_b - M)
 *   o = (w_a o_a + w_b o_b) / (w_a + w_b),  lse = M + ln(w_a + w_b)
 *   A part with lse = -inf has weight 0 (its o is ignored); if both are
 *   -inf, o = 0 and lse = -inf.
 * o_a, o_b, o_out  [rows, num_heads, head_dim] bf16, 16-byte aligned;
 *                  o_out may alias o_a or o_b.
 * lse_a, lse_b     [rows, num_heads] float32.
 * lse_out          [rows, num_heads] float32 or NULL; must not overlap lse_a
 *                  or lse_b.
 * head_dim must be a multiple of 8.
 */
pa_status pa_merge_lse(const void* o_a, const float* lse_a, const void* o_b, const float* lse_b, void* o_out,
                       float* lse_out, int64_t rows, int32_t num_heads, int32_t head_dim, pa_stream_t stream);

/*
 * Error word.  pa_get_device_error copies the word at the start of
 * `workspace` to the host (synchronous: call it after the stream that used
 * the workspace has been synchronised) and stores PA_OK or the first
 * PA_ERR_DEVICE_* recorded.  pa_clear_device_error zeroes it on `stream`.
 */
pa_status pa_get_device_error(const void* workspace, int32_t* code_out);
pa_status pa_clear_device_error(void* workspace, pa_stream_t stream);

/*
 * Tuning and diagnostics.
 *   pa_set_decode_ctas(n): n > 0 asks for a persistent decode grid of n CTAs
 *     (capped by the plan limits and the workspace bound), 0 restores the
 *     automatic plan (one CTA per SM for the warp-granular kernel, three
 *     per SM for the CTA-granular one).  Process-wide.  pa_decode_step and
 *     pa_decode_step_workspace_size use it too (rounded up to whole kv
 *     heads, and raised where a segment would exceed 1024 pages).
 *   pa_set_prefill_ctas(n): for a call whose batch has decode rows and rows
 *     with qo_len > 1 (bf16 pages, no shared prefix, no forced decode grid,
 *     at most 1536 query tiles of 32 and 1024 decode rows: one launch each):
 *     n > 0 runs the tensor-core jobs of the qo_len > 1 rows on n persistent
 *     CTAs beside the decode launch (at most one fewer than the jobs and
 *     half the SMs), -1 never (the jobs first, one CTA each, then the decode
 *     launch), 0 restores the automatic choice (a cost model).  For a call
 *     whose batch has only rows with qo_len > 1 (bf16 pages, no shared
 *     prefix, no forced decode grid, at most 1536 query tiles of 32), n > 0
 *     runs its jobs on n persistent CTAs (at most one fewer than the jobs),
 *     each running its jobs in turn with the next one's start overlapping
 *     this one's end; 0 does so when
 *     every such row has at most 32 queries (verify rows) and there are at
 *     least two jobs per SM, on a grid a cost model picks (at most one CTA
 *     per SM), else one CTA per job; -1 always one CTA per job.
 *     Process-wide; n outside [-1, 1024] gives PA_ERR_INVALID_ARG.
 *   pa_launch_count(): kernels this library has launched in this process.
 *   pa_trace_enable(1): from now on every launch records a CUDA event before
 *     and after itself on its stream (at most 16384 launches are kept; the
 *     events are created by this call, on the current device);
 *     pa_trace_read() waits for the recorded events, returns per launch the
 *     kernel kind (pa_kernel_kind) and its duration in milliseconds, and
 *     clears the trace.  pa_trace_enable(0) stops recording.
 */
typedef enum {
  PA_KERNEL_KV_APPEND = 1,
  PA_KERNEL_DECODE = 2,
  PA_KERNEL_COMBINE = 3, /* reserved: the split merge is fused into PA_KERNEL_DECODE */
  PA_KERNEL_PREFILL = 4,
  PA_KERNEL_MERGE = 5,       /* pa_merge_lse; key ranges of pa_attention_varlen_q4 */
  PA_KERNEL_PREFIX = 6,      /* shared-prefix pass of pa_attention_varlen_shared_prefix */
  PA_KERNEL_PREFIX_MERGE = 7, /* merge of that pass's key-chunk partials */
  PA_KERNEL_COPY_BLOCKS = 8,  /* pa_copy_blocks */
  PA_KERNEL_DECODE_STEP = 9,  /* pa_decode_step */
  PA_KERNEL_KV_READ = 10,     /* pa_kv_read_q4 */
  PA_KERNEL_STEP_TABLES = 11, /* pa_step_tables */
  PA_KERNEL_NORM_ROPE = 12    /* pa_qk_norm_rope, pa_qk_norm_rope_append */
} pa_kernel_kind;

pa_status pa_set_decode_ctas(int32_t n);
pa_status pa_set_prefill_ctas(int32_t n);
/*
 * pa_plan_tile_grid(job_tiles, n_jobs, decode_slabs, sms, ctas) -- the
 * persistent CTA count the library picks for a batch's tensor-core jobs
 * (rows with qo_len > 1), computed on the host alone (no device is touched):
 * job_tiles[i] is job i's number of 128-key tiles in the kernel's job order
 * (for each kv head, the batch's 32-query tiles by decreasing key extent),
 * sms the device's SM count.  With decode_slabs > 0 (the batch's decode rows
 * hold that many 8 KiB (page, kv head) K+V slabs) it is the count beside the
 * decode launch that pa_set_prefill_ctas(0) leads to (0: the jobs first, one
 * CTA each); with decode_slabs = 0 the count for the jobs alone, which
 * pa_attention_varlen uses when every such row has at most 32 queries (0:
 * one CTA per job).  Ownership: job_tiles is read, *ctas written; both host
 * memory.  Errors: PA_ERR_INVALID_ARG for a null ctas, n_jobs outside
 * [0, 393216] (1536 query tiles x 256 kv heads), a null job_tiles with
 * n_jobs > 0, a tile count below 1, sms outside [1, 1024] or decode_slabs < 0
 * (*ctas is then 0).
 */
pa_status pa_plan_tile_grid(const int32_t* job_tiles, int32_t n_jobs, int64_t decode_slabs, int32_t sms,
                            int32_t* ctas);
/*
 * pa_plan_decode_grid(seq_lens, n_rows, num_kv_heads, sms, grid,
 * warp_granular) -- the decode launch pa_attention_varlen plans for a batch
 * of n_rows decode rows (qo_len 1, bf16 pages, no shared prefix, no rows with
 * qo_len > 1) of these seq_lens on a device of sms SMs, computed on the host
 * alone (no device is touched): *grid CTAs (0: nothing to do) of the
 * warp-granular decode kernel (*warp_granular = 1) or of the CTA-granular one
 * (0).  A grid forced by pa_set_decode_ctas applies here as in the call.
 * Ownership: seq_lens is read, *grid and *warp_granular written; all host
 * memory.  Errors: PA_ERR_INVALID_ARG for a null output, n_rows outside
 * [0, 1024], a null seq_lens with n_rows > 0, a seq_len below 1, num_kv_heads
 * outside [1, 256] or sms outside [1, 1024]; PA_ERR_UNSUPPORTED when no plan
 * fits the kernels' limits, as the call would return.
 */
pa_status pa_plan_decode_grid(const int32_t* seq_lens, int32_t n_rows, int32_t num_kv_heads, int32_t sms,
                              int32_t* grid, int32_t* warp_granular);
/*
 * pa_set_decode_fault_injection(on) -- a test of the bounded-wait path, off
 * (0) by default, process-wide.  With on = 1, decode launches of
 * pa_attention_varlen and pa_attention_varlen_shared_prefix over bf16 pages
 * use a diagnostic build of the decode kernel in which CTA 0 arms the
 * barrier of its second page without issuing that page's copies, and every
 * wait gives up after 1 ms instead of 2 s.  Nothing faults or hangs: the
 * waiting warps give up, record PA_ERR_DEVICE_TIMEOUT in the error word, let
 * the copies they did issue land and return; the other CTAs finish
 * normally.  What such a call leaves: the error word set; the outputs of
 * the rows whose keys CTA 0 holds undefined; for rows cut between CTAs, their
 * counters in the workspace non-zero -- zero the workspace before its next
 * use, as after any PA_ERR_DEVICE_* error.  on outside {0, 1} gives
 * PA_ERR_INVALID_ARG.
 */
pa_status pa_set_decode_fault_injection(int32_t on);
int64_t pa_launch_count(void);
pa_status pa_trace_enable(int32_t on);
pa_status pa_trace_read(int32_t* kinds, float* ms, int32_t capacity, int32_t* count);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
