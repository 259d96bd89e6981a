/*
 * pa.h -- C ABI of the paged-KV attention step (libpagedattn.so, CUDA, sm_103a).
 *
 * One continuous-batching attention step over a paged KV cache has two calls:
 *
 *   pa_cache_append  writes each new token's key and value into its slot of the block pool.
 *                    "Serving LLMs with vLLM: Continuous Batching and PagedAttention
 *                    Explained", section "Growing During Decode": each step appends the token
 *                    into the last block of its sequence; section "Blocks and Block Tables":
 *                    blocks are fixed-size (e.g. 16 tokens) and found through a per-sequence
 *                    block table.  The caller has already folded the table into a slot.
 *
 *   pa_attention     attends a ragged batch of query tokens (decode tokens and chunked-prefill
 *                    pieces) to their own sequence's keys and values, fetched block by block
 *                    through the block tables.  Same page, section "Attention Over Scattered
 *                    Blocks": the mathematics is ordinary attention, softmax of the query times
 *                    the keys over the whole history; only the addressing changes.  Sections
 *                    "Prefill Versus Decode" and "Chunked Prefill": one step mixes prompt chunks
 *                    with decode tokens.  Section "Shared Prefixes": several tables may point at
 *                    the same physical blocks.
 *
 * Conventions shared by every call
 *   - Memory: every pointer argument named *_cache, q, k, v, out, slot_mapping, block_tables,
 *     context_lens, query_start_loc, key_weights and workspace is a DEVICE pointer on the current device.
 *     `cache` descriptors are HOST pointers.  The caller allocates and owns all of it; the
 *     library never allocates or frees device memory.  A workspace serves one call at a time: calls
 *     (or captured graphs of them) whose GPU work may overlap need one each.
 *   - Execution: calls are asynchronous on `stream` (0 = legacy default stream) and ordered by
 *     it; nothing synchronises the host except pa_check_error.  pa_cache_append must precede
 *     pa_attention on the same stream when the step's new tokens are to be attended.
 *   - Errors: argument errors are detected on the host and returned before anything is
 *     launched (PA_ERR_INVALID_ARG / PA_ERR_UNSUPPORTED).  Errors that only the device can see
 *     (a block id or slot outside the pool, inconsistent lengths, an internal wait that timed
 *     out) make the kernel skip the offending access and set a bit in the error word held in
 *     the first bytes of `workspace`; pa_check_error reports and clears it.  No call traps,
 *     aborts or hangs on bad input.  pa_last_error_string describes the last host-side error
 *     of the calling thread.
 *
 * Layouts (all row-major, contiguous)
 *   block pool:  k_cache, v_cache = [num_blocks][num_kv_heads][block_size][head_dim], elements
 *                bf16, or OCP E4M3 bytes holding x / k_scale (resp. v_scale) with fp32 per-tensor
 *                scales.  One (block, kv head) tile of block_size x head_dim is contiguous.
 *                PA_MXFP4 pools (microscaled 4-bit floating point): 32 neighbouring dims of a row
 *                share a scale byte e (E8M0: 2^(e - 127), 255 = NaN, with codes of zero), and a dim
 *                is a 4-bit E2M1 code c (0 .5 1 1.5 2 3 4 6, bit 3 the sign): value = code *
 *                2^(e - 127), subnormal results included.  One
 *                (block, kv head) tile is 17 * head_dim / 2 contiguous bytes: 16 rows of
 *                head_dim / 2 bytes of codes, then 16 rows of head_dim / 32 scale bytes.  With
 *                nb = head_dim / 32, 16-bit word g * nb + b of a row (little endian) holds dims
 *                32 b + 4 g .. 32 b + 4 g + 3, the lowest dim in its lowest four bits.
 *   slot:        physical_block * block_size + offset; a negative slot means "skip".
 *   new k, v:    [num_tokens][num_kv_heads][head_dim] bf16.
 *   q, out:      [num_q_tokens][num_q_heads][head_dim]; q bf16, out fp32 or bf16.
 *   block_tables [num_seqs][max_blocks_per_seq] int32; entries past ceil(context_len/block_size)
 *                are never read.
 *   context_lens [num_seqs] int32: keys of the sequence after this step's append.
 *   query_start_loc [num_seqs + 1] int32: exclusive prefix sum of per-sequence query counts
 *                n_s, starting at 0.  The n_s queries of sequence s are its last n_s positions
 *                p_i = context_len - n_s + i, and query i attends keys 0..p_i.
 *   GQA:         q head h reads kv head h / (num_q_heads / num_kv_heads); groups of up to 16
 *                q heads per kv head are built.
 */
#ifndef PAGED_KV_PA_H_
#define PAGED_KV_PA_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,  /* null pointer, negative size, inconsistent shapes, small workspace */
  PA_ERR_UNSUPPORTED = 2,  /* valid but not built: head_dim, block_size, dtype or GQA group */
  PA_ERR_OUT_OF_RANGE = 3, /* device saw a block id or slot outside the pool, or bad lengths */
  PA_ERR_TIMEOUT = 4,      /* a bounded device-side wait gave up (results are not valid) */
  PA_ERR_CUDA = 5          /* a CUDA runtime call failed; see pa_last_error_string */
} pa_status;

typedef enum { PA_BF16 = 0, PA_FP8_E4M3 = 1, PA_FP32 = 2, PA_MXFP4 = 3 } pa_dtype;

/* Geometry of one pool (both k_cache and v_cache).  Supported: block_size 16; head_dim 64 or
 * 128 for bf16 and PA_MXFP4, 128 for PA_FP8_E4M3; num_blocks * num_kv_heads * block_size (the pool's rows)
 * at most 2^31 - 1.  k_scale / v_scale are used only for PA_FP8_E4M3. */
typedef struct {
  int32_t num_blocks;
  int32_t block_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t cache_dtype; /* pa_dtype: PA_BF16, PA_FP8_E4M3 or PA_MXFP4 */
  float k_scale;
  float v_scale;
} pa_cache_desc;

/* Bytes at the start of every workspace that hold the device error word; a workspace passed
 * to pa_cache_append needs at least this many bytes (pa_attention's workspace qualifies). */
#define PA_WORKSPACE_HEADER_BYTES 256

/* Device error-word bits (pa_check_error maps them to its status and returns the raw word
 * through its word_out argument). */
#define PA_DEVERR_BLOCK_ID 0x1u    /* block table entry outside [0, num_blocks) */
#define PA_DEVERR_SLOT 0x2u        /* slot >= num_blocks * block_size */
#define PA_DEVERR_LENGTHS 0x4u     /* n_s < 0, n_s > context_len, or a host hint exceeded */
#define PA_DEVERR_TIMEOUT 0x8u     /* bounded wait expired */
#define PA_DEVERR_WEIGHT_ROW 0x10u /* weight row >= num_weight_rows */

/* Scatter new keys/values into the pool.
 *   k, v          [num_tokens][num_kv_heads][head_dim] bf16 (device).
 *   slot_mapping  [num_tokens] int64 (device); slot of token t; < 0 skips the token.
 *   k_cache, v_cache  pool tensors described by `cache` (device, written in place).
 *   workspace     >= PA_WORKSPACE_HEADER_BYTES bytes (device); receives PA_DEVERR_SLOT.
 * bf16 pools receive the bits unchanged.  E4M3 pools receive, per element, the E4M3 encoding
 * (round to nearest even, saturating to +-448) of the fp32 quotient x / scale rounded to
 * nearest.  MXFP4 pools receive, per block of 32 dims, the scale 2^e with e = floor(log2(amax)) -
 * 2 (at least -127; amax the block's largest magnitude) and, per element, x / 2^e rounded to the
 * nearest E2M1 value (ties to the even code, saturating at +-6); a block with a NaN receives the
 * NaN scale and zero codes.  num_tokens == 0 is a no-op.  A slot written twice in one call ends up
 * holding one of the writes; in an MXFP4 pool its codes and scales may be of different ones, so
 * there a call's slots must differ. */
pa_status pa_cache_append(const void* k, const void* v, const int64_t* slot_mapping,
                          int32_t num_tokens, void* k_cache, void* v_cache,
                          const pa_cache_desc* cache, void* workspace, cudaStream_t stream);

/* Read slots back: the values that the pool holds for slot_mapping[t], rounded once to out_dtype
 * (exact for bf16 and MXFP4 pools, and in fp32 for E4M3 up to the product with its scale).
 *   slot_mapping  [num_tokens] int64 (device).  The rows of a negative slot are zeros, and so are
 *                 those of a slot past the pool, which also sets PA_DEVERR_SLOT.
 *   k, v          [num_tokens][num_kv_heads][head_dim], out_dtype PA_FP32 or PA_BF16 (device).
 *   workspace     >= PA_WORKSPACE_HEADER_BYTES bytes (device). */
pa_status pa_cache_read(const int64_t* slot_mapping, int32_t num_tokens, const void* k_cache,
                        const void* v_cache, const pa_cache_desc* cache, void* k, void* v,
                        int32_t out_dtype, void* workspace, cudaStream_t stream);

/* Copy whole blocks inside the pool: for each pair i, block block_pairs[2i] (source) is copied
 * to block block_pairs[2i+1] (destination), all kv heads, K and V, bit for bit.
 * "Serving LLMs with vLLM: Continuous Batching and PagedAttention Explained", section
 * "Copy-on-Write": before a sequence writes into a shared block, the engine copies it to a
 * fresh block and points only that sequence's table at the copy.
 *   block_pairs  [num_pairs][2] int32 (device); num_pairs <= 65535.
 *   workspace    >= PA_WORKSPACE_HEADER_BYTES bytes (device); a block id outside the pool sets
 *                PA_DEVERR_BLOCK_ID and that pair is skipped.
 * Pairs must not overlap (no block is both a source and a destination, no destination twice);
 * otherwise the result is undefined. */
pa_status pa_copy_blocks(void* k_cache, void* v_cache, const pa_cache_desc* cache,
                         const int32_t* block_pairs, int32_t num_pairs, void* workspace,
                         cudaStream_t stream);

/* Workspace bytes pa_attention needs for a step of this shape (host-only, no device call).
 * max_context_len / max_query_len are upper bounds of context_lens[s] and n_s. */
size_t pa_attention_workspace_size(int32_t num_seqs, int32_t num_q_tokens, int32_t num_q_heads,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                   int32_t max_context_len, int32_t max_query_len);

/* The same for a pool of the given cache_dtype, with what makes its steps fast: for PA_MXFP4 and runs
 * of more than 32 (token x q head) rows up to 256 MiB more, for the bf16 copies that pa_attention then
 * makes.  For other pools it is pa_attention_workspace_size. */
size_t pa_attention_workspace_size_for(int32_t cache_dtype, int32_t num_seqs, int32_t num_q_tokens,
                                       int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                       int32_t block_size, int32_t max_context_len,
                                       int32_t max_query_len);

/* Ragged paged attention of one step.
 *   q             [num_q_tokens][num_q_heads][head_dim] bf16 (device).
 *   k_cache, v_cache, cache   the pool (device / host descriptor).
 *   block_tables  [num_seqs][max_blocks_per_seq] int32 (device).
 *   context_lens  [num_seqs] int32 (device).  query_start_loc [num_seqs + 1] int32 (device),
 *                 query_start_loc[num_seqs] must equal num_q_tokens.
 *   max_context_len, max_query_len   host upper bounds of context_lens and n_s (checked on
 *                 the device; a violation sets PA_DEVERR_LENGTHS and skips that sequence).
 *   scale         multiplies q.k before the softmax (e.g. 1/sqrt(head_dim)).
 *   out           [num_q_tokens][num_q_heads][head_dim], out_dtype PA_FP32 or PA_BF16 (device).
 *   workspace     device buffer of workspace_bytes >= pa_attention_workspace_size(...); its
 *                 first PA_WORKSPACE_HEADER_BYTES hold the error word.
 * A sequence with n_s == 0 produces nothing.  Accumulation is fp32; scores use exp2 of
 * log2(e)-prescaled logits.
 * Kernels: every kernel of the call runs on `stream`, each launched early (programmatic
 * dependent launch) and waiting for what it reads: a plan, then, with a bf16 pool of head_dim
 * 128 or 64 or an E4M3 pool of head_dim 128 and query runs of more than 16 tokens or more than
 * 16 (token x q head) rows, the tensor-core prefill tiles on the part of the SMs the plan gives
 * them, the split-KV kernel on the rest, and the merge of split sequences.
 * MXFP4 pools have their own split-KV kernel for runs of up to 32 (token x q head) rows.  The
 * sequences of longer runs are written out as bf16 into the end of the workspace and go to the
 * prefill tiles, if the heads allow those (128 divisible by the group, at most 8); a workspace of
 * pa_attention_workspace_size_for holds all of that copy (up to its limit); a smaller one, down to
 * pa_attention_workspace_size, is accepted, and the split-KV kernel then also takes the runs for
 * whose sequences it has no room.
 * Work enqueued on `stream` after the call sees all of it complete.  The call records no event
 * and creates no stream, so it can be captured into a CUDA graph like any kernel launch. */
pa_status pa_attention(const void* q, int32_t num_q_tokens, const void* k_cache,
                       const void* v_cache, const pa_cache_desc* cache,
                       const int32_t* block_tables, int32_t max_blocks_per_seq,
                       const int32_t* context_lens, const int32_t* query_start_loc,
                       int32_t num_seqs, int32_t max_context_len, int32_t max_query_len,
                       int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                       void* out, int32_t out_dtype, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream);

/* Workspace bytes pa_attention_key_weights needs for a step of this shape (host-only): what
 * pa_attention needs, the rows' log-sum-exps, and, where they are at most 1 GiB, the scores of the
 * decode tokens and short runs (with more, those runs' keys are read a second time). */
size_t pa_attention_key_weights_workspace_size(int32_t num_seqs, int32_t num_q_tokens,
                                               int32_t num_q_heads, int32_t num_kv_heads,
                                               int32_t head_dim, int32_t block_size,
                                               int32_t max_context_len, int32_t max_query_len);

/* The same for a pool of the given cache_dtype (see pa_attention_workspace_size_for). */
size_t pa_attention_key_weights_workspace_size_for(int32_t cache_dtype, int32_t num_seqs,
                                                   int32_t num_q_tokens, int32_t num_q_heads,
                                                   int32_t num_kv_heads, int32_t head_dim,
                                                   int32_t block_size, int32_t max_context_len,
                                                   int32_t max_query_len);

/* pa_attention that also accumulates how much attention every cached key received, the measure by
 * which pa_evict_keys chooses.  Of a sequence s with query tokens, for every kv head h and key j
 * of its context_lens[s] keys:
 *   W[row][h][j] <- decay * W[row][h][j] + sum of the softmax weights of key j over the step's
 *                   query tokens that attend it and the q heads of h's group.
 *   key_weights   [num_weight_rows][num_kv_heads][max_keys] fp32 (device), updated in place;
 *                 max_keys >= max_context_len.  A caller zeroes a row when a sequence starts to
 *                 use it: positions appended later then begin at 0.
 *   weight_rows   [num_seqs] int32 (device): the row of each sequence, or NULL for row s.  The
 *                 weights of a sequence with a negative row, or without query tokens, are left as
 *                 they are; a row >= num_weight_rows sets PA_DEVERR_WEIGHT_ROW and is skipped.
 *                 Two sequences must not share a row: it ends up with one of the results.
 *   decay         >= 0; 1 sums over all steps.
 * The other arguments, the output and the errors are pa_attention's (a sequence that it skips
 * accumulates nothing; nor does a key in a block outside the pool).  The sums are fp32 and their
 * order is fixed: the same call gives the same bits.
 * If a wait of the attention runs out (PA_DEVERR_TIMEOUT), the weights stay as they are, and so they
 * do in later calls until pa_check_error has cleared the error word.  If a wait of the accumulation
 * itself runs out, some of the step's keys have their sums and others do not: the rows of its
 * sequences are lost, and the caller zeroes them. */
pa_status pa_attention_key_weights(
    const void* q, int32_t num_q_tokens, const void* k_cache, const void* v_cache,
    const pa_cache_desc* cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* context_lens, const int32_t* query_start_loc, int32_t num_seqs,
    int32_t max_context_len, int32_t max_query_len, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, float scale, void* out, int32_t out_dtype, float* key_weights,
    const int32_t* weight_rows, int32_t num_weight_rows, int32_t max_keys, float decay,
    void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes pa_evict_keys needs (host-only). */
size_t pa_evict_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t max_context_len,
                               int32_t max_keep_len);

/* Drop the keys that received the least attention.  Of a sequence's L = context_lens[s] keys, k =
 * min(keep_lens[s], L) stay, chosen per kv head: the last min(recent, k) and, of the others, those
 * of the largest key_weights (ties: the lowest position; NaN counts as -infinity).  Kept keys
 * and values move, in their order, to positions 0 .. k - 1 of dst_tables; a later step attends
 * them with context_lens[s] = new_lens[s] (and its new tokens after them).
 *   block_tables  [num_seqs][max_blocks_per_seq] int32 (device): where the keys are.
 *   dst_tables    the same shape: where they go, or NULL for block_tables (in place).  Entry i may
 *                 be block_tables' entry i, or a block that no sequence of the call reads; no
 *                 block may be a destination of two sequences, and none that another sequence
 *                 reads may be a destination (one pa_bm_evict_batch call gives such tables for its
 *                 sequences; several pa_bm_evict calls do not); otherwise the blocks' contents are
 *                 undefined.  (A key that keeps its place is neither read nor written.)
 *   keep_lens     [num_seqs] int32 (device), >= 0.
 *   max_context_len, max_keep_len   host upper bounds of context_lens and of k.
 *   key_weights, weight_rows, num_weight_rows, max_keys   as in pa_attention_key_weights.  The
 *                 weights of the kept keys move with them to row dst_weight_rows[s] (NULL: the
 *                 same row), whose positions k .. L - 1 become 0; later positions stay as they
 *                 are.  A destination row must not be another sequence's row of either kind.
 *   kept          [num_seqs][num_kv_heads][max_keep_len] int32 (device): the old positions of the
 *                 kept keys, ascending, then -1.
 *   new_lens      [num_seqs] int32 (device): k.  It may not overlap context_lens, keep_lens or the
 *                 row tables.
 *   workspace     >= pa_evict_workspace_size(...) bytes (device).
 * Built for the caches that pa_attention reads.
 * A sequence with a negative length, more keys than max_context_len or its table hold, a k above
 * max_keep_len (PA_DEVERR_LENGTHS), or a row past key_weights (PA_DEVERR_WEIGHT_ROW) or negative
 * (no error) is left as it is: its new_lens is its context length and its kept are -1.  A block
 * outside the pool sets PA_DEVERR_BLOCK_ID and its keys do not move. */
pa_status pa_evict_keys(void* k_cache, void* v_cache, const pa_cache_desc* cache,
                        const int32_t* block_tables, const int32_t* dst_tables,
                        int32_t max_blocks_per_seq, const int32_t* context_lens,
                        const int32_t* keep_lens, int32_t num_seqs, int32_t max_context_len,
                        int32_t max_keep_len, int32_t recent, float* key_weights,
                        const int32_t* weight_rows, const int32_t* dst_weight_rows,
                        int32_t num_weight_rows, int32_t max_keys, int32_t* kept,
                        int32_t* new_lens, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream);

/* Scratch bytes built into the library for pa_attention_noalloc (32 MiB per device). */
#define PA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

/* pa_attention for callers that cannot allocate device memory.  (The pages have no
 * counterpart: this is a library convenience, not part of the method.)
 *
 * Some callers are not allowed to call cudaMalloc: code running under a memory manager that
 * owns all device memory, code that must not grow its footprint after start-up, or code on a
 * path where an allocation could stall the device.  They can still pass inputs and outputs but
 * not a workspace, so this call uses a scratch array built into the library instead:
 * PA_NOALLOC_SCRATCH_BYTES per device, held by every GPU that loads the library until the
 * process exits.  A step whose pa_attention_workspace_size exceeds it is rejected with
 * PA_ERR_INVALID_ARG and a message; use pa_attention with a workspace for larger steps.
 *   Arguments are those of pa_attention without workspace/workspace_bytes, plus
 *   error_word    optional DEVICE pointer (may be NULL) that receives, asynchronously on
 *                 `stream`, this call's PA_DEVERR_* bits (0 for a step with nothing to do).  It
 *                 is written only when the call returns PA_OK; a call rejected on the host
 *                 changes neither *error_word nor the scratch array.
 * Each call looks up the scratch array's device address in the current context
 * (cudaGetSymbolAddress); the first lookup in a context may load the library's device code, so
 * make the first call before any stream capture.  Every call shares the
 * one array and overwrites it, starting from a cleared header: calls whose GPU work overlaps
 * (other streams, other threads) race on it and must be serialised by the caller. */
pa_status pa_attention_noalloc(const void* q, int32_t num_q_tokens, const void* k_cache,
                               const void* v_cache, const pa_cache_desc* cache,
                               const int32_t* block_tables, int32_t max_blocks_per_seq,
                               const int32_t* context_lens, const int32_t* query_start_loc,
                               int32_t num_seqs, int32_t max_context_len, int32_t max_query_len,
                               int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                               float scale, void* out, int32_t out_dtype, uint32_t* error_word,
                               cudaStream_t stream);

/* Synchronise `stream`, read and clear the device error word at the start of `workspace`.
 * Returns PA_OK, PA_ERR_OUT_OF_RANGE (block id / slot / length bits), PA_ERR_TIMEOUT, or
 * PA_ERR_CUDA.  *word_out (may be NULL) receives the raw PA_DEVERR_* bits. */
pa_status pa_check_error(void* workspace, cudaStream_t stream, uint32_t* word_out);

/* Zero the error word (asynchronously, on `stream`).  Call once on a fresh workspace. */
pa_status pa_workspace_init(void* workspace, cudaStream_t stream);

/* Text of the calling thread's last host-side error ("" if none). */
const char* pa_last_error_string(void);

/* Library version, e.g. "0.1.0". */
const char* pa_version(void);

/* Benchmark hook.  When both events are non-NULL (cudaEvent_t handles), every later
 * pa_attention call of the calling thread records `before` immediately before, and `after`
 * immediately after, its split-KV attention kernel, on the call's stream.  An event between
 * two of the call's kernels makes the later one wait for the earlier one to finish, so with
 * these events the kernels run one after the other and each is timed alone.  Pass NULLs to
 * stop. */
void pa_set_kernel_timing_events(void* before, void* after);

/* Benchmark hook, like pa_set_kernel_timing_events, for the tensor-core prefill-tile kernel
 * (launched only by steps that hold runs of more than 16 tokens or 16 token x head rows over a
 * bf16 pool with head_dim 128 or 64).  Pass NULLs to stop. */
void pa_set_prefill_timing_events(void* before, void* after);

/* Benchmark hook that times kernels while they overlap: when `device_buffer` is non-NULL
 * (four uint64_t in device memory, set by the caller to {UINT64_MAX, 0, UINT64_MAX, 0}), every
 * later pa_attention call of the calling thread has its split-KV kernel lower [0] to the
 * GPU's global timer (ns) when a CTA starts and raise [1] to it when a CTA finishes its work,
 * and its prefill-tile kernel do the same with [2] and [3].  Pass NULL to stop. */
void pa_set_kernel_span_buffer(uint64_t* device_buffer);

/* Limit of every bounded device-side wait in the calling thread's later pa_attention calls, in
 * nanoseconds of the GPU's global timer; 0 restores the default of 1 s.  A wait that reaches
 * the limit gives up: the kernel sets PA_DEVERR_TIMEOUT, lets the copies it still has in flight
 * land (each with its own bounded wait), and returns; pa_check_error then reports
 * PA_ERR_TIMEOUT and that call's output is not valid.  (Not a step of the method: it bounds
 * how long a lost copy can hold the GPU.) */
void pa_set_wait_limit_ns(uint64_t ns);

/* Test hook, off by default; never enable it outside tests.  While enabled, every pa_attention
 * call of the calling thread leaves out exactly one tile copy of each attention kernel it
 * launches (the first copy of the first work item claimed) while that copy's barrier still
 * expects the bytes, so that the bounded waits on it expire and the call ends with
 * PA_ERR_TIMEOUT without any fault: the expiry and drain paths of the kernels can be exercised
 * on a real GPU.  2 leaves the attention kernels whole and does the same in
 * pa_attention_key_weights' tensor-core kernel over bf16 pools.  (The split-KV kernel of MXFP4 pools
 * has no wait that could run out and ignores the hook.) */
void pa_test_skip_one_copy(int32_t enable);

/* Self-test of the bounded wait: one thread waits, for limit_ns (in (0, 10 s]), on an mbarrier
 * phase that nothing completes, then sets PA_DEVERR_TIMEOUT in the error word at the start of
 * `workspace` (>= 4 bytes, device) and returns; read it with pa_check_error.  Asynchronous on
 * `stream`.  (Not a step of the method: it checks the library's failure signal.) */
pa_status pa_selftest_wait_timeout(void* workspace, uint64_t limit_ns, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_KV_PA_H_ */
