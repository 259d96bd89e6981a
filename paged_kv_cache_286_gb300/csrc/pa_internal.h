// Host-side interfaces between the C-ABI layer (api.cu) and the kernel files.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <utility>

#include "pa.h"

namespace pa {

// Per-device launch facts of one kernel (SM count, resident CTAs per SM), with its dynamic
// shared-memory limit raised once per device: computed on first use and cached.
struct LaunchInfo {
  int sms = 0;
  int per_sm = 0;
};

// Cached per (kernel address, device): the function's C++ type is shared by every
// instantiation of a kernel template, so the key must be the address.
cudaError_t launch_info_impl(const void* kern, int threads, int smem_bytes, LaunchInfo* out);

template <typename Kernel>
cudaError_t launch_info(Kernel kern, int threads, int smem_bytes, LaunchInfo* out) {
  return launch_info_impl(reinterpret_cast<const void*>(kern), threads, smem_bytes, out);
}

// Where the keys and values of MXFP4 sequences with long query runs are written out as bf16 for
// the prefill tiles (mx_stage.cu); capacity 0: nowhere.
struct MxStage {
  int32_t* prefix = nullptr;   // [S + 1] prefix sums of the staged sequences' blocks
  int32_t* table = nullptr;    // [S][table_stride] block tables into the area
  void* k = nullptr;           // [capacity][Hkv][16][D] bf16
  void* v = nullptr;
  int32_t capacity = 0;        // blocks
  int32_t table_stride = 0;
};

// Everything pa_attention received, after host validation.
struct AttnArgs {
  const void* q;
  int32_t num_q_tokens;
  const void* k_cache;
  const void* v_cache;
  pa_cache_desc cache;
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  int32_t num_seqs;
  int32_t max_context_len;
  int32_t max_query_len;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  float scale;
  void* out;
  int32_t out_dtype;
  void* workspace;
  size_t workspace_bytes;
  cudaStream_t stream;
  cudaEvent_t pf_before = nullptr;  // benchmark hook: recorded around the prefill kernel
  cudaEvent_t pf_after = nullptr;
  uint64_t* span = nullptr;         // benchmark hook: kernel start / end times (pa.h)
  uint64_t wait_ns = 0;             // limit of every bounded device-side wait
  int32_t skip_copy = 0;            // test hook (pa_test_skip_one_copy)
  float* lse = nullptr;             // [T][Hq] log2-domain log-sum-exp of every row, or NULL
  float* scores = nullptr;          // scores of the split-KV path's rows, or NULL (DecodeParams)
  int32_t score_rows = 0;
  int32_t score_stride = 0;
  MxStage stage;                    // MXFP4 pools with long query runs
};

// Workspace carve-up; a pure function of the step's shape (see workspace_layout).
struct WsLayout {
  size_t item_start;  // int32 [num_seqs + 1], decode work-item prefix sums, by place in item_order
  size_t pf_item_start;  // int32 [num_seqs + 1], prefill work-item prefix sums, by claim rank
  size_t pf_order;    // int32 [num_seqs], the sequence of each prefill claim rank
  size_t merge_start;  // int32 [num_seqs + 1], prefix sums of the rows (token x q head) that
                       // the merge combines: those of split-KV sequences with 2+ partitions
  size_t item_order;  // int32 [num_seqs], the sequences in the order of their decode items
  size_t part_lse;    // float [num_q_tokens][num_q_heads][pmax], log2-domain log-sum-exp
  size_t part_o;      // float [num_q_tokens][num_q_heads][pmax][head_dim], normalised partials
  size_t total;
  int32_t pblk;       // blocks per KV partition
  int32_t pmax;       // partitions per sequence at most
};

// Bytes beyond the layouts above in which an MXFP4 step with long query runs stages their keys and
// values: what they can be at most, but no more than 256 MiB (sequences past that take the split-KV
// kernel).  0 for steps without such runs.
size_t mx_stage_bytes(int32_t num_seqs, int32_t num_q_tokens, int32_t num_q_heads,
                      int32_t num_kv_heads, int32_t head_dim, int32_t max_context_len,
                      int32_t max_query_len);

WsLayout workspace_layout(int32_t num_seqs, int32_t num_q_tokens, int32_t num_q_heads,
                          int32_t num_kv_heads, int32_t head_dim, int32_t max_context_len,
                          int32_t max_query_len);

// The attention's workspace followed by what the key weights need.
struct KeyWeightsLayout {
  size_t lse;          // float [num_q_tokens][num_q_heads], log2 domain
  size_t scores;       // float [num_seqs][num_kv_heads][score_rows][score_stride]
  int32_t score_rows;  // 0: none are kept
  int32_t score_stride;
  size_t chunk_start;  // int32 [num_seqs + 1], prefix sums of the sequences' key chunks
  size_t total;
};
KeyWeightsLayout key_weights_layout(int32_t num_seqs, int32_t num_q_tokens, int32_t num_q_heads,
                                    int32_t num_kv_heads, int32_t head_dim,
                                    int32_t max_context_len, int32_t max_query_len);

cudaError_t launch_cache_append(const void* k, const void* v, const int64_t* slots,
                                int32_t num_tokens, void* k_cache, void* v_cache,
                                const pa_cache_desc& c, uint32_t* err, cudaStream_t stream);

void set_last_error(const char* msg);

// Host checks of pa_attention's arguments other than the workspace (clears, then sets, the
// calling thread's last error).  *nothing is set when the step has no query token or sequence.
pa_status check_attention_args(const void* q, int32_t num_q_tokens, const void* k_cache,
                               const void* v_cache, const pa_cache_desc* cache,
                               const int32_t* block_tables, int32_t max_blocks_per_seq,
                               const int32_t* context_lens, const int32_t* query_start_loc,
                               int32_t num_seqs, int32_t max_context_len, int32_t max_query_len,
                               int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                               float scale, const void* out, int32_t out_dtype, bool* nothing);

cudaError_t launch_cache_read(const int64_t* slots, int32_t num_tokens, const void* k_cache,
                              const void* v_cache, const pa_cache_desc& c, void* k_out,
                              void* v_out, bool out_bf16, uint32_t* err, cudaStream_t stream);

// Arguments of the eviction kernels (evict.cu).
struct EvictArgs {
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int32_t* block_tables;
  const int32_t* dst_tables;
  const int32_t* context_lens;
  const int32_t* keep_lens;
  float* key_weights;       // [num_weight_rows][Hkv][max_keys]
  const int32_t* weight_rows;
  const int32_t* dst_weight_rows;
  int32_t* kept;            // [S][Hkv][max_keep_len]
  int32_t* new_lens;        // [S]
  uint32_t* err;
  int32_t num_seqs, num_blocks, num_kv_heads, head_dim, cache_dtype, max_blocks_per_seq;
  int32_t max_context_len, max_keep_len, recent, num_weight_rows, max_keys;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

cudaError_t launch_wait_timeout_selftest(uint32_t* err, uint64_t limit_ns, cudaStream_t stream);

cudaError_t launch_copy_blocks(void* k_cache, void* v_cache, const pa_cache_desc& c,
                               const int32_t* pairs, int32_t num_pairs, uint32_t* err,
                               cudaStream_t stream);

// True when chunks with more than kDecodeMaxQuery queries run on the tcgen05 tile kernel
// (bf16 pool of head_dim 128 or 64, or E4M3 of 128; GQA group dividing 128); otherwise every
// sequence takes the split-KV kernel.
// Kv heads per split-KV work item (1 or 2) for a step of this shape; the pool's tensor maps
// then take boxes of 16 x that many rows.
int decode_heads_per_item(const pa_cache_desc& c, int32_t num_q_heads, int32_t num_kv_heads,
                          int32_t max_query_len);
bool prefill_geometry(int32_t num_q_heads, int32_t num_kv_heads);  // its heads' part of that
bool prefill_path_enabled(const pa_cache_desc& c, int32_t num_q_heads, int32_t num_kv_heads);

// `qmap` (3-D view of q) is needed only when the prefill path is enabled and
// max_query_len > kDecodeMaxQuery; it may be NULL otherwise.
// Launch with programmatic stream serialization: the kernel may start while the previous kernel
// of the stream finishes, and waits (grid_dependency_wait) before reading its results.
template <typename... Params, typename... Args>
inline cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, dim3 block, int smem,
                                    cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

struct PoolMaps;
cudaError_t launch_attention(const AttnArgs& a, const WsLayout& ws, const PoolMaps& maps,
                             bool prefill, cudaEvent_t before, cudaEvent_t after);

// Arguments of the key-weight kernels (key_weights.cu): the step's, the rows' log-sum-exps and
// the weights.
struct KeyWeightsArgs {
  const __nv_bfloat16* q;
  const uint8_t* k_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* qsl;
  const float* lse;         // [T][Hq], log2 domain
  const float* scores;      // of the runs of up to score_rows rows (DecodeParams), or NULL
  int32_t score_rows, score_stride;
  int32_t chunk_keys;       // keys of an item of that kernel (set by launch_key_weights)
  int32_t k_pass;           // some run may have more rows than that: the kernel that reads K runs
  const int32_t* weight_rows;
  float* key_weights;       // [num_weight_rows][Hkv][max_keys]
  int32_t* chunk_start;     // [S + 1] scratch
  uint32_t* err;
  int32_t num_seqs, num_blocks, max_blocks_per_seq, max_context_len, max_query_len;
  int32_t num_q_heads, num_kv_heads, head_dim, cache_dtype;
  int32_t num_weight_rows, max_keys;
  float score_log2, decay;
  uint64_t wait_ns;         // limit of every bounded wait
  int32_t skip_copy;        // test hook (pa_test_skip_one_copy)
};
struct PoolMaps;
// `maps`: of q and K for the tensor-core kernel (bf16 pools with enough items), or NULL.
constexpr int kKeyWeightsTcKeys = 256;  // keys of an item of the tensor-core kernel
cudaError_t launch_key_weights(KeyWeightsArgs a, const PoolMaps* maps, cudaStream_t stream);
cudaError_t launch_key_weights_tc(const KeyWeightsArgs& a, const PoolMaps& maps,
                                  cudaStream_t stream);

struct DecodeParams;
// MXFP4 pools (decode_mx.cu): row tiles of 8 rows of an item, and the attention kernel.
int mx_row_tiles(int32_t max_query_len, int32_t group);
int mx_heads_per_item(const AttnArgs& a, const DecodeParams& p, int min_pblk, int* pblk);
// Sequences with more rows than its tiles: bf16 copies of their keys and values.
cudaError_t launch_mx_stage_plan(const AttnArgs& a, const DecodeParams& p);
cudaError_t launch_mx_stage(const AttnArgs& a, const DecodeParams& p);
cudaError_t launch_decode_mx(const AttnArgs& a, int pmax, const DecodeParams& p);

struct WsHeader;

// Parameters of the tensor-core prefill kernels (prefill.cu, chunk.cu).
struct PrefillParams {
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* qsl;
  const int32_t* item_start;  // [S+1] prefix sums of prefill items over the runs in claim order
  const int32_t* order;       // [S] the sequence of each run in claim order
  void* out;
  WsHeader* hdr;
  int32_t max_blocks_per_seq;
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;
  int32_t num_blocks;
  int32_t out_bf16;
  float score_log2;   // scale * log2(e) (* k_scale for E4M3 pools)
  float v_out_scale;  // v_scale for E4M3 pools, else 1
  uint64_t wait_ns;   // limit of every bounded wait
  int32_t skip_copy;  // test hook: the first item claimed leaves out its first K copy
  uint64_t* span;     // benchmark hook: [first CTA start, last CTA end] in ns, or NULL
  float* part_lse;       // [T][Hq][pmax] log2-domain log-sum-exp of split partials
  float* part_o;         // [T][Hq][pmax][128] normalised split partials
  int32_t pmax;          // partials per row the workspace holds (>= the splits of a pair)
  float* lse;            // [T][Hq] log2-domain log-sum-exp of rows that are not split, or NULL
};

// Where split prefill tiles keep their partials (the workspace's split-KV arrays).
struct PrefillScratch {
  float* part_lse;
  float* part_o;
  int32_t pmax;
};


// Tensor maps of one call: the pool as 2-D rows (split-KV kernel, verify tiles), the pool as
// 4-D whole (block, kv head) tiles and q as 3-D tiles (prefill kernels; NULL when unused).
struct PoolMaps {
  CUtensorMap k2, v2, k4, v4, q3;
  bool has_k4 = false, has_q3 = false;
};

cudaError_t launch_prefill(const AttnArgs& a, const int32_t* item_start, const int32_t* order,
                           WsHeader* hdr,
                           const PoolMaps& maps, const PrefillScratch& scratch);


}  // namespace pa
