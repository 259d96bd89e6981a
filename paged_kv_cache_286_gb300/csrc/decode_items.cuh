// Work items of the split-KV kernels (decode.cu for bf16 and E4M3 pools, decode_mx.cu for MXFP4
// pools): the parameters that the plan, the attention kernels and the merge share, how many items
// a sequence has, and how a CTA claims its next one.
#pragma once

#include "pa_common.cuh"

namespace pa {

struct DecodeParams {
  const __nv_bfloat16* q;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* qsl;
  int32_t* item_start;     // [S+1] item prefix sums over the sequences in item_order
  int32_t* item_order;     // [S] the sequences, those of the longest items first, or NULL: as they are
  int32_t* pf_item_start;  // [S+1] prefill item prefix sums over the runs in claim order
  int32_t* pf_order;       // [S] the runs with prefill items, longest item first
  int32_t* merge_start;    // [S+1] prefix sums of the rows the merge combines
  float* part_lse;
  float* part_o;
  void* out;
  WsHeader* hdr;
  int32_t max_blocks_per_seq;
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;           // q heads per kv head
  int32_t num_blocks;
  int32_t max_context_len;
  int32_t max_query_len;
  int32_t pblk;
  int32_t pmax;
  int32_t decode_max_query;  // longer query runs go to the prefill-tile path
  int32_t decode_max_rows;   // so do runs of more (token x head) rows than one decode tile
  int32_t rows_per_tile;   // 8 * RT of the decode kernel instance
  int32_t heads_per_item;  // HPI of the decode kernel instance
  int32_t out_bf16;
  float score_log2;        // scale * log2(e) (* k_scale for E4M3)
  float v_out_scale;       // v_scale for E4M3, else 1
  uint64_t* span;          // benchmark hook: [first CTA start, last CTA end] in ns, or NULL
  int32_t wait_at_end;     // launched after the prefill kernel: wait for it only at the end
  int32_t sms;             // SMs of the device (the plan's SM split)
  int32_t kv_tile_bytes;   // bytes of one (block, kv head) tile of K plus V
  uint64_t wait_ns;        // limit of every bounded wait
  int32_t skip_copy;       // test hook: item 0 leaves out its first tile copy (see pa.h)
  float* lse;              // [T][Hq] log2-domain log-sum-exp of every row, or NULL
  float* scores;           // [S][Hkv][score_rows][score_stride] log2-domain scores of the runs of
                           // up to score_rows rows (row = token x group + head), or NULL
  int32_t score_rows;
  int32_t score_stride;
  const int32_t* stage_pre;  // [S + 1] staged blocks (mx_stage.cu): sequences that have some go to
                             // the prefill tiles, and no others; NULL: by decode_max_query / _rows
  float sm_rate;             // cost model: HBM bytes per microsecond of one SM's split-KV CTAs
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Partitions of a decode-path sequence of L keys.
__device__ __forceinline__ int partitions_of(const DecodeParams& p, int L) {
  return ceil_div(ceil_div(L, kBlockSize), p.pblk);
}

// Items of sequence s on the decode path (0 if it belongs to the prefill path or is invalid).
__device__ __forceinline__ int decode_items_of(const DecodeParams& p, int s, int n, int L,
                                               bool* bad) {
  *bad = false;
  if (n <= 0) {
    *bad = (n < 0);
    return 0;
  }
  if (n > L || L > p.max_context_len || n > p.max_query_len ||
      L > p.max_blocks_per_seq * kBlockSize) {
    *bad = true;
    return 0;
  }
  if (p.stage_pre ? p.stage_pre[s + 1] > p.stage_pre[s]
                  : n > p.decode_max_query || n * p.group > p.decode_max_rows)
    return 0;
  const int tpt = p.rows_per_tile / (p.group * p.heads_per_item);  // query tokens per tile
  const int qtiles = ceil_div(n, tpt);
  const int nparts = partitions_of(p, L);
  return p.num_kv_heads / p.heads_per_item * qtiles * nparts;
}

struct ItemInfo {
  int s, h, qt, part, t0, n, L, nparts, blk_begin, blk_end, pos_base, rows, valid, idx, run;
};

// Claims the next item from the step's counter: R rows per tile, HPI kv heads per item.
template <int R, int HPI>
__device__ __forceinline__ ItemInfo claim_item(const DecodeParams& p, int total_items) {
  ItemInfo info;
  const int item = static_cast<int>(atomicAdd(&p.hdr->decode_counter, 1u));
  info.valid = item < total_items;
  info.idx = item;
  if (info.valid) {
    int lo = 0, hi = p.num_seqs;  // largest s with item_start[s] <= item
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.item_start[mid] <= item) lo = mid; else hi = mid;
    }
    const int s = p.item_order ? p.item_order[lo] : lo;
    const int t0 = p.qsl[s];
    const int n = p.qsl[s + 1] - t0;
    const int L = p.context_lens[s];
    const int tpt = R / (p.group * HPI);
    const int istart = p.item_start[lo];
    const int qtiles = ceil_div(n, tpt);
    const int nblk = ceil_div(L, kBlockSize);
    const int nparts = ceil_div(nblk, p.pblk);
    int local = item - istart;
    const int part = local % nparts;
    local /= nparts;
    const int qt = local % qtiles;
    const int h = (local / qtiles) * HPI;                // first kv head of the item
    const int tok_begin = qt * tpt;
    const int tok_end = min(n, tok_begin + tpt);
    const int pos_max = L - n + tok_end - 1;           // last position in the tile
    const int blk_tile = pos_max / kBlockSize + 1;     // blocks the tile can see
    info.s = s; info.h = h; info.qt = qt; info.part = part; info.t0 = t0 + tok_begin;
    info.n = tok_end - tok_begin; info.L = L; info.nparts = nparts;
    info.blk_begin = min(part * p.pblk, blk_tile);
    info.blk_end = min((part + 1) * p.pblk, blk_tile);
    info.pos_base = L - n + tok_begin;                 // position of the tile's first token
    info.rows = info.n * p.group * HPI;
    info.run = n;                                      // query tokens of the whole run
  }
  return info;
}

}  // namespace pa
