// Paged attention over MXFP4 pools: decode tokens, short query runs and prompt chunks.
//
// What it computes: softmax(scale * q . k_j) v_j over keys j <= p_i, where element d of key j is
// code[j][d] * 2^(e[j][d / 32] - 127) and the same for values (mxfp4.cuh has the tile).
//
//  * Work items, plan and merge are those of the split-KV kernel (decode.cu): an item is
//    (sequence, kv head, tile of 8 RT rows = tokens x heads of the group, KV partition), each of
//    the CTA's 4 warps takes every 4th block of the partition through its own ring of shared
//    memory stages, filled by 16-byte asynchronous copies of the whole warp: a tile is 68 of them
//    and contiguous, so it takes three instructions, and their completion one more, where an
//    elected lane's bulk copies with an mbarrier take some 60 issue slots a block.  (The codes are
//    a quarter of bf16's bytes: issue slots, not bytes in flight, are what this kernel runs out
//    of.)
//  * Two kv heads of a small group share an item and its tile of rows (below).
//  * The MMAs (m16n8k16, f16) have the keys (S^T = K q^T) and the head dims (O^T = V^T P^T) as M:
//    a block's 16 keys fill M where the rows would leave half of it empty, codes are converted
//    to f16 (exact) once for all row tiles, and S^T's accumulators become P^T's B operand by one
//    8 x 8 transpose per 8 keys.
//  * K: the two MMAs of a scale block accumulate into their own fp32 sum, which the block's scale
//    then multiplies: no rounding is added to the products.  q is f16, made exact by a power of
//    two per row.
//  * V: the value's scale goes into P, in fp32, before P is rounded to f16 (2^-12 relative, as in
//    the E4M3 kernel): P * 2^(e - R_b), where R_b is the largest exponent seen in scale block b
//    so far (moved only when a scale exceeds it by more than 2^7, when O's columns of the block
//    are rescaled).  Smaller scales lose nothing but what is below f16's subnormals, 2^-24 of
//    the block's largest scale.
//  * Measured: 256 sequences of 1,000 keys on average, 32 q heads on 8 of 128 dims: 93 us for 388 MB
//    of tiles (4.2 TB/s); 16 x 32,768 keys 106 us (5.4 TB/s).  A (block, kv head) takes some 270
//    warp instructions (conversions, scales, softmax, copies): half of the SM's issue slots and of
//    its ALU's, with dependent chains in three warps per scheduler for the rest, while DRAM waits.
//  * The softmax base of a row moves only when a score exceeds it by more than 2^8, so that the
//    usual block needs one warp vote and no maximum across lanes.
#include <math_constants.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "decode_items.cuh"
#include "mxfp4.cuh"
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

// max of three, NaN if one of them is
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int D, int RT, int HPI>
struct MxCfg {
  static constexpr int kStages = HPI == 1 && RT == 1 ? 4 : 3;
  static constexpr int kStageBytes = 2 * HPI * Mx<D>::kTileBytes;  // K tiles, then V tiles
  static constexpr int kOwn = HPI == 1 ? 32 : 64;  // blocks of an item that a warp can own
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kScratch = 8 * RT * D * 4 + 2 * 8 * RT * 4;  // O, max and sum of a warp
  static constexpr int kQBytes = RT * Mx<D>::kBlocks * 512;  // q fragments of an item
  static constexpr int kSmem = kDecodeWarps * (kWarpBytes + kScratch) + 2 * kQBytes +
                               2 * 8 * RT * 4 /*row scales*/ + 3 * 64 /*items*/ + 128 /*alignment*/ +
                               2 * kDecodeWarps * kOwn * 4 /*tiles*/;
  static constexpr int kCtas = RT == 1 ? (HPI == 1 ? 4 : 3) : RT == 2 ? 3 : 2;  // CTAs per SM
  static_assert(kStageBytes % 16 == 0 && sizeof(ItemInfo) <= 64, "");
  static_assert(HPI == 1 || RT == 1, "several heads per item use one 8-row tile");
};

// kScores: the scores of runs of up to kDecodeMaxRows rows are also written out, for the key
// weights (key_weights.cu): 256 sequences of 2,000 keys, 32 q heads on 8, 130 -> 158 us with the
// weights made of them.
// HPI kv heads per item: row r of a token is q head h * G + r, and the rows of head h + i take
// their scores from, and add P V into O from, head i's tiles alone.  A lane's two rows are of one
// head (an even group).
template <int D, int RT, int HPI, bool kScores>
__global__ void __launch_bounds__(kDecodeWarps * 32, MxCfg<D, RT, HPI>::kCtas)
    decode_mx_kernel(const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool,
                     const DecodeParams p) {
  using C = MxCfg<D, RT, HPI>;
  using M = Mx<D>;
  constexpr int NB = M::kBlocks;
  constexpr int NST = C::kStages;
  constexpr int R = 8 * RT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  float* scratch = reinterpret_cast<float*>(smem + kDecodeWarps * C::kWarpBytes);  // [warp]
  uint4* s_q = reinterpret_cast<uint4*>(smem + kDecodeWarps * (C::kWarpBytes + C::kScratch));
  float* s_scale = reinterpret_cast<float*>(s_q + 2 * C::kQBytes / 16);
  int* s_tile = reinterpret_cast<int*>(s_scale + 2 * R);  // [2][warp][kOwn]
  ItemInfo* s_item = reinterpret_cast<ItemInfo*>(s_tile + 2 * kDecodeWarps * C::kOwn);

  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int quad = lane >> 2;
  const int qc = lane & 3;
  uint8_t* wbuf = smem + warp * C::kWarpBytes;
  // Key of the block that row `quad` of the MMA's upper half stands for (quad + 8: that key + 8).
  // P^T's k indices 2 qc, 2 qc + 1 then are keys qc and 4 + (qc ^ 1), so that the lanes of one
  // shared memory access touch rows of both parities for K's 16-byte and for V's 8-byte loads
  // (natural order: V's conflict four ways).  With 64-byte rows, the 32-byte halves of V's rows
  // with bit 1 set are swapped on the way in, which makes V's loads free of conflicts.
  const int my_key = (quad & 1) ? 4 + ((quad >> 1) ^ 1) : quad >> 1;

  // after the prefill tiles (which waited for the plan) it starts beside them and waits for them
  // only before it ends
  if (!p.wait_at_end) grid_dependency_wait();
  if (p.span && threadIdx.x == 0)
    atomicMin(reinterpret_cast<unsigned long long*>(p.span),
              static_cast<unsigned long long>(global_ns()));
  const int total_items = p.item_start[p.num_seqs];
  // This lane's 16-byte pieces of a tile: `lane`, 32 + lane, ... ; where they land (V: swapped).
  // The few pieces past whole warps (64-wide: scale bytes) of all the stage's tiles go in one
  // instruction.
  constexpr int kPieces = M::kTileBytes / 16;
  constexpr int kFull = kPieces / 32, kTail = kPieces % 32;
  const uint32_t kdst = smem_u32(wbuf) + lane * 16;
  const uint32_t vdst = smem_u32(wbuf) + HPI * M::kTileBytes +
                        (NB == 4 ? lane ^ ((lane >> 3 & 1) << 1) : lane) * 16;
  static_assert(2 * HPI * kTail <= 32, "a lane per tail piece");
  const bool tail = lane < 2 * HPI * kTail;
  const int tail_tile = lane / kTail;  // K tiles, then V tiles
  const int64_t tail_at =
      (tail_tile % HPI) * M::kTileBytes + (32 * kFull + lane % kTail) * 16;
  const uint8_t* tail_src = (tail_tile < HPI ? k_pool : v_pool) + tail_at;
  const uint32_t tail_dst =
      smem_u32(wbuf) + tail_tile * M::kTileBytes + (32 * kFull + lane % kTail) * 16;
  // head of the item of this lane's rows 2 qc, 2 qc + 1, and of row `quad`
  const int my_head = HPI > 1 ? 2 * qc % (p.group * HPI) / p.group : 0;
  const int quad_head = HPI > 1 ? quad % (p.group * HPI) / p.group : 0;

  // Items follow one another without a pause of the copies: while an item runs, thread 0 claims
  // the one after the next, the next one's table entries and q fragments are brought in, and the
  // copies run on into its blocks.
  auto blocks_of = [&](const ItemInfo& I) {  // blocks of the item that are this warp's
    const int first = I.blk_begin + warp;
    return I.valid && first < I.blk_end ? ceil_div(I.blk_end - first, kDecodeWarps) : 0;
  };
  // (block, first kv head) tiles of the warp's blocks of the item, -1 for a bad one
  auto own_tiles = [&](int buf) { return s_tile + (buf * kDecodeWarps + warp) * C::kOwn; };
  auto find_tiles = [&](const ItemInfo& I, int nb, int buf) {
    for (int i = lane; i < nb; i += 32) {
      const int b = I.blk_begin + warp + i * kDecodeWarps;
      const int phys = __ldg(p.block_tables + static_cast<int64_t>(I.s) * p.max_blocks_per_seq + b);
      const bool there = phys >= 0 && phys < p.num_blocks;
      if (!there) set_error(&p.hdr->error, PA_DEVERR_BLOCK_ID);
      // (the pool has fewer than 2^31 rows)
      own_tiles(buf)[i] = there ? phys * p.num_kv_heads + I.h : -1;
    }
  };
  // copies of one block (tile < 0: none) into stage `to`, one group whatever is copied
  auto issue = [&](int tile, int to) {
    if (tile >= 0) {
      const int64_t at = static_cast<int64_t>(tile) * M::kTileBytes;
      const uint32_t so = to * C::kStageBytes;
      const uint8_t* ks = k_pool + at + lane * 16;
      const uint8_t* vs = v_pool + at + lane * 16;
#pragma unroll
      for (int hi = 0; hi < HPI; ++hi)
#pragma unroll
        for (int i = 0; i < kFull; ++i) {
          cp_async16(kdst + so + hi * M::kTileBytes + 512 * i, ks + hi * M::kTileBytes + 512 * i);
          cp_async16(vdst + so + hi * M::kTileBytes + 512 * i, vs + hi * M::kTileBytes + 512 * i);
        }
      if (tail) cp_async16(tail_dst + so, tail_src + at);
    }
    cp_async_commit();
  };
  // q fragments (B operand, n = row quad of the tile) of an item, one warp per row tile: of scale
  // block b, the pairs of dims 32 b + 8 qc + {0 1, 2 3} (first MMA) and {4 5, 6 7} (second), and
  // the rows' score scales.  They stay in shared memory: in registers they would cost a CTA per SM.
  static_assert(RT <= kDecodeWarps, "a warp per row tile");
  auto stage_q = [&](const ItemInfo& I, int buf) {
    if (warp >= RT) return;
    const int row = 8 * warp + quad;
    const bool ok = row < I.rows;
    const int tok = ok ? row / (p.group * HPI) : 0, g = ok ? row - tok * (p.group * HPI) : 0;
    const __nv_bfloat16* qrow =
        p.q + (static_cast<int64_t>(I.t0 + tok) * p.num_q_heads + I.h * p.group + g) * D;
    uint4 raw[NB];
    float amax = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      raw[b] = ok ? __ldg(reinterpret_cast<const uint4*>(qrow + 32 * b + 8 * qc))
                  : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        amax = fmaxf(amax, fmaxf(fabsf(bf16lo_to_f32(w[i])), fabsf(bf16hi_to_f32(w[i]))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // power of two e with amax * 2^e < 2^15 (f16 range), exact scaling; both 2^e and 2^-e are normal
    const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 126;  // -126 .. 129
    const int e = min(126, 15 - ex);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
      uint32_t f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i] = pack_f16x2(bf16lo_to_f32(w[i]) * up, bf16hi_to_f32(w[i]) * up);
      s_q[((buf * RT + warp) * NB + b) * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
    }
    if (qc == 0)
      s_scale[buf * R + row] = p.score_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  };

  if (threadIdx.x == 0) {
    s_item[0] = claim_item<R, HPI>(p, total_items);
    s_item[1] = claim_item<R, HPI>(p, total_items);
  }
  __syncthreads();
  int nb_w = blocks_of(s_item[0]);
  find_tiles(s_item[0], nb_w, 0);
  __syncwarp();
  if (s_item[0].valid) stage_q(s_item[0], 0);
  uint32_t there = 0;  // bit i: a tile was copied i issues ago
  for (int k = 0; k < NST - 1; ++k) {
    const int tile = k < nb_w ? own_tiles(0)[k] : -1;
    issue(tile, k);
    there = there << 1 | (tile >= 0 ? 1u : 0u);
  }
  int st = 0;       // stage of the block that comes next
  int slot = 0;     // item's place in s_item
  int buf = 0;      // its place in s_q and s_tile

  while (true) {
    __syncthreads();  // the item's q, the next item and the scratch are ready
    const ItemInfo I = s_item[slot];
    if (!I.valid) break;
    const int next_slot = slot == 2 ? 0 : slot + 1;
    int nb_next;
    {
      const ItemInfo N = s_item[next_slot];
      nb_next = blocks_of(N);
      find_tiles(N, nb_next, buf ^ 1);
      if (N.valid) stage_q(N, buf ^ 1);
    }
    if (threadIdx.x == 0) s_item[next_slot == 2 ? 0 : next_slot + 1] = claim_item<R, HPI>(p, total_items);
    const int my_first = I.blk_begin + warp;
    const int pos_last = I.pos_base + I.n - 1;
    const uint4* q_frag = s_q + buf * RT * NB * 32 + lane;  // [(rt * NB + b) * 32]
    float row_scale[RT][2];  // of rows 2 qc, 2 qc + 1 of each tile
    int row_pos[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        row_scale[rt][j] = s_scale[buf * R + 8 * rt + 2 * qc + j];
        row_pos[rt][j] = I.pos_base + (8 * rt + 2 * qc + j) / (p.group * HPI);
      }

    float m_run[RT][2], l_run[RT][2];  // base (log2 domain) and this lane's share of the sum
    float oacc[RT][2 * NB][4];         // [row tile][2 b + t]: dims 32 b + 4 quad + 2 t + {0, 1}
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m_run[rt][0] = m_run[rt][1] = -FLT_MAX;  // any score but -infinity exceeds it
      l_run[rt][0] = l_run[rt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j)
        oacc[rt][j][0] = oacc[rt][j][1] = oacc[rt][j][2] = oacc[rt][j][3] = 0.f;
    }
    // 2^(127 - R_b), R_b as a scale byte; R_b = 0: none yet (the first block with larger scales
    // sets it)
    float vinv[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) vinv[b] = __uint_as_float(254u << 23);

    // scores of this lane's first row and key: rows are (token, q head) of the head's run, so the
    // next row, and with one head per item row 8, follow at their stride
    [[maybe_unused]] float* my_scores = nullptr;
    if constexpr (kScores) {
      const int per_tok = p.group * HPI, row = 2 * qc;
      my_scores = p.scores + ((static_cast<int64_t>(I.s) * p.num_kv_heads + I.h + my_head) * p.score_rows +
                              (I.qt * (R / per_tok) + row / per_tok) * p.group +
                              (HPI == 1 ? row % per_tok : row % p.group)) * p.score_stride + my_key;
    }
    bool fresh = true;  // no block of the item is in O yet
    // One block: `diag` if some row of the item does not see some of its keys.
    auto tile_step = [&](int k, int st, auto diag_tag) {
      constexpr bool diag = decltype(diag_tag)::value;
        const int key0 = (my_first + k * kDecodeWarps) * kBlockSize;
        const uint8_t* kt = wbuf + st * C::kStageBytes;
        const uint8_t* vt = kt + HPI * M::kTileBytes;
        const uint8_t* kt_mine = kt + my_head * M::kTileBytes;  // of this lane's rows' head
        const uint8_t* vt_mine = vt + my_head * M::kTileBytes;

        // ---- S^T = K q^T ---------------------------------------------------------------
        float s[RT][4];  // (key lo, row 2qc), (key lo, row 2qc + 1), (key hi, ...)
        uint32_t ks[2];  // scale bytes of this lane's two keys
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (NB == 4)
            ks[i] = *reinterpret_cast<const uint32_t*>(kt_mine + M::kCodeBytes + (my_key + 8 * i) * NB);
          else
            ks[i] = *reinterpret_cast<const uint16_t*>(kt_mine + M::kCodeBytes + (my_key + 8 * i) * NB);
        }
#pragma unroll
        for (int hi = 0; hi < HPI; ++hi) {
          uint32_t kw[2][NB];  // codes of this lane's dims of its two keys
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint8_t* at = kt + hi * M::kTileBytes + (my_key + 8 * i) * M::kRowBytes;
            if constexpr (NB == 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(at + qc * 16);
              kw[i][0] = x.x; kw[i][1] = x.y; kw[i][2] = x.z; kw[i][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(at + qc * 8);
              kw[i][0] = x.x; kw[i][1] = x.y;
            }
          }
          float sh[RT][4];
#pragma unroll
          for (int bp = 0; bp < NB / 2; ++bp) {  // scale blocks 2 bp and 2 bp + 1
            const uint32_t sc2_lo = e8m0x2_to_bf16x2(ks[0], bp), sc2_hi = e8m0x2_to_bf16x2(ks[1], bp);
            // words of dims 4 g .. of both blocks: g = 2 qc in word bp, 2 qc + 1 in NB / 2 + bp
            uint32_t lo[2][4], up[2][4];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              e2m1x8_to_f16x2x4(kw[0][g * (NB / 2) + bp], lo[g]);
              e2m1x8_to_f16x2x4(kw[1][g * (NB / 2) + bp], up[g]);
            }
#pragma unroll
            for (int bb = 0; bb < 2; ++bb) {
              const int b = 2 * bp + bb;
              const float sc_lo = bb ? bf16hi_to_f32(sc2_lo) : bf16lo_to_f32(sc2_lo);
              const float sc_hi = bb ? bf16hi_to_f32(sc2_hi) : bf16lo_to_f32(sc2_hi);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                if (RT > 1 && 8 * rt >= I.rows) break;
                float acc[4];
                const uint4 qf = q_frag[(rt * NB + b) * 32];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                  const uint32_t a[4] = {lo[g][2 * bb], up[g][2 * bb], lo[g][2 * bb + 1],
                                         up[g][2 * bb + 1]};
                  if (g == 0) mma_f16_zero(acc, a, qf.x, qf.y);
                  else mma_f16(acc, a, qf.z, qf.w);
                }
                if (b == 0) {
                  sh[rt][0] = acc[0] * sc_lo; sh[rt][1] = acc[1] * sc_lo;
                  sh[rt][2] = acc[2] * sc_hi; sh[rt][3] = acc[3] * sc_hi;
                } else {
                  sh[rt][0] = fmaf(acc[0], sc_lo, sh[rt][0]);
                  sh[rt][1] = fmaf(acc[1], sc_lo, sh[rt][1]);
                  sh[rt][2] = fmaf(acc[2], sc_hi, sh[rt][2]);
                  sh[rt][3] = fmaf(acc[3], sc_hi, sh[rt][3]);
                }
              }
            }
          }
          // (the scales are those of the lane's own head: of another head's scores nothing is kept)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (hi == 0 || my_head == hi) s[rt][i] = sh[rt][i];
        }

        // ---- V's scales: 2^(e - R_b) of this lane's two keys -----------------------------
        uint32_t vs[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int key = my_key + 8 * i;
          if constexpr (NB == 4)
            vs[i] = *reinterpret_cast<const uint32_t*>(vt_mine + M::kCodeBytes + key * NB);
          else
            vs[i] = *reinterpret_cast<const uint16_t*>(vt_mine + M::kCodeBytes + key * NB);
        }
        uint32_t hidden[RT];  // bit i: element i of s[rt] is of a key that its row does not see
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) hidden[rt] = 0;
        if (diag) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              hidden[rt] |= (key0 + my_key + 8 * (i >> 1) > row_pos[rt][i & 1] ? 1u : 0u) << i;
          // a stale slot's bytes may be anything
          if (key0 + my_key > pos_last) vs[0] = 0u;
          if (key0 + my_key + 8 > pos_last) vs[1] = 0u;
        }
        // the scores of short runs, for the key weights
        if constexpr (kScores) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            if (I.run * p.group > p.score_rows) break;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (8 * rt + 2 * qc + (i & 1) < I.rows)
                my_scores[(8 * rt + (i & 1)) * p.score_stride + key0 + 8 * (i >> 1)] =
                    s[rt][i] * row_scale[rt][i & 1];
          }
        }

        // ---- an item's first block: its first key's scores and scales are the first bases ------
        if (fresh) {
          uint32_t v0;
          if constexpr (NB == 4) v0 = *reinterpret_cast<const uint32_t*>(vt_mine + M::kCodeBytes);
          else v0 = *reinterpret_cast<const uint16_t*>(vt_mine + M::kCodeBytes);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t e = (v0 >> (8 * b)) & 255u;  // (NaN: no reference yet)
            vinv[b] = __uint_as_float((254u - (e == 255u ? 0u : min(e, 253u))) << 23);
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float first = __shfl_sync(0xffffffffu, s[rt][j] * row_scale[rt][j], qc);
              if (key0 <= row_pos[rt][j] && first > -FLT_MAX && first < FLT_MAX) m_run[rt][j] = first;
            }
        }

        // ---- softmax: P and V's factors against the bases there are; where one of them has to
        // move (rarely), it moves and they are computed again ------------------------------------
        float fv[2][NB], pr[RT][4];
#pragma unroll 1
        for (bool again = true;; again = false) {
#pragma unroll
          for (int b = 0; b < NB; b += 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t f = e8m0x2_to_bf16x2(vs[i], b / 2);
              fv[i][b] = bf16lo_to_f32(f) * vinv[b];
              fv[i][b + 1] = bf16hi_to_f32(f) * vinv[b + 1];
            }
          }
          float fmax = 0.f, pmax = 0.f;
#pragma unroll
          for (int b = 0; b < NB; ++b) fmax = fmax3_nan(fmax, fv[0][b], fv[1][b]);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            if (RT > 1 && 8 * rt >= I.rows) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              pr[rt][i] = fmaf(s[rt][i], row_scale[rt][i & 1], -m_run[rt][i & 1]);
              if (diag && ((hidden[rt] >> i) & 1)) pr[rt][i] = -CUDART_INF_F;
              pr[rt][i] = fast_exp2(pr[rt][i]);
            }
            pmax = fmax3(fmax3(pr[rt][0], pr[rt][1], pr[rt][2]), pr[rt][3], pmax);
          }
          if (!__any_sync(0xffffffffu, again && (!(fmax <= 128.f) || pmax > 256.f))) break;
          // (O is rescaled only if something is in it)
          if (__any_sync(0xffffffffu, pmax > 256.f)) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              if (RT > 1 && 8 * rt >= I.rows) break;
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float mx = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (!(diag && ((hidden[rt] >> (2 * i + j)) & 1)))
                    mx = fmaxf(mx, s[rt][2 * i + j] * row_scale[rt][j]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                if (mx > m_run[rt][j] + kLazyRescaleLog2) {
                  const float alpha = fast_exp2(m_run[rt][j] - mx);
                  m_run[rt][j] = mx;
                  l_run[rt][j] *= alpha;
                  if (!fresh) {
#pragma unroll
                    for (int n = 0; n < 2 * NB; ++n) {
                      oacc[rt][n][j] *= alpha;
                      oacc[rt][n][2 + j] *= alpha;
                    }
                  }
                }
              }
            }
          }
          if (__any_sync(0xffffffffu, !(fmax <= 128.f))) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const int e0 = (vs[0] >> (8 * b)) & 255, e1 = (vs[1] >> (8 * b)) & 255;
              // the block's largest scale byte of the lane's head, NaN (255) aside
              const int mine = max(e0 == 255 ? 0 : e0, e1 == 255 ? 0 : e1);
              int top = 0;
#pragma unroll
              for (int hi = 0; hi < HPI; ++hi) {
                const int t = __reduce_max_sync(0xffffffffu, my_head == hi ? mine : 0);
                if (my_head == hi) top = t;
              }
              const int ref = 254 - static_cast<int>(__float_as_uint(vinv[b]) >> 23);
              if (top > ref + 7) {
                // O of the block moves to the new reference (253 at most: what is beyond has no
                // finite value in fp32)
                const int to = min(top, 253);
                vinv[b] = __uint_as_float(static_cast<uint32_t>(254 - to) << 23);
                if (!fresh) {
                  const float down =
                      to - ref > 126
                          ? 0.f
                          : __uint_as_float(static_cast<uint32_t>(127 - (to - ref)) << 23);
#pragma unroll
                  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                      for (int i = 0; i < 4; ++i) oacc[rt][2 * b + t][i] *= down;
                }
              }
              // A NaN block's codes are zeros: with a factor of 2^100, which is finite but makes
              // any weight that counts infinite in f16, their products are NaN for every row that
              // gives the key a weight and 0 for the others.
              const uint32_t big =
                  min(254, 354 - static_cast<int>(__float_as_uint(vinv[b]) >> 23)) << (8 * b);
              if (e0 == 255) vs[0] = (vs[0] & ~(255u << (8 * b))) | big;
              if (e1 == 255) vs[1] = (vs[1] & ~(255u << (8 * b))) | big;
            }
          }
        }
        fresh = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          if (RT > 1 && 8 * rt >= I.rows) break;
#pragma unroll
          for (int j = 0; j < 2; ++j) l_run[rt][j] += pr[rt][j] + pr[rt][2 + j];
        }

        // ---- O^T += V^T P^T ---------------------------------------------------------------
        // half i of P^T with the scales of block b, B operand: row quad
        auto p_half = [&](int rt, int b, int i) {
          return movmatrix_t(pack_f16x2(pr[rt][2 * i] * fv[i][b], pr[rt][2 * i + 1] * fv[i][b]));
        };
        [[maybe_unused]] uint32_t pt[NB][2];  // (several heads: used for each)
        if constexpr (HPI > 1) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            pt[b][0] = p_half(0, b, 0);
            pt[b][1] = p_half(0, b, 1);
          }
        }
#pragma unroll
        for (int hi = 0; hi < HPI; ++hi) {
          uint32_t vw[4][NB / 2];  // codes of dims 4 quad .. of each block, keys of k = 2qc, 2qc + 1,
                                   // 2qc + 8, 2qc + 9
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = ((i & 1) ? 4 + (qc ^ 1) : qc) + 8 * (i >> 1);
            const uint8_t* at = vt + hi * M::kTileBytes + key * M::kRowBytes;
            if constexpr (NB == 4) {
              const uint2 x =
                  *reinterpret_cast<const uint2*>(at + ((quad * 8) ^ ((qc >> 1) << 5)));
              vw[i][0] = x.x; vw[i][1] = x.y;
            } else {
              vw[i][0] = *reinterpret_cast<const uint32_t*>(at + quad * 4);
            }
          }
#pragma unroll
          for (int bp = 0; bp < NB / 2; ++bp) {
            // bytes of (key of even k, key of odd k): even dims in the first word, odd in the
            // second
            uint32_t ev[2][4], od[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t x = vw[2 * i][bp], y = vw[2 * i + 1][bp];
              e2m1x8_to_f16x2x4((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), ev[i]);
              e2m1x8_to_f16x2x4(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), od[i]);
            }
#pragma unroll
            for (int bb = 0; bb < 2; ++bb) {
              const int b = 2 * bp + bb;
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                if (RT > 1 && 8 * rt >= I.rows) break;
                uint32_t b0, b1;
                if constexpr (HPI == 1) {
                  b0 = p_half(rt, b, 0);
                  b1 = p_half(rt, b, 1);
                } else {  // rows of other heads add nothing
                  b0 = quad_head == hi ? pt[b][0] : 0u;
                  b1 = quad_head == hi ? pt[b][1] : 0u;
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                  const uint32_t a[4] = {ev[0][2 * bb + t], od[0][2 * bb + t], ev[1][2 * bb + t],
                                         od[1][2 * bb + t]};
                  mma_f16(oacc[rt][2 * b + t], a, b0, b1);
                }
              }
            }
          }
        }
    };
    // (at least NST - 1 rounds, so that the copies reach the next item's first blocks)
    const int rounds = max(nb_w, NST - 1);
    auto tile_at = [&](int k) {
      return k < nb_w ? own_tiles(buf)[k]
             : k >= rounds && k - rounds < nb_next ? own_tiles(buf ^ 1)[k - rounds] : -1;
    };
    __syncwarp();  // the next item's tiles are there
    int tile = tile_at(NST - 1);
    for (int k = 0; k < rounds; ++k) {
      cp_async_wait<NST - 2>();  // block k's copies have landed
      __syncwarp();              // for every lane; and every lane has read the block before
      issue(tile, st == 0 ? NST - 1 : st - 1);
      there = there << 1 | (tile >= 0 ? 1u : 0u);
      tile = tile_at(k + NST);
      if (there >> (NST - 1) & 1) {
        if ((my_first + k * kDecodeWarps + 1) * kBlockSize - 1 > I.pos_base)
          tile_step(k, st, std::true_type());
        else
          tile_step(k, st, std::false_type());
      }
      st = st + 1 == NST ? 0 : st + 1;
    }

    // ---- per-warp state -> shared memory ------------------------------------------------------
    float* so = scratch + warp * (C::kScratch / 4);  // [R][D]
    float* sm = so + R * D;                      // [R]
    float* sl = sm + R;                          // [R]
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (RT > 1 && 8 * rt >= I.rows) break;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 8 * rt + 2 * qc + j;
        float l = l_run[rt][j];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (quad == 0) {
          sm[row] = m_run[rt][j];
          sl[row] = l;
        }
#pragma unroll
        for (int n = 0; n < 2 * NB; ++n) {
          // 2^(R_b - 127)
          const float up = e8m0_to_f32(254u - (__float_as_uint(vinv[n >> 1]) >> 23));
          *reinterpret_cast<float2*>(so + row * D + 32 * (n >> 1) + 4 * quad + 2 * (n & 1)) =
              make_float2(oacc[rt][n][j] * up, oacc[rt][n][2 + j] * up);
        }
      }
    }
    __syncthreads();

    // ---- merge the 4 warps and write the output or the partial ---------------------------
    for (int e = threadIdx.x; e < I.rows * (D / 4); e += kDecodeWarps * 32) {
      const int r = e / (D / 4), d = 4 * (e % (D / 4));
      float mx = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w)
        mx = fmaxf(mx, scratch[w * (C::kScratch / 4) + R * D + r]);
      float lsum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) {
        const float* wso = scratch + w * (C::kScratch / 4);
        const float f = fast_exp2(wso[R * D + r] - mx);  // (1 where no warp has a base: zeros or NaN)
        lsum += wso[R * D + R + r] * f;
        const float4 x = *reinterpret_cast<const float4*>(wso + r * D + d);
        o[0] += x.x * f;
        o[1] += x.y * f;
        o[2] += x.z * f;
        o[3] += x.w * f;
      }
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = lsum == 0.f ? 0.f : o[i] * inv;
      const int t = r / (p.group * HPI);
      const int64_t orow = static_cast<int64_t>(I.t0 + t) * p.num_q_heads + I.h * p.group +
                           (r - t * (p.group * HPI));
      const float lse = lsum == 0.f ? -CUDART_INF_F : mx + __log2f(lsum);
      if (I.nparts == 1) {
        if (p.out_bf16)
          *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow * D + d) =
              make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
        else
          *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + orow * D + d) =
              make_float4(o[0], o[1], o[2], o[3]);
        if (p.lse && d == 0) p.lse[orow] = lse;
      } else {
        const int64_t prow = orow * p.pmax + I.part;
        *reinterpret_cast<float4*>(p.part_o + prow * D + d) = make_float4(o[0], o[1], o[2], o[3]);
        if (d == 0) p.part_lse[prow] = lse;
      }
    }
    slot = next_slot;
    buf ^= 1;
    nb_w = nb_next;
  }
  if (p.span && threadIdx.x == 0)
    atomicMax(reinterpret_cast<unsigned long long*>(p.span) + 1,
              static_cast<unsigned long long>(global_ns()));
  if (p.wait_at_end) grid_dependency_wait();
}

template <int D, int RT, int HPI, bool kScores = false>
static cudaError_t run_mx(const AttnArgs& a, int pmax, const DecodeParams& p) {
  if constexpr (!kScores) {
    if (p.scores) return run_mx<D, RT, HPI, true>(a, pmax, p);
  }
  auto kern = decode_mx_kernel<D, RT, HPI, kScores>;
  constexpr int smem = MxCfg<D, RT, HPI>::kSmem;
  LaunchInfo li;
  cudaError_t e = launch_info(kern, kDecodeWarps * 32, smem, &li);
  if (e != cudaSuccess) return e;
  const int tpt = 8 * RT / (p.group * HPI);
  const int64_t upper = static_cast<int64_t>(a.num_seqs) * (a.num_kv_heads / HPI) *
                        ((a.max_query_len + tpt - 1) / tpt) * pmax;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(upper, int64_t(li.sms) * li.per_sm));
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(kDecodeWarps * 32), smem,
                          a.stream, static_cast<const uint8_t*>(a.k_cache),
                          static_cast<const uint8_t*>(a.v_cache), p);
}

// Row tiles of an item.  (Tiles of 32 rows spilled at 255 registers and two CTAs per SM: 64 runs of
// 8 tokens x 4 heads over 4,000 keys, 8 kv heads, took 696 us, two 16-row tiles each 315.)
int mx_row_tiles(int32_t max_query_len, int32_t group) {
  const int64_t rows = static_cast<int64_t>(max_query_len) * group;
  return rows <= 8 ? 1 : 2;
}

// Two kv heads per item where their rows fill an 8-row tile that one head's would leave half
// empty: what a block costs beside its codes (softmax, scales, the copies' and items' bookkeeping)
// is then paid once for two.  256 decodes of 1,000 tokens on average, 32 q heads on 8: 121 -> 104
// us.
//
// With the bound on the contexts, few items may come to a CTA, and their last round then leaves
// CTAs idle: in steps of fewer than four rounds the partitions are cut so that the rounds come out
// even (a partition has ws.pblk blocks at least, for which the partials have room), and where even
// that leaves more than a fifth idle, items stay those of single heads.  16 x 32,768 tokens, 8 kv
// heads: 1,024 items of 128 blocks on 456 CTAs 143 us, 896 of 147 blocks 112 us; single heads 137.
int mx_heads_per_item(const AttnArgs& a, const DecodeParams& p, int min_pblk, int* pblk) {
  if ((p.group != 2 && p.group != 4) || a.num_kv_heads % 2) return 1;
  // (of a staged step the runs that are left are short)
  if (a.stage.capacity == 0 && static_cast<int64_t>(a.max_query_len) * p.group * 2 > 8) return 1;
  using C = MxCfg<128, 1, 2>;
  const int64_t ctas = int64_t{C::kCtas} * p.sms;
  const int64_t maxblk = (int64_t{a.max_context_len} + kBlockSize - 1) / kBlockSize;
  auto rounds = [&](int64_t parts) {
    return (static_cast<int64_t>(a.num_seqs) * (a.num_kv_heads / 2) * parts + ctas - 1) / ctas;
  };
  const int64_t parts = (maxblk + p.pblk - 1) / p.pblk;
  if (rounds(parts) >= 4) return 2;
  // blocks a CTA reads one after the other, and 4 for an item's own cost
  int64_t best = INT64_MAX;
  for (int64_t n = (maxblk + min_pblk - 1) / min_pblk; n > 0; --n) {
    const int64_t blocks = std::max<int64_t>((maxblk + n - 1) / n, min_pblk);
    if (blocks > kDecodeWarps * C::kOwn) break;
    if (rounds(n) * (blocks + 4) < best) {
      best = rounds(n) * (blocks + 4);
      *pblk = static_cast<int>(blocks);
    }
  }
  const int64_t work = static_cast<int64_t>(a.num_seqs) * (a.num_kv_heads / 2) * maxblk;
  return work * 5 >= best * ctas * 4 ? 2 : 1;
}

cudaError_t launch_decode_mx(const AttnArgs& a, int pmax, const DecodeParams& p) {
  const int rt = p.rows_per_tile / 8;
  if (a.head_dim == 128) {
    if (p.heads_per_item == 2) return run_mx<128, 1, 2>(a, pmax, p);
    return rt == 1 ? run_mx<128, 1, 1>(a, pmax, p) : run_mx<128, 2, 1>(a, pmax, p);
  }
  if (p.heads_per_item == 2) return run_mx<64, 1, 2>(a, pmax, p);
  return rt == 1 ? run_mx<64, 1, 1>(a, pmax, p) : run_mx<64, 2, 1>(a, pmax, p);
}

}  // namespace pa
