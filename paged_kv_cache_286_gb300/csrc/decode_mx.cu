// Paged attention over MXFP4 pools: decode tokens, short query runs and prompt chunks.
//
// What it computes: softmax(scale * q . k_j) v_j over keys j <= p_i, where element d of key j is
// code[j][d] * 2^(e[j][d / 32] - 127) and the same for values (mxfp4.cuh has the tile).
//
//  * Work items, plan and merge are those of the split-KV kernel (decode.cu): an item is
//    (sequence, kv head, tile of 8 RT rows = tokens x heads of the group, KV partition), each of
//    the CTA's 4 warps takes every 4th block of the partition through its own ring of shared
//    memory stages.  A (block, head) tile is contiguous, so one untiled bulk copy each brings the
//    K and the V tile.
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
//  * The softmax base of a row moves only when a score exceeds it by more than 2^8, so that the
//    usual block needs one warp vote and no maximum across lanes.
#include <math_constants.h>

#include <algorithm>

#include "decode_items.cuh"
#include "mxfp4.cuh"
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

template <int D, int RT>
struct MxCfg {
  static constexpr int kStages = RT == 1 ? 6 : 8;
  static constexpr int kStageBytes = 2 * Mx<D>::kTileBytes;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kScratch = 8 * RT * D * 4 + 2 * 8 * RT * 4;  // O, max and sum of a warp
  static constexpr int kSmem =
      kDecodeWarps * kWarpBytes + kDecodeWarps * kStages * 8 + 2 * 64 + 128 /*alignment*/;
  static constexpr int kCtas = RT == 1 ? 4 : RT == 2 ? 3 : 2;  // CTAs per SM
  static_assert(kScratch <= kWarpBytes, "merge scratch must fit in a warp's stages");
  static_assert(kStageBytes % 16 == 0 && sizeof(ItemInfo) <= 64, "");
};

// kScores: the scores of runs of up to kDecodeMaxRows rows are also written out, for the key
// weights (key_weights.cu).
template <int D, int RT, bool kScores>
__global__ void __launch_bounds__(kDecodeWarps * 32, MxCfg<D, RT>::kCtas)
    decode_mx_kernel(const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool,
                     const DecodeParams p) {
  using C = MxCfg<D, RT>;
  using M = Mx<D>;
  constexpr int NB = M::kBlocks;
  constexpr int NST = C::kStages;
  constexpr int R = 8 * RT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kDecodeWarps * C::kWarpBytes);
  ItemInfo* s_item = reinterpret_cast<ItemInfo*>(bars + kDecodeWarps * NST);

  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int quad = lane >> 2;
  const int qc = lane & 3;
  uint8_t* wbuf = smem + warp * C::kWarpBytes;
  uint64_t* wbars = bars + warp * NST;
  // Key of the block that row `quad` of the MMA's upper half stands for (quad + 8: that key + 8).
  // P^T's k indices 2 qc, 2 qc + 1 then are keys qc and 4 + (qc ^ 1): the 64-byte rows that the
  // lanes of one shared memory access touch have both parities for K's 16-byte and for V's
  // 8-byte loads (natural order: V's conflict four ways).
  const int my_key = (quad & 1) ? 4 + ((quad >> 1) ^ 1) : quad >> 1;

  if (lane == 0) {
    for (int st = 0; st < NST; ++st) mbar_init(&wbars[st], 1);
    fence_barrier_init();
  }
  __syncthreads();
  grid_dependency_wait();
  if (p.span && threadIdx.x == 0)
    atomicMin(reinterpret_cast<unsigned long long*>(p.span),
              static_cast<unsigned long long>(global_ns()));
  const int total_items = p.item_start[p.num_seqs];
  uint32_t it = 0;
  bool timed_out = false;
  auto fetch_item = [&](ItemInfo* dst) { *dst = claim_item<R, 1>(p, total_items); };
  if (threadIdx.x == 0) fetch_item(&s_item[0]);
  int cur = 0;

  while (true) {
    const bool any_timeout = __syncthreads_or(timed_out) != 0;
    const ItemInfo I = s_item[cur];
    if (!I.valid || any_timeout) break;
    const uint32_t it0 = it;
    const int pos_last = I.pos_base + I.n - 1;

    // ---- table entries of this warp's blocks, one per lane -----------------------------
    const int my_first = I.blk_begin + warp;
    const int nb_w = my_first < I.blk_end ? ceil_div(I.blk_end - my_first, kDecodeWarps) : 0;
    int phys_lane = -1;
    if (lane < nb_w) {
      const int b = my_first + lane * kDecodeWarps;
      phys_lane = __ldg(p.block_tables + static_cast<int64_t>(I.s) * p.max_blocks_per_seq + b);
      if (phys_lane < 0 || phys_lane >= p.num_blocks) {
        set_error(&p.hdr->error, PA_DEVERR_BLOCK_ID);
        phys_lane = -1;
      }
    }
    auto issue = [&](int k) {  // stage load for the warp's k-th block (all lanes call)
      const int phys = __shfl_sync(0xffffffffu, phys_lane, k);
      if (lane == 0) {
        const uint32_t st = (it0 + k) % NST;
        uint64_t* bar = &wbars[st];
        if (phys >= 0) {
          uint8_t* kt = wbuf + st * C::kStageBytes;
          const int64_t tile = static_cast<int64_t>(phys) * p.num_kv_heads + I.h;
          mbar_arrive_expect_tx(bar, C::kStageBytes);
          // test hook: the first stage of the first item claimed expects its bytes but gets no
          // copy, so that the bounded wait on it expires
          if (!(p.skip_copy && I.idx == 0 && warp == 0 && k == 0)) {
            bulk_load(kt, k_pool + tile * M::kTileBytes, M::kTileBytes, bar);
            bulk_load(kt + M::kTileBytes, v_pool + tile * M::kTileBytes, M::kTileBytes, bar);
          }
        } else {
          mbar_arrive(bar);
        }
      }
    };
    const int npre = min(NST, nb_w);
    for (int k = 0; k < npre; ++k) issue(k);
    if (threadIdx.x == 0) fetch_item(&s_item[cur ^ 1]);  // read after the next loop-top barrier

    // ---- q fragments (B operand, n = row quad of the tile): of scale block b, the pairs of
    // dims 32 b + 8 qc + {0 1, 2 3} (first MMA) and {4 5, 6 7} (second) ---------------------
    uint32_t qf[RT][NB][4];
    float row_scale[RT][2];  // of rows 2 qc, 2 qc + 1 of each tile
    int row_pos[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = 8 * rt + quad;
      const bool ok = row < I.rows;
      const int tok = ok ? row / p.group : 0, g = ok ? row - tok * p.group : 0;
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
      int ex = 0;  // power of two e with amax * 2^e < 2^15 (f16 range), exact scaling
      if (amax > 0.f && amax < CUDART_INF_F) frexpf(amax, &ex);
      const int e = max(-100, min(100, 15 - ex));
      const float up = ldexpf(1.f, e);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          qf[rt][b][i] = pack_f16x2(bf16lo_to_f32(w[i]) * up, bf16hi_to_f32(w[i]) * up);
      }
      const float rs = p.score_log2 * ldexpf(1.f, -e);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        row_scale[rt][j] = __shfl_sync(0xffffffffu, rs, 4 * (2 * qc + j));
        row_pos[rt][j] = I.pos_base + (8 * rt + 2 * qc + j) / p.group;
      }
    }

    float m_run[RT][2], l_run[RT][2];  // base (log2 domain) and this lane's share of the sum
    float oacc[RT][2 * NB][4];         // [row tile][2 b + t]: dims 32 b + 4 quad + 2 t + {0, 1}
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m_run[rt][0] = m_run[rt][1] = -CUDART_INF_F;
      l_run[rt][0] = l_run[rt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j)
        oacc[rt][j][0] = oacc[rt][j][1] = oacc[rt][j][2] = oacc[rt][j][3] = 0.f;
    }
    int vref[NB];  // R_b as a scale byte; 0: none yet (the first block with larger ones sets it)
#pragma unroll
    for (int b = 0; b < NB; ++b) vref[b] = 0;

    for (int k = 0; k < nb_w; ++k) {
      const uint32_t st = it % NST;
      if (!__all_sync(0xffffffffu, mbar_wait(&wbars[st], (it / NST) & 1u, p.wait_ns))) {
        if (lane == 0) set_error(&p.hdr->error, PA_DEVERR_TIMEOUT);
        timed_out = true;
        for (int k2 = k + 1; k2 < min(nb_w, k + NST); ++k2)
          mbar_wait(&wbars[(it + (k2 - k)) % NST], ((it + (k2 - k)) / NST) & 1u, p.wait_ns);
        break;
      }
      const int phys = __shfl_sync(0xffffffffu, phys_lane, k);
      if (phys >= 0) {
        const int key0 = (my_first + k * kDecodeWarps) * kBlockSize;
        const uint8_t* kt = wbuf + st * C::kStageBytes;
        const uint8_t* vt = kt + M::kTileBytes;
        const bool diag = key0 + kBlockSize - 1 > I.pos_base;  // some row may not see some key

        // ---- S^T = K q^T ---------------------------------------------------------------
        float s[RT][4];  // (key lo, row 2qc), (key lo, row 2qc + 1), (key hi, ...)
        {
          uint32_t kw[2][NB];  // codes of this lane's dims of its two keys
          uint32_t ks[2];      // their scale bytes
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = my_key + 8 * i;
            if constexpr (NB == 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(kt + key * M::kRowBytes + qc * 16);
              kw[i][0] = x.x; kw[i][1] = x.y; kw[i][2] = x.z; kw[i][3] = x.w;
              ks[i] = *reinterpret_cast<const uint32_t*>(kt + M::kCodeBytes + key * NB);
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(kt + key * M::kRowBytes + qc * 8);
              kw[i][0] = x.x; kw[i][1] = x.y;
              ks[i] = *reinterpret_cast<const uint16_t*>(kt + M::kCodeBytes + key * NB);
            }
          }
#pragma unroll
          for (int bp = 0; bp < NB / 2; ++bp) {  // scale blocks 2 bp and 2 bp + 1
            // words of dims 4 g .. of both blocks: g = 2 qc in word bp, 2 qc + 1 in NB / 2 + bp
            uint32_t lo[2][4], hi[2][4];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              e2m1x8_to_f16x2x4(kw[0][g * (NB / 2) + bp], lo[g]);
              e2m1x8_to_f16x2x4(kw[1][g * (NB / 2) + bp], hi[g]);
            }
#pragma unroll
            for (int bb = 0; bb < 2; ++bb) {
              const int b = 2 * bp + bb;
              const float sc_lo = e8m0_to_f32(ks[0], b), sc_hi = e8m0_to_f32(ks[1], b);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                if (RT > 1 && 8 * rt >= I.rows) break;
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                  const uint32_t a[4] = {lo[g][2 * bb], hi[g][2 * bb], lo[g][2 * bb + 1],
                                         hi[g][2 * bb + 1]};
                  mma_f16(acc, a, qf[rt][b][2 * g], qf[rt][b][2 * g + 1]);
                }
                if (b == 0) {
                  s[rt][0] = acc[0] * sc_lo; s[rt][1] = acc[1] * sc_lo;
                  s[rt][2] = acc[2] * sc_hi; s[rt][3] = acc[3] * sc_hi;
                } else {
                  s[rt][0] = fmaf(acc[0], sc_lo, s[rt][0]); s[rt][1] = fmaf(acc[1], sc_lo, s[rt][1]);
                  s[rt][2] = fmaf(acc[2], sc_hi, s[rt][2]); s[rt][3] = fmaf(acc[3], sc_hi, s[rt][3]);
                }
              }
            }
          }
        }

        // ---- softmax: P over S ------------------------------------------------------------
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          if (RT > 1 && 8 * rt >= I.rows) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[rt][i] *= row_scale[rt][i & 1];
            if (diag && key0 + my_key + 8 * (i >> 1) > row_pos[rt][i & 1]) s[rt][i] = -CUDART_INF_F;
          }
          if constexpr (kScores) {
            if (I.run * p.group <= p.score_rows) {  // one tile then: its rows are the run's
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int row = 8 * rt + 2 * qc + (i & 1);
                if (row < I.rows)
                  p.scores[((static_cast<int64_t>(I.s) * p.num_kv_heads + I.h) * p.score_rows + row) *
                               p.score_stride + key0 + my_key + 8 * (i >> 1)] = s[rt][i];
              }
            }
          }
          const bool over = s[rt][0] > m_run[rt][0] + kLazyRescaleLog2 ||
                            s[rt][2] > m_run[rt][0] + kLazyRescaleLog2 ||
                            s[rt][1] > m_run[rt][1] + kLazyRescaleLog2 ||
                            s[rt][3] > m_run[rt][1] + kLazyRescaleLog2;
          if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float mx = fmaxf(s[rt][j], s[rt][2 + j]);
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              if (mx > m_run[rt][j] + kLazyRescaleLog2) {
                const float alpha =
                    m_run[rt][j] == -CUDART_INF_F ? 0.f : fast_exp2(m_run[rt][j] - mx);
                m_run[rt][j] = mx;
                l_run[rt][j] *= alpha;
#pragma unroll
                for (int n = 0; n < 2 * NB; ++n) {
                  oacc[rt][n][j] *= alpha;
                  oacc[rt][n][2 + j] *= alpha;
                }
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float m_use = m_run[rt][j] == -CUDART_INF_F ? 0.f : m_run[rt][j];
            s[rt][j] = fast_exp2(s[rt][j] - m_use);
            s[rt][2 + j] = fast_exp2(s[rt][2 + j] - m_use);
            l_run[rt][j] += s[rt][j] + s[rt][2 + j];
          }
        }

        // ---- V's scales: 2^(e - R_b) of this lane's two keys -----------------------------
        uint32_t vs[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int key = my_key + 8 * i;
          if constexpr (NB == 4)
            vs[i] = *reinterpret_cast<const uint32_t*>(vt + M::kCodeBytes + key * NB);
          else
            vs[i] = *reinterpret_cast<const uint16_t*>(vt + M::kCodeBytes + key * NB);
          if (key0 + key > pos_last) vs[i] = 0u;  // a stale slot's bytes may be anything
        }
        float fv[2][NB];
        float fmax = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float inv = __uint_as_float(static_cast<uint32_t>(254 - vref[b]) << 23);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            fv[i][b] = e8m0_to_f32(vs[i], b) * inv;
            fmax = fmaxf(fmax, fv[i][b]);
          }
        }
        if (__any_sync(0xffffffffu, fmax > 128.f)) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const int lo = (vs[0] >> (8 * b)) & 255, hi = (vs[1] >> (8 * b)) & 255;
            // (255 is NaN whatever the reference)
            int top = max(lo == 255 ? 0 : lo, hi == 255 ? 0 : hi);
            top = __reduce_max_sync(0xffffffffu, top);
            if (top > vref[b] + 7) {
              // O of the block moves to the new reference (253 at most: what is beyond has no
              // finite value in fp32)
              const int to = min(top, 253);
              const float down =
                  to - vref[b] > 126 ? 0.f
                                     : __uint_as_float(static_cast<uint32_t>(127 - (to - vref[b])) << 23);
              vref[b] = to;
#pragma unroll
              for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                  for (int i = 0; i < 4; ++i) oacc[rt][2 * b + t][i] *= down;
            }
            const float inv = __uint_as_float(static_cast<uint32_t>(254 - vref[b]) << 23);
            fv[0][b] = e8m0_to_f32(vs[0], b) * inv;
            fv[1][b] = e8m0_to_f32(vs[1], b) * inv;
          }
        }

        // ---- O^T += V^T P^T ---------------------------------------------------------------
        uint32_t vw[4][NB / 2];  // codes of dims 4 quad .. of each block, keys of k = 2qc, 2qc + 1,
                                 // 2qc + 8, 2qc + 9
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = ((i & 1) ? 4 + (qc ^ 1) : qc) + 8 * (i >> 1);
          if constexpr (NB == 4) {
            const uint2 x = *reinterpret_cast<const uint2*>(vt + key * M::kRowBytes + quad * 8);
            vw[i][0] = x.x; vw[i][1] = x.y;
          } else {
            vw[i][0] = *reinterpret_cast<const uint32_t*>(vt + key * M::kRowBytes + quad * 4);
          }
        }
#pragma unroll
        for (int bp = 0; bp < NB / 2; ++bp) {
          // bytes of (key of even k, key of odd k): even dims in the first word, odd in the second
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
              float pv[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                pv[i] = s[rt][i] * fv[i >> 1][b];
                // a key that the row does not see adds nothing, whatever its scale
                if (diag && s[rt][i] == 0.f) pv[i] = 0.f;
              }
              const uint32_t b0 = movmatrix_t(pack_f16x2(pv[0], pv[1]));
              const uint32_t b1 = movmatrix_t(pack_f16x2(pv[2], pv[3]));
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
      __syncwarp();
      ++it;
      if (k + NST < nb_w) issue(k + NST);
    }
    if (timed_out) it = 0;  // results are void; phase tracking no longer matters

    // ---- per-warp state -> shared memory (this warp's own stages) --------------------------
    __syncwarp();
    float* so = reinterpret_cast<float*>(wbuf);  // [R][D]
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
          const float up = __uint_as_float(static_cast<uint32_t>(vref[n >> 1]) << 23);
          *reinterpret_cast<float2*>(so + row * D + 32 * (n >> 1) + 4 * quad + 2 * (n & 1)) =
              make_float2(oacc[rt][n][j] * up, oacc[rt][n][2 + j] * up);
        }
      }
    }
    __syncthreads();

    // ---- merge the 4 warps and write the output or the partial ---------------------------
    for (int e = threadIdx.x; e < I.rows * D; e += kDecodeWarps * 32) {
      const int r = e / D, d = e - r * D;
      float mx = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w)
        mx = fmaxf(mx, reinterpret_cast<const float*>(smem + w * C::kWarpBytes)[R * D + r]);
      float lsum = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) {
        const float* wso = reinterpret_cast<const float*>(smem + w * C::kWarpBytes);
        const float mw = wso[R * D + r];
        // without a base (no key seen: zeros, or only NaN scores) the sums count as they are
        const float f = mw == -CUDART_INF_F ? 1.f : fast_exp2(mw - mx);
        lsum += wso[R * D + R + r] * f;
        o += wso[r * D + d] * f;
      }
      const float val = lsum == 0.f ? 0.f : o / lsum;
      const int t = I.t0 + r / p.group;
      const int64_t orow = static_cast<int64_t>(t) * p.num_q_heads + I.h * p.group + r % p.group;
      const float lse = lsum == 0.f ? -CUDART_INF_F : mx + __log2f(lsum);
      if (I.nparts == 1) {
        if (p.out_bf16)
          reinterpret_cast<__nv_bfloat16*>(p.out)[orow * D + d] = __float2bfloat16_rn(val);
        else
          reinterpret_cast<float*>(p.out)[orow * D + d] = val;
        if (p.lse && d == 0) p.lse[orow] = lse;
      } else {
        const int64_t prow = orow * p.pmax + I.part;
        p.part_o[prow * D + d] = val;
        if (d == 0) p.part_lse[prow] = lse;
      }
    }
    __syncthreads();
    fence_proxy_async_smem();  // generic accesses to the stages before the next copies
    cur ^= 1;
  }
  if (p.span && threadIdx.x == 0)
    atomicMax(reinterpret_cast<unsigned long long*>(p.span) + 1,
              static_cast<unsigned long long>(global_ns()));
}

template <int D, int RT, bool kScores = false>
static cudaError_t run_mx(const AttnArgs& a, int pmax, const DecodeParams& p) {
  if constexpr (!kScores) {
    if (p.scores) return run_mx<D, RT, true>(a, pmax, p);
  }
  auto kern = decode_mx_kernel<D, RT, kScores>;
  constexpr int smem = MxCfg<D, RT>::kSmem;
  LaunchInfo li;
  cudaError_t e = launch_info(kern, kDecodeWarps * 32, smem, &li);
  if (e != cudaSuccess) return e;
  const int tpt = 8 * RT / p.group;
  const int64_t upper = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads *
                        ((a.max_query_len + tpt - 1) / tpt) * pmax;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(upper, int64_t(li.sms) * li.per_sm));
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(kDecodeWarps * 32), smem,
                          a.stream, static_cast<const uint8_t*>(a.k_cache),
                          static_cast<const uint8_t*>(a.v_cache), p);
}

// Row tiles of an item: enough for the longest run, at most 32 rows.
int mx_row_tiles(int32_t max_query_len, int32_t group) {
  const int64_t rows = static_cast<int64_t>(max_query_len) * group;
  return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}

cudaError_t launch_decode_mx(const AttnArgs& a, int pmax, const DecodeParams& p) {
  const int rt = p.rows_per_tile / 8;
  if (a.head_dim == 128)
    return rt == 1 ? run_mx<128, 1>(a, pmax, p)
                   : rt == 2 ? run_mx<128, 2>(a, pmax, p) : run_mx<128, 4>(a, pmax, p);
  return rt == 1 ? run_mx<64, 1>(a, pmax, p)
                 : rt == 2 ? run_mx<64, 2>(a, pmax, p) : run_mx<64, 4>(a, pmax, p);
}

}  // namespace pa
