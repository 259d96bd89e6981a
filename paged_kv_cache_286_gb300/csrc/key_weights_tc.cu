// Accumulated key weights of long query runs on the tensor cores (tcgen05).
//
// W[j] <- decay * W[j] + sum over the rows (query token, q head of the group) that see key j of
// 2^(s_j - lse_row), as in key_weights.cu, for runs whose scores the attention did not keep.
//
//  * The scores of 128 keys and 128 rows are one accumulator of S^T = K Q^T: the keys are M, so that
//    a key is a TMEM lane and its sum over rows stays in the two threads that read that lane (one
//    per half of the columns) from the first row to the last.  No maximum, no exchange per tile, and
//    no atomics: the two halves meet once per item, in a fixed order.
//  * A CTA holds an item's keys (256 of one kv head, 64 KiB, two accumulators) while the rows pass:
//    128 / G tokens x G heads a tile, one 3-D TMA box per 64 columns, four tiles in flight, two pairs
//    of accumulators.  Warp 0 copies, warp 1 issues the MMAs, warps 2-17 read the accumulators.
//  * E4M3 and MXFP4 keys become bf16 (exact: four significant bits and two) on their way in, by the
//    warps 2-17, once per item; copied K tiles cost less, but a conversion beforehand would write
//    and read four or eight times the bytes.
//  * A score costs the epilogue an FMA, a 2^x and an add: the 2^x (32 a cycle and SM) take 0.5 us of a
//    tile of 256 x 128, the MMAs 0.7.  A tile takes 1.8: latency bounds it, as a warp reads 32 columns
//    of an accumulator, waits, and works on them with no read of its own in flight.  Two runs of 2,048
//    tokens x 32 heads after 6,144 (8 kv heads of 128): 338 us for bf16 keys, 712 TFLOP/s, 341 us for
//    E4M3 and 344 us for MXFP4, where the mma.sync kernel took 1,280; one run of 512 x 32 in 2,560 keys
//    beside one of 512 x 32 in 512 31 us.
//  * Every wait is bounded; when one runs out the CTA records PA_DEVERR_TIMEOUT, stops, lets its
//    copies and MMAs finish (bounded again) and frees its tensor memory.
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pool_keys.cuh"

namespace pa {

namespace {

constexpr int kTcKeys = kKeyWeightsTcKeys;  // keys of an item: two accumulators' rows
static_assert(kTcKeys == 256, "two accumulators of 128 lanes");
constexpr int kTcEpilogue = 16;             // warps 2 .. 17: eight for each 128 keys
constexpr int kTcThreads = 32 * (2 + kTcEpilogue);
constexpr int kTcQStages = 4, kTcKStages = 1, kTcBufs = 2;
constexpr uint32_t kTcCols = 512;           // tensor memory: two pairs of accumulators of 128 columns

template <int D>
struct TcLayout {
  static constexpr int kTile = 128 * D * 2;  // 128 keys or rows
  static constexpr int kK = 0;
  static constexpr int kQ = kTcKStages * 2 * kTile;
  static constexpr int kSmem = 1024 + kQ + kTcQStages * kTile;
};

struct TcCtl {
  uint64_t k_full[kTcKStages], k_empty[kTcKStages], q_full[kTcQStages], q_empty[kTcQStages],
      d_full[kTcBufs], d_empty[kTcBufs], sum_full, sum_free, drain;
  uint32_t tmem_base;
  int abort_flag;
};

// The item's part of its run, the same for every role.
struct TcItem {
  int s, h, t0, n, L, base;  // base: first key
  int first_tok, tiles;
};

__device__ __forceinline__ TcItem tc_item(const KeyWeightsArgs& a, int64_t item, int tpt) {
  TcItem it;
  const int chunk_id = static_cast<int>(item / a.num_kv_heads);
  it.h = static_cast<int>(item - static_cast<int64_t>(chunk_id) * a.num_kv_heads);
  int lo = 0, hi = a.num_seqs;  // largest s with chunk_start[s] <= chunk_id
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.chunk_start[mid] <= chunk_id) lo = mid; else hi = mid;
  }
  it.s = lo;
  it.t0 = a.qsl[lo];
  it.n = a.qsl[lo + 1] - it.t0;
  it.L = a.context_lens[lo];
  it.base = (chunk_id - a.chunk_start[lo]) * kTcKeys;
  it.first_tok = max(0, it.base - (it.L - it.n));  // the first that sees some key of the item
  it.tiles = (it.n - it.first_tok + tpt - 1) / tpt;
  return it;
}

template <Pool kPool, int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    key_weights_tc_kernel(const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ CUtensorMap kmap, const KeyWeightsArgs a) {
  using L = TcLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ TcCtl ctl;
  __shared__ __align__(16) float s_lse[kTcEpilogue][64];  // negated, of each warp's columns
  __shared__ float s_part[2][kTcKeys];  // sums by half of the columns
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kTcKStages; ++i) {
      mbar_init(&ctl.k_full[i], kPool == Pool::kBf16 ? 1 : kTcEpilogue);
      mbar_init(&ctl.k_empty[i], 1);
    }
    for (int i = 0; i < kTcQStages; ++i) {
      mbar_init(&ctl.q_full[i], 1);
      mbar_init(&ctl.q_empty[i], 1);
    }
    for (int i = 0; i < kTcBufs; ++i) {
      mbar_init(&ctl.d_full[i], 1);
      mbar_init(&ctl.d_empty[i], kTcEpilogue);
    }
    mbar_init(&ctl.sum_full, kTcEpilogue);
    mbar_init(&ctl.sum_free, kTcEpilogue);
    mbar_init(&ctl.drain, 1);
    ctl.abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&qmap);
    if (kPool == Pool::kBf16) prefetch_tensormap(&kmap);
  }
  if (warp == 1) tmem_alloc(&ctl.tmem_base, kTcCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  grid_dependency_wait();
  grid_launch_dependents();  // the finishing kernel, which has other sequences, may start beside
  const int G = a.num_q_heads / a.num_kv_heads, tpt = 128 / G;
  const int64_t total = static_cast<int64_t>(a.chunk_start[a.num_seqs]) * a.num_kv_heads;

  // all lanes wait; the outcome is warp-uniform
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, a.wait_ns));
    if (!ok && lane == 0) {
      set_error(a.err, PA_DEVERR_TIMEOUT);
      ctl.abort_flag = 1;
    }
    return ok && !__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&ctl.abort_flag));
  };

  uint32_t kc = 0, qc = 0;  // items and tiles so far (rings and phases)
  bool ok = true;
  if (warp == 0) {
    // ---------------------------------------------------------------- producer (TMA)
    for (int64_t item = blockIdx.x; ok && item < total; item += gridDim.x, ++kc) {
      const TcItem I = tc_item(a, item, tpt);
      if constexpr (kPool == Pool::kBf16) {
        const uint32_t ks = kc % kTcKStages;
        const int jb = I.base / kBlockSize + lane;  // this lane's block of the keys
        int phys = -1;
        if (lane < kTcKeys / kBlockSize && jb * kBlockSize < I.L) {
          phys = __ldg(a.block_tables + static_cast<int64_t>(I.s) * a.max_blocks_per_seq + jb);
          if (phys >= a.num_blocks) phys = -1;  // (flagged by the attention)
        }
        if (!(ok = wait(&ctl.k_empty[ks], ((kc / kTcKStages) & 1u) ^ 1u))) break;
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, phys >= 0)) * (kBlockSize * D * 2);
        if (lane == 0) {
          if (bytes) mbar_arrive_expect_tx(&ctl.k_full[ks], bytes);
          else mbar_arrive(&ctl.k_full[ks]);
        }
        __syncwarp();
        // test hook: the first item's first copy is left out while its bytes are expected
        if (phys >= 0 && !(a.skip_copy && item == 0 && lane == 0)) {
          uint8_t* dst = smem + L::kK + ks * 2 * L::kTile + lane * (kBlockSize * D * 2);
          const int group = (phys * a.num_kv_heads + I.h) * 2;  // its first group of 8 pool rows
          if constexpr (D == 128) tma_load_4d(dst, &kmap, 0, 0, 0, group, &ctl.k_full[ks]);
          else tma_load_2d(dst, &kmap, 0, group * 8, &ctl.k_full[ks]);
        }
      }
      for (int t = 0; t < I.tiles; ++t, ++qc) {
        const uint32_t qs = qc % kTcQStages;
        if (!(ok = wait(&ctl.q_empty[qs], ((qc / kTcQStages) & 1u) ^ 1u))) break;
        if (lane == 0) {
          uint8_t* dst = smem + L::kQ + qs * L::kTile;
          mbar_arrive_expect_tx(&ctl.q_full[qs], L::kTile);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(dst + c * 16384, &qmap, 64 * c, I.h * G, I.t0 + I.first_tok + t * tpt,
                        &ctl.q_full[qs]);
        }
        __syncwarp();
      }
    }
    // the latest fill of each stage is the only one that can still be in flight
    for (uint32_t g = kc > kTcKStages ? kc - kTcKStages : 0;
         kPool == Pool::kBf16 && g < kc + (ok ? 0 : 1); ++g)
      mbar_wait(&ctl.k_full[g % kTcKStages], (g / kTcKStages) & 1u, a.wait_ns);
    for (uint32_t g = qc > kTcQStages ? qc - kTcQStages : 0; g < qc; ++g)
      mbar_wait(&ctl.q_full[g % kTcQStages], (g / kTcQStages) & 1u, a.wait_ns);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const uint32_t idesc = idesc_bf16_f32(128, 128, false);
    for (int64_t item = blockIdx.x; ok && item < total; item += gridDim.x, ++kc) {
      const TcItem I = tc_item(a, item, tpt);
      const uint32_t ks = kc % kTcKStages;
      if (!(ok = wait(&ctl.k_full[ks], (kc / kTcKStages) & 1u))) break;
      for (int t = 0; t < I.tiles; ++t, ++qc) {
        const uint32_t qs = qc % kTcQStages, b = qc % kTcBufs;
        if (!(ok = wait(&ctl.d_empty[b], ((qc / kTcBufs) & 1u) ^ 1u))) break;
        if (!(ok = wait(&ctl.q_full[qs], (qc / kTcQStages) & 1u))) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t k_addr = smem_u32(smem + L::kK + ks * 2 * L::kTile);
          const uint32_t q_addr = smem_u32(smem + L::kQ + qs * L::kTile);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              // 64-column halves of a K block 1 KiB apart (8-key groups 2 KiB apart; one half for
              // head_dim 64: 1 KiB), of the q tile 16 KiB apart (8-row groups 1 KiB apart)
              tc_mma_bf16(tmem + b * 256u + m * 128u,
                          smem_desc_sw128(k_addr + m * L::kTile + (k >> 2) * 1024 + (k & 3) * 32, 16,
                                          D == 128 ? 2048 : 1024),
                          smem_desc_sw128(q_addr + (k >> 2) * 16384 + (k & 3) * 32, 16, 1024), idesc,
                          k > 0);
          tc_commit(&ctl.d_full[b]);
          tc_commit(&ctl.q_empty[qs]);
          if (t == I.tiles - 1) tc_commit(&ctl.k_empty[ks]);
        }
        __syncwarp();
      }
    }
    if (lane == 0) tc_commit(&ctl.drain);
    __syncwarp();
    mbar_wait(&ctl.drain, 0, a.wait_ns);  // no MMA is in flight when the CTA ends
  } else {
    // ---------------------------------------------------------------- epilogue
    const int e = warp - 2, m = e >> 3, half = (e >> 2) & 1;
    const int quarter = warp & 3;                 // TMEM lane quarter of the warp
    const int k = m * 128 + quarter * 32 + lane;  // key of the item: TMEM lane of accumulator m
    const uint32_t cols = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + m * 128u + half * 64u;
    const float scale = a.score_log2;
    // token and head, within a tile, of this lane's two columns of the warp's 64
    const int r0 = half * 64 + lane, r1 = r0 + 32;
    const int tok_0 = r0 / G, g_0 = r0 - tok_0 * G, tok_1 = r1 / G, g_1 = r1 - tok_1 * G;
    for (int64_t item = blockIdx.x; ok && item < total; item += gridDim.x, ++kc) {
      const TcItem I = tc_item(a, item, tpt);
      const int key = I.base + k;
      // negated log-sum-exp of a column of tile t (its token and head within the tile)
      auto lse_of = [&](int t, int tok_in, int g) {
        const int tok = I.first_tok + t * tpt + tok_in;
        return t < I.tiles && tok < I.n
                   ? -a.lse[static_cast<int64_t>(I.t0 + tok) * a.num_q_heads + I.h * G + g]
                   : -CUDART_INF_F;
      };
      float next0 = lse_of(0, tok_0, g_0), next1 = lse_of(0, tok_1, g_1);
      if constexpr (kPool != Pool::kBf16) {
        // the item's keys, converted by these warps: 16-byte pieces (8 dims) of the K tiles' layout
        constexpr int kEach = kTcKeys * (D / 8) / (32 * kTcEpilogue);
        const uint32_t ks = kc % kTcKStages;
        // (without branches, so that all the table's entries, then all the keys load at once; what
        // is not there reads the pool's first block and becomes zeros)
        int phys[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int kk = ((i * kTcEpilogue + e) * 32 + lane) / (D / 8);
          phys[i] = __ldg(a.block_tables + static_cast<int64_t>(I.s) * a.max_blocks_per_seq +
                          min(I.base + kk, I.L - 1) / kBlockSize);
        }
        uint32_t w[kEach][4];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int piece = (i * kTcEpilogue + e) * 32 + lane, kk = piece / (D / 8), c = piece % (D / 8);
          const bool there = I.base + kk < I.L && phys[i] >= 0 && phys[i] < a.num_blocks;
          load_dims<kPool, D>(a.k_cache, (there ? int64_t{phys[i]} : 0) * a.num_kv_heads + I.h,
                              kk % kBlockSize, c >> 2, c & 3, w[i]);
#pragma unroll
          for (int x = 0; x < 4; ++x) w[i][x] = there ? w[i][x] : 0u;  // (bad blocks are flagged by the attention)
        }
        if (!(ok = wait(&ctl.k_empty[ks], ((kc / kTcKStages) & 1u) ^ 1u))) break;
        const uint32_t base = smem_u32(smem + L::kK + ks * 2 * L::kTile);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int piece = (i * kTcEpilogue + e) * 32 + lane, kk = piece / (D / 8), c = piece % (D / 8);
          st_shared_v4(base + (kk >> 3) * (D * 16) + (c >> 3) * 1024 + (kk & 7) * 128 +
                           (((c & 7) ^ (kk & 7)) << 4),
                       w[i][0], w[i][1], w[i][2], w[i][3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.k_full[ks]);
      }
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int t = 0; t < I.tiles; ++t, ++qc) {
        const uint32_t b = qc % kTcBufs;
        __syncwarp();
        s_lse[e][lane] = next0;
        s_lse[e][lane + 32] = next1;
        __syncwarp();
        next0 = lse_of(t + 1, tok_0, g_0);
        next1 = lse_of(t + 1, tok_1, g_1);
        if (!(ok = wait(&ctl.d_full[b], (qc / kTcBufs) & 1u))) break;
        tc_fence_after();
        // columns of rows that see the key: from `from` on, and rows of the run only
        const int tok0 = I.first_tok + t * tpt;
        const int from = (key - (I.L - I.n) - tok0) * G - half * 64;
        const int upto = min(64, (I.n - tok0) * G - half * 64);
        const bool all = __all_sync(0xffffffffu, from <= 0) && upto == 64;
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 32) {
          uint32_t acc[32];
          tmem_ld32(cols + b * 256u + c0, acc);
          tmem_wait_ld();
          if (c0 == 32) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.d_empty[b]);
          }
          auto add = [&](auto all_tag) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 l = *reinterpret_cast<const float4*>(&s_lse[e][c0 + c]);
              const float v[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float w = fast_exp2(fmaf(__uint_as_float(acc[c + i]), scale, v[i]));
                if (decltype(all_tag)::value || (c0 + c + i >= from && c0 + c + i < upto)) sum[i] += w;
              }
            }
          };
          if (all) add(std::true_type());
          else add(std::false_type());
        }
      }
      if (!ok) break;
      // the sums of the item before are read
      if (kc > 0 && !(ok = wait(&ctl.sum_free, (kc - 1) & 1u))) break;
      s_part[half][k] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.sum_full);
      if (!(ok = wait(&ctl.sum_full, kc & 1u))) break;
      if (half == 0 && key < I.L) {
        float x = s_part[0][k] + s_part[1][k];
        const int phys = __ldg(a.block_tables + static_cast<int64_t>(I.s) * a.max_blocks_per_seq +
                               key / kBlockSize);
        // keys of bad blocks, which the attention leaves out, receive nothing
        if (phys < 0 || phys >= a.num_blocks) x = 0.f;
        const int64_t row = a.weight_rows ? a.weight_rows[I.s] : I.s;
        float* W = a.key_weights + (row * a.num_kv_heads + I.h) * static_cast<int64_t>(a.max_keys);
        W[key] = fmaf(a.decay, W[key], x);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.sum_free);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTcCols);
}

template <Pool kPool, int D>
cudaError_t run_tc(const KeyWeightsArgs& a, const PoolMaps& maps, cudaStream_t stream) {
  auto kern = key_weights_tc_kernel<kPool, D>;
  LaunchInfo li;
  cudaError_t e = launch_info(kern, kTcThreads, TcLayout<D>::kSmem, &li);
  if (e != cudaSuccess) return e;
  const int64_t upper = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads *
                        ((a.max_context_len + int64_t(kTcKeys) - 1) / kTcKeys);
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(upper, li.sms));
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(kTcThreads),
                          TcLayout<D>::kSmem, stream, maps.q3, D == 128 ? maps.k4 : maps.k2, a);
}

}  // namespace

cudaError_t launch_key_weights_tc(const KeyWeightsArgs& a, const PoolMaps& maps,
                                  cudaStream_t stream) {
  if (a.cache_dtype == PA_FP8_E4M3) return run_tc<Pool::kE4m3, 128>(a, maps, stream);
  if (a.cache_dtype == PA_MXFP4)
    return a.head_dim == 128 ? run_tc<Pool::kMx, 128>(a, maps, stream)
                             : run_tc<Pool::kMx, 64>(a, maps, stream);
  return a.head_dim == 128 ? run_tc<Pool::kBf16, 128>(a, maps, stream)
                           : run_tc<Pool::kBf16, 64>(a, maps, stream);
}

}  // namespace pa
