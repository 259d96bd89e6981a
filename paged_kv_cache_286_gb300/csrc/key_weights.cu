// Accumulated attention weight of every cached key, for eviction by weight.
//
// What it computes, after the attention of the step has left each row's log-sum-exp (a row is a
// query token and q head): for every key j of a sequence with query tokens, per kv head,
//   W[j] <- decay * W[j] + sum over the rows that see j of 2^(s_j - lse_row),
// s_j = scale * log2(e) * q . k_j, i.e. the sum of the softmax weights that j received.
//
//  * Decode tokens and short verify runs: the attention's split-KV kernel writes its scores (4 bytes
//    per row and key) and kw_finish_kernel reads them; K is not read again.
//    256 sequences of 1,000 keys on average, 32 q heads on 8: 21 us; of 64 x 32 kv heads, 16 us.
//  * Longer runs, whose scores would be more bytes than K, where there are not enough keys for the
//    tensor-core kernel (key_weights_tc.cu): the keys stay and the rows pass.  A warp
//    holds 32 keys of one kv head as MMA fragments (M = keys, two m16 tiles) and the rows of the
//    group pass through shared memory as the N operand, eight at a time, so a key's sum over rows
//    stays in the lanes that own it and is written once, in a fixed order: no atomics, the same
//    bits every time.  A cluster of four CTAs shares the rows of 128 keys, so that a single chunk
//    (512 tokens after 2,048: 160 items) fills the GPU.  It reaches 165 to 190 TFLOP/s, bound by
//    the mma.sync rate with an FMA, a 2^x and an add beside every score.
//  * The log-sum-exp is known, so there is no running maximum: a score costs one FMA, one 2^x and
//    one add.
//  * Every pool type becomes bf16 fragments, exactly (E4M3 has four significant bits, E2M1 times
//    a power of two has two), so q is used as it is and the loop over the rows is the same.
#include <math_constants.h>

#include <algorithm>
#include <climits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pool_keys.cuh"

namespace pa {

namespace {

constexpr int kKwKeys = 128;    // keys of an item: four groups of 32
constexpr int kKwWarps = 8;     // key group x half of the staged rows
constexpr int kKwRows = 64;     // rows staged in shared memory at a time
constexpr int kKwCluster = 4;   // CTAs that share an item's rows


// Whether a wait of the attention before has run out (in this call, or in an earlier one whose error
// nobody has read): its log-sum-exps and scores are not all there, and the weights, which last over
// steps, stay as they are.
__device__ __forceinline__ bool kw_timed_out(const KeyWeightsArgs& a) {
  return *a.err & PA_DEVERR_TIMEOUT;
}

// Whether a sequence accumulates weights in this step.
__device__ __forceinline__ bool kw_accumulates(const KeyWeightsArgs& a, int s,
                                               uint32_t* err_bits) {
  const int n = a.qsl[s + 1] - a.qsl[s], L = a.context_lens[s];
  // (what the attention's plan flags and skips is skipped here too)
  if (n <= 0 || n > L || L > a.max_context_len || n > a.max_query_len ||
      L > a.max_blocks_per_seq * kBlockSize)
    return false;
  const int row = a.weight_rows ? a.weight_rows[s] : s;
  if (row < 0) return false;
  if (row >= a.num_weight_rows) {
    *err_bits |= PA_DEVERR_WEIGHT_ROW;
    return false;
  }
  return true;
}

// Items of a sequence for the kernel that reads K: its key chunks, if its scores were not kept.
__device__ __forceinline__ int kw_chunks(const KeyWeightsArgs& a, int s, uint32_t* err_bits) {
  if (!kw_accumulates(a, s, err_bits)) return 0;
  if ((a.qsl[s + 1] - a.qsl[s]) * (a.num_q_heads / a.num_kv_heads) <= a.score_rows) return 0;
  return (a.context_lens[s] + a.chunk_keys - 1) / a.chunk_keys;
}

// Runs whose scores the attention kept: one CTA per (sequence, kv head) and equal share of its
// keys, four neighbouring keys (of one block) to a thread.  Bound by the scores' bytes (mostly
// L2's) and by launch.
constexpr int kFinThreads = 256;
constexpr int kFinShare = 4096;  // keys of a share at least (of the longest sequence)
template <bool kBeside>
__device__ __forceinline__ void finish_share(const KeyWeightsArgs& a) {
  __shared__ float s_lse[kDecodeMaxRows];
  const int s = blockIdx.x, h = blockIdx.y;
  uint32_t bits = 0;
  const bool lost = kw_timed_out(a);
  const bool ok = kw_accumulates(a, s, &bits);
  if (bits && threadIdx.x == 0) set_error(a.err, bits);
  // (beside the tensor-core kernel, which may set the bit meanwhile: one answer for the CTA)
  if (kBeside ? __syncthreads_or(!ok || lost) : !ok || lost) return;
  const int t0 = a.qsl[s], n = a.qsl[s + 1] - t0, L = a.context_lens[s];
  const int G = a.num_q_heads / a.num_kv_heads;
  if (n * G > a.score_rows || (blockIdx.z && blockIdx.z * kFinShare >= L)) return;
  const int rows = n * G;
  if (threadIdx.x < rows)
    s_lse[threadIdx.x] = a.lse[static_cast<int64_t>(t0 + threadIdx.x / G) * a.num_q_heads + h * G +
                               threadIdx.x % G];
  const int row = a.weight_rows ? a.weight_rows[s] : s;
  float* W = a.key_weights + (static_cast<int64_t>(row) * a.num_kv_heads + h) * a.max_keys;
  const float* sc = a.scores + (static_cast<int64_t>(s) * a.num_kv_heads + h) * a.score_rows *
                                   a.score_stride;
  const int32_t* table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  const int groups = (L + 3) / 4;
  const int share = gridDim.z == 1 ? groups
                                   : max(kFinShare / 4, static_cast<int>((groups + gridDim.z - 1) / gridDim.z));
  const int end = min(groups, share * (static_cast<int>(blockIdx.z) + 1));
  // rounds of the CTA; a round's loads (up to four rows of scores) go out together, the first
  // round's before the log-sum-exps are there
  for (int first = share * blockIdx.z; first < end; first += kFinThreads) {
    const int g = first + threadIdx.x, key = 4 * g;
    const bool mine = g < end;
    float w[4], sum[4] = {0.f, 0.f, 0.f, 0.f};
    float4 x[4];
    int phys = -1;
    const float* col = sc + key;
    if (mine) {
      phys = __ldg(table + key / kBlockSize);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = key + i < L ? W[key + i] : 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < rows) x[r] = *reinterpret_cast<const float4*>(col + static_cast<int64_t>(r) * a.score_stride);
    }
    if (first == share * static_cast<int>(blockIdx.z)) __syncthreads();
    if (!mine) break;
    if (phys >= 0 && phys < a.num_blocks) {  // (the attention leaves bad blocks out)
      for (int r0 = 0; r0 < rows; r0 += 4) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (r0 + r >= rows) break;
          // the row's position: it sees keys up to this one
          const int pos = n == 1 ? L - 1 : L - n + (r0 + r) / G;
          const float v[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key + i <= pos) sum[i] += fast_exp2(v[i] - s_lse[r0 + r]);
          if (r0 + 4 + r < rows)
            x[r] = *reinterpret_cast<const float4*>(col + static_cast<int64_t>(r0 + 4 + r) * a.score_stride);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (key + i < L) W[key + i] = fmaf(a.decay, w[i], sum[i]);
  }
}

// kBeside: launched after the tensor-core kernel, which has other sequences and lets it start once the
// attention is complete, it waits for that kernel only at its end.  In 40 registers a CTA fits in
// what one of that kernel's leaves of an SM (48 decodes beside two runs of 512: 138.8 -> 133.9 us,
// with 60 registers 137.6).  Alone, five CTAs to an SM: 256 sequences of 1,000 keys on average,
// the whole step 159 us; with six 161, with three 163.
template <bool kBeside>
__global__ void __launch_bounds__(kFinThreads, kBeside ? 6 : 5)
    kw_finish_kernel(const KeyWeightsArgs a) {
  if (!kBeside) grid_dependency_wait();
  finish_share<kBeside>(a);
  if (kBeside) grid_dependency_wait();
}

// One CTA: exclusive prefix sums of the sequences' chunks.
__global__ void __launch_bounds__(1024) kw_plan_kernel(const KeyWeightsArgs a) {
  grid_dependency_wait();
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int carry = 0;
  uint32_t bits = 0;
  const bool lost = __syncthreads_or(kw_timed_out(a));  // then there are no items
  for (int base = 0; base < a.num_seqs; base += 1024) {
    const int s = base + tid;
    const int c = s < a.num_seqs && !lost ? kw_chunks(a, s, &bits) : 0;
    int x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int w = warp_sums[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      warp_sums[lane] = w;
    }
    __syncthreads();
    if (s < a.num_seqs) a.chunk_start[s] = carry + (warp ? warp_sums[warp - 1] : 0) + x - c;
    carry += warp_sums[31];
    __syncthreads();
  }
  if (tid == 0) a.chunk_start[a.num_seqs] = carry;
  if (bits) set_error(a.err, bits);
}

template <int D>
constexpr int kKwStride = D * 2 + 16;  // bytes of a row in shared memory: ldmatrix without conflicts
template <int D>
constexpr int kKwSmem = (kKwKeys + 2 * kKwRows) * kKwStride<D>;

// A cluster has an item (128 keys of a kv head); its CTAs take the item's 64-row tiles in turn, and
// their sums meet through distributed shared memory, CTA 0's first.
template <Pool kPool, int D>
__global__ void __cluster_dims__(kKwCluster, 1, 1) __launch_bounds__(kKwWarps * 32, 2)
    key_weights_kernel(const KeyWeightsArgs a) {
  constexpr int KS = D / 16;               // MMA k-steps
  constexpr int kStride = kKwStride<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* s_k = smem;                               // [128 keys][kStride]
  uint8_t* s_q[2] = {smem + kKwKeys * kStride, smem + (kKwKeys + kKwRows) * kStride};
  __shared__ __align__(8) float s_lse[2][kKwRows];
  __shared__ float s_half[2][kKwKeys];     // sums of the two halves of the rows
  __shared__ float s_sum[kKwKeys];         // of the CTA
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quad = lane >> 2, qc = lane & 3;
  const int group = warp & 3, half = warp >> 2;
  const int rank = blockIdx.x % kKwCluster;
  const int total = a.chunk_start[a.num_seqs];
  const int G = a.num_q_heads / a.num_kv_heads;
  // x / G for 0 <= x < 2^28 (G <= 16): the high word of x * ceil(2^32 / G) is off by less than
  // x * 16 / 2^32 < 1 / G
  const uint32_t magic = static_cast<uint32_t>(((1ull << 32) + G - 1) / G);
  auto div_g = [&](int x) {
    return G == 1 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), magic));
  };

  for (int64_t item = blockIdx.x / kKwCluster;
       item < static_cast<int64_t>(total) * a.num_kv_heads; item += gridDim.x / kKwCluster) {
    const int chunk_id = static_cast<int>(item / a.num_kv_heads);
    const int h = static_cast<int>(item - static_cast<int64_t>(chunk_id) * a.num_kv_heads);
    int lo = 0, hi = a.num_seqs;  // largest s with chunk_start[s] <= chunk_id
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.chunk_start[mid] <= chunk_id) lo = mid; else hi = mid;
    }
    const int s = lo;
    const int t0 = a.qsl[s], n = a.qsl[s + 1] - t0, L = a.context_lens[s];
    const int base = (chunk_id - a.chunk_start[s]) * kKwKeys;  // first key of the item
    const int key_w = base + 32 * group;                        // first key of the warp
    // the rows of the tokens that see some key of the item, in tiles of 64
    const int first_tok = max(0, base - (L - n));
    const int rows = (n - first_tok) * G;
    const int tiles = (rows + kKwRows - 1) / kKwRows;
    auto stage = [&](int tile, int buf) {
      const int r0 = tile * kKwRows, nr = min(kKwRows, rows - r0);
      for (int e = threadIdx.x; e < kKwRows * (D / 8); e += kKwWarps * 32) {
        const int r = e / (D / 8), c = e - r * (D / 8);
        const int at = r0 + min(r, nr - 1);  // (rows past the run: zeros)
        const int tok = div_g(at);
        cp_async16_zfill(
            smem_u32(s_q[buf] + r * kStride + 16 * c),
            a.q + (static_cast<int64_t>(t0 + first_tok + tok) * a.num_q_heads + h * G + at - tok * G) * D +
                8 * c,
            r < nr ? 16 : 0);
      }
      if (threadIdx.x < kKwRows) {
        const int r = threadIdx.x, at = r0 + r, tok = div_g(at);
        if (r < nr)
          cp_async4(smem_u32(&s_lse[buf][r]),
                    a.lse + static_cast<int64_t>(t0 + first_tok + tok) * a.num_q_heads + h * G + at -
                        tok * G);
        else
          s_lse[buf][r] = CUDART_INF_F;  // 2^(0 - inf) = 0
      }
      cp_async_commit();
    };
    // ---- the item's keys as bf16 in shared memory, then as MMA fragments (A operand): keys
    // key_w + 16 m + quad (+ 8).  (Loaded straight into registers, a key's 16 bytes are four
    // registers of two fragments, and moving them cost as much as the MMAs.) -----------------
    if (rank < tiles) {
      for (int e = threadIdx.x; e < kKwKeys * (D / 8); e += kKwWarps * 32) {
        const int k = e / (D / 8), c = e - k * (D / 8), key = base + k;
        int phys = -1;
        if (key < L)
          phys = __ldg(a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq +
                       key / kBlockSize);
        const bool ok = phys >= 0 && phys < a.num_blocks;
        const int64_t tile = static_cast<int64_t>(ok ? phys : 0) * a.num_kv_heads + h;
        uint8_t* dst = s_k + k * kStride + 16 * c;
        if constexpr (kPool == Pool::kBf16) {
          cp_async16_zfill(
              smem_u32(dst),
              a.k_cache + ((tile * kBlockSize + key % kBlockSize) * D + 8 * c) * 2, ok ? 16 : 0);
        } else {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
          if (ok) load_dims<kPool, D>(a.k_cache, tile, key % kBlockSize, c >> 2, c & 3, w);
          *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      cp_async_commit();
      stage(rank, 0);
      cp_async_wait<1>();
    }
    __syncthreads();
    uint32_t kf[2][KS][4];
    float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};  // [m][i]
    if (rank < tiles) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
          ldsm_x4(smem_u32(s_k + (32 * group + 16 * m + (lane & 15)) * kStride + 32 * ks +
                           (lane >> 4) * 16),
                  kf[m][ks][0], kf[m][ks][1], kf[m][ks][2], kf[m][ks][3]);
    }

    int buf = 0;
    for (int tile = rank; tile < tiles; tile += kKwCluster, buf ^= 1) {
      const int r0 = tile * kKwRows, nr = min(kKwRows, rows - r0);
      cp_async_wait<0>();
      __syncthreads();  // the tile is staged, and everyone is done with the buffer of the last one
      if (tile + kKwCluster < tiles) stage(tile + kKwCluster, buf ^ 1);
      for (int rt = 32 * half; rt < min(nr, 32 * half + 32); rt += 8) {
        float acc[2][4];
#pragma unroll
        for (int k2 = 0; k2 < KS / 2; ++k2) {  // two k-steps of the tile's eight rows
          uint32_t b[4];
          ldsm_x4(smem_u32(s_q[buf] + (rt + (lane & 7)) * kStride + 64 * k2 + (lane >> 3) * 16),
                  b[0], b[1], b[2], b[3]);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (k2 == 0) mma_bf16_zero(acc[m], kf[m][0], b[0], b[1]);
            else mma_bf16(acc[m], kf[m][2 * k2], b[0], b[1]);
            mma_bf16(acc[m], kf[m][2 * k2 + 1], b[2], b[3]);
          }
        }
        const float2 lse = *reinterpret_cast<const float2*>(&s_lse[buf][rt + 2 * qc]);
        // rows that do not see a key add nothing to it; every row sees the warp's keys if the
        // tile's first does.  (Rows that the run does not fill take the other way: they are zeros, but
        // zero times a key's infinity is NaN.)
        if (rt + 8 <= nr && key_w + 31 <= L - n + first_tok + div_g(r0 + rt)) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              sum[m][i] += fast_exp2(fmaf(acc[m][2 * i], a.score_log2, -lse.x));
              sum[m][i] += fast_exp2(fmaf(acc[m][2 * i + 1], a.score_log2, -lse.y));
            }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = rt + 2 * qc + j;
            const int pos = r < nr ? L - n + first_tok + div_g(r0 + r) : -1;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float w =
                    fast_exp2(fmaf(acc[m][2 * i + j], a.score_log2, j ? -lse.y : -lse.x));
                if (key_w + 16 * m + quad + 8 * i <= pos) sum[m][i] += w;
              }
          }
        }
      }
    }
    // ---- sums over the four lanes of a key, the halves and the CTAs, and the update ---------
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = sum[m][i];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (qc == 0) s_half[half][32 * group + 16 * m + quad + 8 * i] = x;
      }
    __syncthreads();
    if (threadIdx.x < kKwKeys) s_sum[threadIdx.x] = s_half[0][threadIdx.x] + s_half[1][threadIdx.x];
    cluster_arrive();
    cluster_wait();  // every CTA's sums are there
    constexpr int kShare = kKwKeys / kKwCluster;  // keys that this CTA updates
    if (threadIdx.x < kShare) {
      const int k = rank * kShare + threadIdx.x, key = base + k;
      float x = 0.f;
#pragma unroll
      for (int c = 0; c < kKwCluster; ++c) x += ld_cluster(&s_sum[k], c);
      if (key < L) {
        const int phys = __ldg(a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq +
                               key / kBlockSize);
        // keys of bad blocks, which the attention leaves out, receive nothing
        if (phys < 0 || phys >= a.num_blocks) x = 0.f;
        const int64_t row = a.weight_rows ? a.weight_rows[s] : s;
        float* W = a.key_weights + (row * a.num_kv_heads + h) * static_cast<int64_t>(a.max_keys);
        W[key] = fmaf(a.decay, W[key], x);
      }
    }
    cluster_arrive();
    cluster_wait();  // the sums are read before they are written again
  }
}

template <Pool kPool, int D>
cudaError_t run_key_weights(const KeyWeightsArgs& a, cudaStream_t stream) {
  auto kern = key_weights_kernel<kPool, D>;
  LaunchInfo li;
  cudaError_t e = launch_info(kern, kKwWarps * 32, kKwSmem<D>, &li);
  if (e != cudaSuccess) return e;
  const int64_t upper = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads *
                        ((a.max_context_len + int64_t(kKwKeys) - 1) / kKwKeys);
  const int64_t resident = int64_t(li.sms) * li.per_sm / kKwCluster;
  const int64_t clusters = std::max<int64_t>(1, std::min(upper, resident));
  return launch_dependent(kern, dim3(static_cast<unsigned>(clusters * kKwCluster)),
                          dim3(kKwWarps * 32), kKwSmem<D>, stream, a);
}

}  // namespace

cudaError_t launch_key_weights(KeyWeightsArgs a, const PoolMaps* maps, cudaStream_t stream) {
  a.chunk_keys = maps ? kKeyWeightsTcKeys : kKwKeys;
  const bool beside = a.k_pass && maps;  // of the tensor-core kernel, on the SMs that it leaves idle
  auto finish = [&] {
    const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
    const int64_t shares = std::min<int64_t>((a.max_context_len + int64_t(kFinShare) - 1) / kFinShare, 65535);
    if (pairs > INT32_MAX || a.num_kv_heads > 65535) return cudaErrorInvalidValue;
    return launch_dependent(beside ? kw_finish_kernel<true> : kw_finish_kernel<false>,
                            dim3(a.num_seqs, a.num_kv_heads, unsigned(shares)), dim3(kFinThreads),
                            0, stream, a);
  };
  cudaError_t e = cudaSuccess;
  if (a.scores && !beside && (e = finish()) != cudaSuccess) return e;
  if (!a.k_pass) return cudaSuccess;
  e = launch_dependent(kw_plan_kernel, dim3(1), dim3(1024), 0, stream, a);
  if (e != cudaSuccess) return e;
  if (maps) {
    e = launch_key_weights_tc(a, *maps, stream);
    return e == cudaSuccess && a.scores ? finish() : e;
  }
  if (a.cache_dtype == PA_FP8_E4M3) return run_key_weights<Pool::kE4m3, 128>(a, stream);
  if (a.cache_dtype == PA_MXFP4)
    return a.head_dim == 128 ? run_key_weights<Pool::kMx, 128>(a, stream)
                             : run_key_weights<Pool::kMx, 64>(a, stream);
  return a.head_dim == 128 ? run_key_weights<Pool::kBf16, 128>(a, stream)
                           : run_key_weights<Pool::kBf16, 64>(a, stream);
}

}  // namespace pa
