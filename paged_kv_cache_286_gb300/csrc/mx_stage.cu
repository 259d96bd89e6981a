// Prompt chunks over MXFP4 pools: the keys and values of the sequences with long query runs are
// written out once as bf16 (exact: a code has two significant bits, its scale is a power of two)
// and the tensor-core prefill tiles read those.
//
// A chunk reads each of its sequence's tiles once for every 128 rows of queries, so converting
// them once (2 KiB written per 544 bytes read, the copy of a 2,560-key context for 8 kv heads
// 10 MB) costs less than converting them in every tile; and the MMAs cannot take the codes as they
// are: V's scales change along the keys, the dimension that P V sums over.  Measured: that copy 6.7
// us, the plan before it 2.8; a run of 512 x 32 heads over it beside 16 decodes 74 us in all, where
// the split-KV kernel alone took 327.
#include <algorithm>

#include "decode_items.cuh"
#include "mxfp4.cuh"
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

// One CTA: which sequences are staged (those with runs of more rows than the split-KV kernel's
// largest tile, in order, while the area holds them) and the prefix sums of their blocks.
__global__ void __launch_bounds__(1024) mx_stage_plan_kernel(const DecodeParams p,
                                                             int32_t* __restrict__ stage_pre,
                                                             int32_t capacity) {
  grid_dependency_wait();
  __shared__ int64_t warp_sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t carry = 0;  // blocks of the candidates so far
  for (int base = 0; base < p.num_seqs; base += 1024) {
    const int s = base + tid;
    int64_t c = 0;
    if (s < p.num_seqs) {
      const int n = p.qsl[s + 1] - p.qsl[s], L = p.context_lens[s];
      const bool good = n > 0 && n <= L && L <= p.max_context_len && n <= p.max_query_len &&
                        L <= p.max_blocks_per_seq * kBlockSize;
      if (good && static_cast<int64_t>(n) * p.group > kMxMaxRows) c = ceil_div(L, kBlockSize);
    }
    int64_t x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int64_t w = warp_sums[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      warp_sums[lane] = w;
    }
    __syncthreads();
    const int64_t before = carry + (warp ? warp_sums[warp - 1] : 0) + x - c;
    // candidates past the capacity are not staged: their prefix stays at the last staged block
    if (s < p.num_seqs)
      stage_pre[s] = static_cast<int32_t>(before <= capacity ? before : -1);
    if (s < p.num_seqs && before <= capacity && before + c > capacity)
      stage_pre[p.num_seqs] = static_cast<int32_t>(before);  // the first that does not fit
    carry += warp_sums[31];
    __syncthreads();
  }
  // (one thread's stores of the loop above are visible to the CTA after the barrier)
  if (carry <= capacity) {
    if (tid == 0) stage_pre[p.num_seqs] = static_cast<int32_t>(carry);
  } else {
    const int total = stage_pre[p.num_seqs];
    for (int s = tid; s < p.num_seqs; s += 1024)
      if (stage_pre[s] < 0) stage_pre[s] = total;
  }
}

// One CTA per (staged block, kv head) at a time, K then V: a thread has 8 dims of a row.
template <int D>
__global__ void __launch_bounds__(2 * D) mx_stage_kernel(
    const DecodeParams p, const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool,
    const int32_t* __restrict__ stage_pre, int32_t* __restrict__ table, int32_t table_stride,
    uint4* __restrict__ k_out, uint4* __restrict__ v_out) {
  constexpr int NB = D / 32, VEC = D / 8;
  grid_dependency_wait();
  const int row = threadIdx.x / VEC, c = threadIdx.x % VEC;
  const int b = c >> 2, g = 2 * (c & 3);
  const int64_t units = static_cast<int64_t>(stage_pre[p.num_seqs]) * p.num_kv_heads;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int blk = static_cast<int>(u / p.num_kv_heads);
    const int h = static_cast<int>(u - static_cast<int64_t>(blk) * p.num_kv_heads);
    int lo = 0, hi = p.num_seqs;  // largest s with stage_pre[s] <= blk
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (stage_pre[mid] <= blk) lo = mid; else hi = mid;
    }
    const int j = blk - stage_pre[lo];  // its block of that sequence
    const int phys = __ldg(p.block_tables + static_cast<int64_t>(lo) * p.max_blocks_per_seq + j);
    const bool ok = phys >= 0 && phys < p.num_blocks;
    if (h == 0 && threadIdx.x == 0) table[static_cast<int64_t>(lo) * table_stride + j] = ok ? blk : -1;
    if (!ok) continue;  // (the prefill tiles flag the table's entry)
    const int64_t tile = (static_cast<int64_t>(phys) * p.num_kv_heads + h) * Mx<D>::kTileBytes;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint8_t* t = (kv ? v_pool : k_pool) + tile;
      const uint16_t* src = reinterpret_cast<const uint16_t*>(t + row * Mx<D>::kRowBytes);
      const uint32_t codes = __ldg(src + g * NB + b) |
                             (static_cast<uint32_t>(__ldg(src + (g + 1) * NB + b)) << 16);
      const float sc = e8m0_to_f32(__ldg(t + Mx<D>::kCodeBytes + row * NB + b));
      uint32_t f[4], w[4];
      e2m1x8_to_f16x2x4(codes, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
        w[i] = pack_bf16x2(y.x * sc, y.y * sc);
      }
      (kv ? v_out : k_out)[u * (kBlockSize * VEC) + threadIdx.x] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

cudaError_t launch_mx_stage_plan(const AttnArgs& a, const DecodeParams& p) {
  return launch_dependent(mx_stage_plan_kernel, dim3(1), dim3(1024), 0, a.stream, p,
                          a.stage.prefix, a.stage.capacity);
}

cudaError_t launch_mx_stage(const AttnArgs& a, const DecodeParams& p) {
  LaunchInfo li;
  auto run = [&](auto kern, int threads) {
    cudaError_t e = launch_info(kern, threads, 0, &li);
    if (e != cudaSuccess) return e;
    const int64_t upper = static_cast<int64_t>(a.stage.capacity) * a.num_kv_heads;
    const int64_t grid = std::min<int64_t>(upper, int64_t(li.sms) * li.per_sm);
    return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, a.stream, p,
                            static_cast<const uint8_t*>(a.k_cache),
                            static_cast<const uint8_t*>(a.v_cache), a.stage.prefix, a.stage.table,
                            a.stage.table_stride, static_cast<uint4*>(a.stage.k),
                            static_cast<uint4*>(a.stage.v));
  };
  return a.head_dim == 128 ? run(mx_stage_kernel<128>, 256) : run(mx_stage_kernel<64>, 128);
}

}  // namespace pa
