// Eviction of the keys that received the least attention, per sequence and kv head.
//
// What it computes: of the L keys of a sequence, k = min(keep, L) stay: the last r = min(recent,
// k) and, of the L - r before them, the k - r of the largest accumulated weight (ties: the lowest
// position first; NaN counts as -infinity).  Kept keys move, in their order, to positions
// 0 .. k - 1; their weights move with them and the weights of positions k .. L - 1 become 0.
//
//  * select_kernel: one CTA per (sequence, kv head).  The weights are mapped to integers of the
//    same order; three histogram passes of 11, 11 and 10 bits find the (k - r)-th largest and how
//    many of its equals are kept; a last pass, in order, writes the kept positions and weights.
//  * move_kernel: one CTA per (sequence, kv head, K or V, column slice).  A kept key never moves
//    up, so rows can move in place if a batch of them is read before it is written and batches go
//    in order: every source of a later batch lies above all that is written so far.  Batch c + 1
//    is loaded into registers before batch c is stored, so loads are always in flight.
#include <math_constants.h>

#include <algorithm>
#include <climits>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelPer = 4;  // positions of a lane in a pass of the CTA

struct EvictSeq {
  int L, k, r, row, dst_row;
  bool ok;  // false: the sequence is left as it is
};

__device__ __forceinline__ EvictSeq evict_seq(const EvictArgs& a, int s, uint32_t* bits) {
  EvictSeq e;
  e.L = a.context_lens[s];
  e.row = a.weight_rows ? a.weight_rows[s] : s;
  e.dst_row = a.dst_weight_rows ? a.dst_weight_rows[s] : e.row;
  const int keep = a.keep_lens[s];
  e.ok = true;
  *bits = 0;
  if (e.L < 0 || keep < 0 || e.L > a.max_context_len ||
      (e.L + kBlockSize - 1) / kBlockSize > a.max_blocks_per_seq ||
      min(keep, e.L) > a.max_keep_len) {
    *bits |= PA_DEVERR_LENGTHS;
    e.ok = false;
  }
  if (e.row >= a.num_weight_rows || e.dst_row >= a.num_weight_rows) {
    *bits |= PA_DEVERR_WEIGHT_ROW;
    e.ok = false;
  }
  if (e.row < 0 || e.dst_row < 0) e.ok = false;
  e.k = e.ok ? min(keep, e.L) : 0;
  e.r = min(a.recent, e.k);
  return e;
}

// Integer of the same order as the weight (-0 equals 0, NaN equals -infinity).
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0x007fffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictArgs a) {
  __shared__ int hist[2048];
  __shared__ int warp_gt[kSelWarps], warp_eq[kSelWarps];
  __shared__ int s_digit, s_above;
  grid_dependency_wait();
  grid_launch_dependents();
  const int s = blockIdx.x / a.num_kv_heads, h = blockIdx.x - s * a.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t bits;
  const EvictSeq e = evict_seq(a, s, &bits);
  if (tid == 0 && h == 0) {
    if (bits) set_error(a.err, bits);
    a.new_lens[s] = e.ok ? e.k : e.L;
  }
  int32_t* kept = a.kept + (static_cast<int64_t>(s) * a.num_kv_heads + h) * a.max_keep_len;
  for (int i = e.k + tid; i < a.max_keep_len; i += kSelThreads) kept[i] = -1;
  if (!e.ok) return;
  const float* W = a.key_weights +
                   (static_cast<int64_t>(e.row) * a.num_kv_heads + h) * a.max_keys;
  float* Wd = a.key_weights +
              (static_cast<int64_t>(e.dst_row) * a.num_kv_heads + h) * a.max_keys;
  const int N = e.L - e.r;   // the keys to choose from
  const int m = e.k - e.r;   // how many of them stay
  uint32_t prefix = 0;       // the m-th largest order key, digit by digit
  int need = m;              // how many keys with the prefix so far are kept
  if (m > 0 && m < N) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int nbits = pass == 2 ? 10 : 11;
      for (int i = tid; i < 2048; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j = tid; j < N; j += kSelThreads) {
        const uint32_t u = order_key(W[j]);
        if (pass == 0 || (u >> (shift + nbits)) == prefix)
          atomicAdd(&hist[(u >> shift) & ((1u << nbits) - 1)], 1);
      }
      __syncthreads();
      // the digit at which the count from the top reaches `need`: thread t sums four bins from
      // the top, then a scan over the CTA
      int c[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = hist[2047 - (4 * tid + i)];
        sum += c[i];
      }
      int x = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_gt[warp] = x;
      __syncthreads();
      int before = x - sum;
      for (int w = 0; w < warp; ++w) before += warp_gt[w];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (before < need && need <= before + c[i]) {
          s_digit = 2047 - (4 * tid + i);
          s_above = before;
        }
        before += c[i];
      }
      __syncthreads();
      prefix = (prefix << nbits) | static_cast<uint32_t>(s_digit);
      need -= s_above;
      __syncthreads();
    }
  }
  // kept: order key above `prefix`, the first `need` equal to it, and the last r
  const bool none = m == 0, all = m == N;
  int done = 0, done_eq = 0;  // kept so far; equals so far
  for (int base = 0; base < e.L; base += kSelThreads * kSelPer) {
    float w[kSelPer];
    unsigned gt[kSelPer], eq[kSelPer];
    int n_gt = 0, n_eq = 0;
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const int j = base + warp * (32 * kSelPer) + 32 * i + lane;
      w[i] = j < e.L ? W[j] : 0.f;
      const uint32_t u = order_key(w[i]);
      const bool in = j < N;
      const bool g = j < e.L && (!in || all || (!none && u > prefix));
      gt[i] = __ballot_sync(0xffffffffu, g);
      eq[i] = __ballot_sync(0xffffffffu, in && !all && !none && u == prefix);
      n_gt += __popc(gt[i]);
      n_eq += __popc(eq[i]);
    }
    if (lane == 0) {
      warp_gt[warp] = n_gt;
      warp_eq[warp] = n_eq;
    }
    __syncthreads();  // (and every weight of this pass is read before one is written)
    int b_gt = 0, b_eq = done_eq, t_gt = 0, t_eq = 0;
    for (int v = 0; v < kSelWarps; ++v) {
      if (v < warp) {
        b_gt += warp_gt[v];
        b_eq += warp_eq[v];
      }
      t_gt += warp_gt[v];
      t_eq += warp_eq[v];
    }
    // place of a kept key: those kept before it, done + (above since `base`) + (equals kept
    // since `base`)
    const int eq_kept0 = min(done_eq, need);
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const int j = base + warp * (32 * kSelPer) + 32 * i + lane;
      const unsigned below = (1u << lane) - 1;
      const int rank_eq = b_eq + __popc(eq[i] & below);
      const bool is_eq = (eq[i] >> lane) & 1;
      const bool keep = ((gt[i] >> lane) & 1) || (is_eq && rank_eq < need);
      const int at = done + b_gt + __popc(gt[i] & below) + min(rank_eq, need) - eq_kept0;
      if (keep) {
        kept[at] = j;
        Wd[at] = w[i];
      }
      b_gt += __popc(gt[i]);
      b_eq += __popc(eq[i]);
    }
    done += t_gt + min(done_eq + t_eq, need) - eq_kept0;
    done_eq += t_eq;
    __syncthreads();
  }
  for (int i = e.k + tid; i < e.L; i += kSelThreads) Wd[i] = 0.f;
}

constexpr int kMoveThreads = 256;
constexpr int kMovePer = 4;  // 16-byte pieces of a thread in a batch

// kVec: 16-byte pieces of a row's slice.  MXFP4 rows (kNB > 0) also have kNB scale bytes, which
// the threads with the row's first piece move.
template <int kNB>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictArgs a, int row_bytes,
                                                            int slices, int vec) {
  grid_dependency_wait();
  int id = blockIdx.x;
  const int slice = id % slices;
  id /= slices;
  const int is_v = id & 1;
  id >>= 1;
  const int h = id % a.num_kv_heads, s = id / a.num_kv_heads;
  uint32_t bits;
  const EvictSeq e = evict_seq(a, s, &bits);
  if (!e.ok) return;
  uint8_t* pool = is_v ? a.v_cache : a.k_cache;
  const int32_t* kept = a.kept + (static_cast<int64_t>(s) * a.num_kv_heads + h) * a.max_keep_len;
  const int32_t* src_t = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  const int32_t* dst_t = a.dst_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  const int tile_bytes = row_bytes * kBlockSize + kNB * kBlockSize;
  const int rows = kMoveThreads * kMovePer / vec;  // rows of a batch
  uint4 x[2][kMovePer];
  uint32_t sc[2][kMovePer];
  int64_t to[2][kMovePer];  // byte offset of the destination row, or -1
  auto load = [&](int buf, int first) {
#pragma unroll
    for (int i = 0; i < kMovePer; ++i) {
      const int unit = i * kMoveThreads + threadIdx.x;
      const int r = unit / vec, c = unit - r * vec;
      const int at = first + r;
      to[buf][i] = -1;
      if (at < e.k && r < rows) {
        const int j = kept[at];
        const int from_b = __ldg(src_t + j / kBlockSize), to_b = __ldg(dst_t + at / kBlockSize);
        if (from_b < 0 || from_b >= a.num_blocks || to_b < 0 || to_b >= a.num_blocks) {
          set_error(a.err, PA_DEVERR_BLOCK_ID);
        } else if (from_b != to_b || j % kBlockSize != at % kBlockSize) {
          const int64_t ft = (static_cast<int64_t>(from_b) * a.num_kv_heads + h) * tile_bytes;
          const int64_t tt = (static_cast<int64_t>(to_b) * a.num_kv_heads + h) * tile_bytes;
          const int fo = j % kBlockSize, tof = at % kBlockSize;
          const int col = (slice * vec + c) * 16;
          x[buf][i] = *reinterpret_cast<const uint4*>(pool + ft + fo * row_bytes + col);
          to[buf][i] = tt + tof * row_bytes + col;
          if (kNB == 4 && col == 0)
            sc[buf][i] = *reinterpret_cast<const uint32_t*>(pool + ft + kBlockSize * row_bytes + fo * kNB);
          if (kNB == 2 && col == 0)
            sc[buf][i] = *reinterpret_cast<const uint16_t*>(pool + ft + kBlockSize * row_bytes + fo * kNB);
        }
      }
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kMovePer; ++i) {
      if (to[buf][i] < 0) continue;
      *reinterpret_cast<uint4*>(pool + to[buf][i]) = x[buf][i];
      if (kNB > 0) {
        const int unit = i * kMoveThreads + threadIdx.x;
        if (slice == 0 && unit % vec == 0) {
          const int64_t tile = to[buf][i] / tile_bytes * tile_bytes;
          const int off = static_cast<int>(to[buf][i] - tile) / row_bytes;
          uint8_t* d = pool + tile + kBlockSize * row_bytes + off * kNB;
          if (kNB == 4) *reinterpret_cast<uint32_t*>(d) = sc[buf][i];
          else *reinterpret_cast<uint16_t*>(d) = static_cast<uint16_t>(sc[buf][i]);
        }
      }
    }
  };
  load(0, 0);
  for (int first = 0; first < e.k; first += 2 * rows) {
    load(1, first + rows);
    __syncthreads();  // batch 0 of this round is read by everyone
    store(0);
    load(0, first + 2 * rows);
    __syncthreads();
    store(1);
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  const int row_bytes = a.cache_dtype == PA_MXFP4 ? a.head_dim / 2
                        : a.cache_dtype == PA_FP8_E4M3 ? a.head_dim : 2 * a.head_dim;
  const int vecs = row_bytes / 16;
  const int64_t ctas = 2 * pairs;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = launch_dependent(select_kernel, dim3(static_cast<unsigned>(pairs)),
                                   dim3(kSelThreads), 0, stream, a);
  if (e != cudaSuccess || a.max_keep_len == 0) return e;
  auto kern = a.cache_dtype != PA_MXFP4 ? move_kernel<0>
              : a.head_dim == 128       ? move_kernel<4> : move_kernel<2>;
  return launch_dependent(kern, dim3(static_cast<unsigned>(ctas)), dim3(kMoveThreads), 0, stream,
                          a, row_bytes, 1, vecs);
}

}  // namespace pa
