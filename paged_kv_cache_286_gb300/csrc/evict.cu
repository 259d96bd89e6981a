// Eviction of the keys that received the least attention, per sequence and kv head.
//
// What it computes: of the L keys of a sequence, k = min(keep, L) stay: the last r = min(recent,
// k) and, of the L - r before them, the k - r of the largest accumulated weight (ties: the lowest
// position first; NaN counts as -infinity).  Kept keys move, in their order, to positions
// 0 .. k - 1; their weights move with them and the weights of positions k .. L - 1 become 0.
//
//  * select_kernel: one CTA per (sequence, kv head).  The weights are mapped to integers of the
//    same order, which stay in shared memory; three histogram passes of 11, 11 and 10 bits find
//    the (k - r)-th largest and how many of its equals are kept; a last pass, in order, compacts
//    the kept positions, whose weights are then moved.
//    Instructions bound it, some 80 per 32 keys, then the latency of its eleven barriers: 16 x 8
//    rows of 32,768 weights 24 us, 64 x 32 rows of 2,300 on average 37 us.
//  * move_kernel: one CTA per (sequence, kv head, K or V, column slice).  A kept key never moves
//    up, so rows can move in place if a batch of them is read before it is written and batches go
//    in order: every source of a later batch lies above all that is written so far.  Positions,
//    table entries and rows are loads that wait on one another; they run two, one and no batches
//    ahead.  HBM bounds it: 64 x 32 x 1,001 rows of 256 bytes, K and V, 308 us (2.1 GB read and
//    written, 6.8 TB/s); 16 x 8 x 2,048 rows 45 us (5.9 TB/s).
#include <math_constants.h>

#include <algorithm>
#include <climits>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

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

// Adds 1 to a word of shared memory (predicated: a branch per key costs more than the sum).
__device__ __forceinline__ void inc_shared_if(bool yes, uint32_t at) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %0, 0;\n@p red.shared.add.u32 [%1], 1;\n}"
               ::"r"(static_cast<uint32_t>(yes)), "r"(at) : "memory");
}

constexpr int kSelPer = 8;  // positions of a thread in a round of the last pass

// Exclusive sum over the CTA's warps of each warp's `mine` (the same in all its lanes), through
// `slots`; *all is the total.  A barrier before it is the caller's.
template <int kWarps>
__device__ __forceinline__ int warps_exclusive(int mine, int* slots, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) slots[warp] = mine;
  __syncthreads();
  int x = lane < kWarps ? slots[lane] : 0;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  *all = __shfl_sync(0xffffffffu, x, kWarps - 1);
  return __shfl_sync(0xffffffffu, x, warp) - mine;
}

// `cached`: the order keys of that many first positions stay in shared memory between the passes.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) select_kernel(const EvictArgs a, int cached) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kBins = 2048 / kThreads;  // of a thread
  extern __shared__ __align__(16) uint32_t s_key[];
  __shared__ int hist[2048];
  __shared__ int slots[2][kWarps];
  __shared__ int s_digit, s_above;
  grid_dependency_wait();  // (the moves are not launched early: their CTAs would take SMs from this)
  const int s = blockIdx.x / a.num_kv_heads, h = blockIdx.x - s * a.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t bits;
  const EvictSeq e = evict_seq(a, s, &bits);
  if (tid == 0 && h == 0) {
    if (bits) set_error(a.err, bits);
    a.new_lens[s] = e.ok ? e.k : e.L;
  }
  int32_t* kept = a.kept + (static_cast<int64_t>(s) * a.num_kv_heads + h) * a.max_keep_len;
  for (int i = e.k + tid; i < a.max_keep_len; i += kThreads) kept[i] = -1;
  if (!e.ok) return;
  const float* W = a.key_weights +
                   (static_cast<int64_t>(e.row) * a.num_kv_heads + h) * a.max_keys;
  float* Wd = a.key_weights +
              (static_cast<int64_t>(e.dst_row) * a.num_kv_heads + h) * a.max_keys;
  const int N = e.L - e.r;   // the keys to choose from
  const int m = e.k - e.r;   // how many of them stay
  const uint32_t bins = smem_u32(hist);
  uint32_t prefix = 0;       // the m-th largest order key, digit by digit
  int need = m;              // how many keys with the prefix so far are kept
  if (m > 0 && m < N) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int nbits = pass == 2 ? 10 : 11;
      for (int i = tid; i < 2048; i += kThreads) hist[i] = 0;
      __syncthreads();
      auto count = [&](uint32_t u) {
        inc_shared_if((u >> (shift + nbits)) == prefix,
                      bins + 4 * ((u >> shift) & ((1u << nbits) - 1)));
      };
      if (pass == 0) {
#pragma unroll 4
        for (int j = tid; j < e.L; j += kThreads) {
          const uint32_t u = order_key(W[j]);
          if (j < cached) s_key[j] = u;
          inc_shared_if(j < N, bins + 4 * (u >> 21));
        }
      } else {
        const int quads = min(cached, N) / 4;
        for (int j = tid; j < quads; j += kThreads) {
          const uint4 u = reinterpret_cast<const uint4*>(s_key)[j];
          count(u.x); count(u.y); count(u.z); count(u.w);
        }
        for (int j = 4 * quads + tid; j < N; j += kThreads)
          count(j < cached ? s_key[j] : order_key(W[j]));
      }
      __syncthreads();
      // the digit at which the count from the top reaches `need`: a thread sums kBins bins from
      // the top, then a scan over the CTA
      int c[kBins], sum = 0;
#pragma unroll
      for (int i = 0; i < kBins; ++i) {
        c[i] = hist[2047 - (kBins * tid + i)];
        sum += c[i];
      }
      int x = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      int all;
      int before = warps_exclusive<kWarps>(__shfl_sync(0xffffffffu, x, 31), slots[pass & 1], &all) +
                   x - sum;
#pragma unroll
      for (int i = 0; i < kBins; ++i) {
        if (before < need && need <= before + c[i]) {
          s_digit = 2047 - (kBins * tid + i);
          s_above = before;
        }
        before += c[i];
      }
      __syncthreads();
      prefix = (prefix << nbits) | static_cast<uint32_t>(s_digit);
      need -= s_above;
    }
  }
  // Kept: order key above `prefix`, the first `need` equal to it, and the last r.  (No weight has
  // the order keys 0 and 2^32 - 1.)
  const int keys = m > 0 && m < N ? min(cached, e.L) : 0;  // order keys in shared memory
  if (m == N) prefix = 0;
  if (m == 0) prefix = 0xffffffffu;
  // The kept positions take the places of the order keys, which lie at or above them and were read
  // in this round or one before, and go out from there; if the row does not fit, they go out at
  // once.
  const bool fits = e.L <= cached;
  int done = 0, done_eq = 0;  // kept so far; equals so far
  for (int base = 0, round = 0; base < e.L; base += kThreads * kSelPer, ++round) {
    const int j0 = base + tid * kSelPer;
    uint32_t u[kSelPer];
    if (j0 + kSelPer <= keys) {
#pragma unroll
      for (int i = 0; i < kSelPer; i += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(s_key + j0 + i);
        u[i] = x.x; u[i + 1] = x.y; u[i + 2] = x.z; u[i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kSelPer; ++i) u[i] = j0 + i < N ? order_key(W[j0 + i]) : 0u;
    }
    unsigned gt = 0, eq = 0;  // bit i: position j0 + i
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      gt |= (u[i] > prefix ? 1u : 0u) << i;
      eq |= (u[i] == prefix ? 1u : 0u) << i;
    }
    const unsigned in = (1u << max(0, min(kSelPer, N - j0))) - 1;     // to choose from
    const unsigned there = (1u << max(0, min(kSelPer, e.L - j0))) - 1;
    gt = (gt & in) | (there & ~in);
    eq &= in;
    // counts of both in one word: a round has at most 2^13 positions
    const int mine = __popc(gt) | __popc(eq) << 16;
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    int all;
    // (the barrier in it: every key of the round is read; slots alternate, so their readers of two
    // rounds before are done)
    const int before =
        warps_exclusive<kWarps>(__shfl_sync(0xffffffffu, x, 31), slots[round & 1], &all) + x - mine;
    // place of a kept key: those kept before it, done + (above since `base`) + (equals kept
    // since `base`)
    const int eq_kept0 = min(done_eq, need);
    const int rank_eq = (before >> 16) + done_eq;
    int to = done + (before & 0xffff) + min(rank_eq, need) - eq_kept0;
    for (int more = __popc(eq) - max(0, need - rank_eq); more > 0; --more)
      eq &= ~(0x80000000u >> __clz(eq));  // (equals beyond `need`)
    for (unsigned stay = gt | eq; stay; stay &= stay - 1, ++to) {
      const int j = j0 + __ffs(stay) - 1;
      if (fits) s_key[to] = j;
      else kept[to] = j;
    }
    done += (all & 0xffff) + min(done_eq + (all >> 16), need) - eq_kept0;
    done_eq += all >> 16;
  }
  __syncthreads();
  // their weights: what a round reads lies at or above what it writes, and above what the rounds
  // before have written
  for (int base = 0; base < e.k; base += kThreads * kSelPer) {
    float w[kSelPer];
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const int to = base + i * kThreads + tid;
      if (to >= e.k) break;
      const int j = fits ? static_cast<int>(s_key[to]) : kept[to];
      if (fits) kept[to] = j;
      w[i] = W[j];
    }
    __syncthreads();  // every weight of the round is read
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const int to = base + i * kThreads + tid;
      if (to < e.k) Wd[to] = w[i];
    }
  }
  __syncthreads();  // every weight is read
  for (int i = e.k + tid; i < e.L; i += kThreads) Wd[i] = 0.f;
}

constexpr int kMoveThreads = 256;
constexpr int kMovePer = 4;  // 16-byte pieces of a thread in a batch

// vec: 16-byte pieces of a row's slice.  MXFP4 rows (kNB > 0) also have kNB scale bytes, which the
// threads with the row's first piece move.
template <int kNB>
__global__ void __launch_bounds__(kMoveThreads, 4) move_kernel(const EvictArgs a, int row_bytes,
                                                            int slices, int vec_log2) {
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
  const int vec = 1 << vec_log2;
  const int rows = (kMoveThreads * kMovePer) >> vec_log2;  // rows of a batch
  const int c = threadIdx.x & (vec - 1);                   // this thread's piece of its rows
  const int col = (slice * vec + c) * 16;
  const int my_row = threadIdx.x >> vec_log2, row_step = kMoveThreads >> vec_log2;
  // a row of the pool ((block, kv head) tile x slot) as a byte offset
  auto offset = [&](int32_t row) {
    if constexpr (kNB == 0) return static_cast<int64_t>(row) * row_bytes;
    return static_cast<int64_t>(row >> 4) * (kBlockSize * (row_bytes + kNB)) + (row & 15) * row_bytes;
  };
  auto scales = [&](int32_t row) {
    return pool + static_cast<int64_t>(row >> 4) * (kBlockSize * (row_bytes + kNB)) +
           kBlockSize * row_bytes + (row & 15) * kNB;
  };
  // Of a batch, in three steps that each wait on the one before, so each runs an iteration ahead
  // of the next: the kept positions, the table entries, the rows themselves.
  int32_t j_of[kMovePer], from_b[kMovePer], to_b[kMovePer];
  int32_t from[kMovePer], to[kMovePer];  // pool rows (fewer than 2^31); -1: none
  uint4 x[kMovePer];
  uint32_t sc[kMovePer];
  auto positions = [&](int first) {
#pragma unroll
    for (int i = 0; i < kMovePer; ++i) {
      const int at = first + my_row + i * row_step;
      j_of[i] = at < e.k ? kept[at] : -1;
    }
  };
  int32_t j_in[kMovePer];  // positions of the entries in from_b / to_b
  auto entries = [&](int first) {
#pragma unroll
    for (int i = 0; i < kMovePer; ++i) {
      const int at = first + my_row + i * row_step;
      j_in[i] = j_of[i];
      if (j_in[i] >= 0) {
        from_b[i] = __ldg(src_t + j_in[i] / kBlockSize);
        to_b[i] = __ldg(dst_t + at / kBlockSize);
      }
    }
  };
  auto rows_of = [&](int first) {
#pragma unroll
    for (int i = 0; i < kMovePer; ++i) {
      const int at = first + my_row + i * row_step;
      from[i] = to[i] = -1;
      if (j_in[i] < 0) continue;
      if (from_b[i] < 0 || from_b[i] >= a.num_blocks || to_b[i] < 0 || to_b[i] >= a.num_blocks) {
        set_error(a.err, PA_DEVERR_BLOCK_ID);
      } else if (from_b[i] != to_b[i] || j_in[i] % kBlockSize != at % kBlockSize) {
        from[i] = (from_b[i] * a.num_kv_heads + h) * kBlockSize + j_in[i] % kBlockSize;
        to[i] = (to_b[i] * a.num_kv_heads + h) * kBlockSize + at % kBlockSize;
      }
    }
  };
  positions(0);
  entries(0);
  positions(rows);
  for (int first = 0; first < e.k; first += rows) {
    rows_of(first);
#pragma unroll
    for (int i = 0; i < kMovePer; ++i) {
      if (from[i] < 0) continue;
      x[i] = *reinterpret_cast<const uint4*>(pool + offset(from[i]) + col);
      if (kNB == 4 && col == 0) sc[i] = *reinterpret_cast<const uint32_t*>(scales(from[i]));
      if (kNB == 2 && col == 0) sc[i] = *reinterpret_cast<const uint16_t*>(scales(from[i]));
    }
    entries(first + rows);
    positions(first + 2 * rows);
    __syncthreads();  // everyone has loaded the batch
#pragma unroll
    for (int i = 0; i < kMovePer; ++i) {
      if (to[i] < 0) continue;
      *reinterpret_cast<uint4*>(pool + offset(to[i]) + col) = x[i];
      if (kNB == 4 && col == 0) *reinterpret_cast<uint32_t*>(scales(to[i])) = sc[i];
      if (kNB == 2 && col == 0)
        *reinterpret_cast<uint16_t*>(scales(to[i])) = static_cast<uint16_t>(sc[i]);
    }
  }
}

template <int kThreads>
cudaError_t run_select(const EvictArgs& a, int64_t pairs, cudaStream_t stream) {
  // order keys of as many positions as shared memory holds
  const int cached = std::min(a.max_context_len, 50 * 1024);
  LaunchInfo li;
  cudaError_t e = launch_info(select_kernel<kThreads>, kThreads, 50 * 1024 * 4, &li);
  if (e != cudaSuccess) return e;
  return launch_dependent(select_kernel<kThreads>, dim3(static_cast<unsigned>(pairs)),
                          dim3(kThreads), cached * 4, stream, a, cached);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  const int row_bytes = a.cache_dtype == PA_MXFP4 ? a.head_dim / 2
                        : a.cache_dtype == PA_FP8_E4M3 ? a.head_dim : 2 * a.head_dim;
  const int64_t ctas = 2 * pairs;
  if (4 * ctas > INT32_MAX) return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  // A pass over short rows costs mostly what every warp does once (bins, scans), so few warps a CTA
  // and many CTAs; few rows want the CTA's time short, and of long ones shared memory holds few.
  // With 128, 512 and 1,024 threads: 2,048 rows of 4,096 weights 49, 57 and 106 us, of 16,384 227,
  // 133 and 197; 1,216 of 32,768 565, 232 and 180; 128 rows of 4,096 14, 10 and 10, of 16,384 33,
  // 17 and 14.
  const bool few = pairs <= 2 * int64_t(sms);
  e = a.max_context_len > (few ? 4096 : 16384)   ? run_select<1024>(a, pairs, stream)
      : few || a.max_context_len > 4096          ? run_select<512>(a, pairs, stream)
                                                 : run_select<128>(a, pairs, stream);
  if (e != cudaSuccess || a.max_keep_len == 0) return e;
  // Batches of a (sequence, kv head, K or V) go one after another, but columns are independent:
  // few of them are cut into slices of at least 64 bytes, while they all are resident at once.
  int slices = 1, vec_log2 = 0;
  while ((16 << vec_log2) < row_bytes) ++vec_log2;
  while (ctas * slices * 2 <= 4 * int64_t(sms) && vec_log2 > 2) {
    slices *= 2;
    --vec_log2;
  }
  auto kern = a.cache_dtype != PA_MXFP4 ? move_kernel<0>
              : a.head_dim == 128       ? move_kernel<4> : move_kernel<2>;
  return launch_dependent(kern, dim3(static_cast<unsigned>(ctas * slices)), dim3(kMoveThreads), 0,
                          stream, a, row_bytes, slices, vec_log2);
}

}  // namespace pa
