// Slot-mapped cache append ("Serving LLMs with vLLM: Continuous Batching and PagedAttention
// Explained", section "Growing During Decode": each step appends the new token into the last
// block of its sequence; "Blocks and Block Tables": blocks are fixed-size and found through the
// table, which the caller folds into slot = block * block_size + offset).
//
// One thread moves 8 elements (16 bytes of bf16 input) of one (token, kv head) row for both K
// and V: coalesced 16-byte loads, 16-byte (bf16) or 8-byte (E4M3) stores into
// cache[slot / bs][head][slot % bs][:].  HBM- or launch-bound; no shared memory.
#include <algorithm>
#include <climits>

#include "mxfp4.cuh"
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

template <bool kFp8>
__global__ void __launch_bounds__(256) cache_append_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v, const int64_t* __restrict__ slots,
    int32_t num_tokens, int32_t num_kv_heads, int32_t vec_per_row, int64_t total_slots,
    void* __restrict__ k_cache, void* __restrict__ v_cache, float k_scale, float v_scale,
    uint32_t* __restrict__ err) {
  grid_dependency_wait();    // launched early (programmatic dependent launch): inputs ready
  grid_launch_dependents();  // the step's plan kernel may launch meanwhile
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t per_token = static_cast<int64_t>(num_kv_heads) * vec_per_row;
  if (gid >= per_token * num_tokens) return;
  const int32_t t = static_cast<int32_t>(gid / per_token);
  const int64_t within = gid - static_cast<int64_t>(t) * per_token;  // head * vec + vec index
  const int32_t h = static_cast<int32_t>(within / vec_per_row);
  const int32_t c = static_cast<int32_t>(within - static_cast<int64_t>(h) * vec_per_row);
  const int64_t slot = __ldg(slots + t);
  if (slot < 0) return;
  if (slot >= total_slots) {
    if (c == 0 && h == 0) set_error(err, PA_DEVERR_SLOT);
    return;
  }
  const int64_t blk = slot / kBlockSize;
  const int64_t off = slot - blk * kBlockSize;
  // destination row (blk, h, off) of a [NB][Hkv][bs][D] pool, in 8-element units
  const int64_t row = (blk * num_kv_heads + h) * kBlockSize + off;
  const int64_t dst = row * vec_per_row + c;
  const uint4 kv = __ldg(k + gid);
  const uint4 vv = __ldg(v + gid);
  if constexpr (!kFp8) {
    reinterpret_cast<uint4*>(k_cache)[dst] = kv;
    reinterpret_cast<uint4*>(v_cache)[dst] = vv;
  } else {
    auto quant = [](uint4 x, float s) {
      // fl32(x) / s rounded to nearest (IEEE division), then E4M3 round-to-nearest-even with
      // saturation to +-448.
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t out[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint16_t lo = f32x2_to_e4m3x2(__fdiv_rn(bf16lo_to_f32(w[2 * i]), s),
                                            __fdiv_rn(bf16hi_to_f32(w[2 * i]), s));
        const uint16_t hi = f32x2_to_e4m3x2(__fdiv_rn(bf16lo_to_f32(w[2 * i + 1]), s),
                                            __fdiv_rn(bf16hi_to_f32(w[2 * i + 1]), s));
        out[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
      }
      return make_uint2(out[0], out[1]);
    };
    reinterpret_cast<uint2*>(k_cache)[dst] = quant(kv, k_scale);
    reinterpret_cast<uint2*>(v_cache)[dst] = quant(vv, v_scale);
  }
}

// Division of 0 <= n < 2^31 by a fixed d (Granlund and Montgomery's division by invariant integers):
// (n + high word of n * mul) >> shift, with 2^shift the next power of two from d and mul = floor(2^32
// (2^shift - d) / d) + 1.  (A 64-bit division by a run-time
// value took more instructions than all else that a thread of these kernels does.)
struct FastDiv {
  uint32_t d, mul, shift;
  explicit FastDiv(uint32_t div) : d(div), mul(0), shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return (__umulhi(n, mul) + n) >> shift;
  }
};

// Between a thread's dims and a pool row's words.  The four threads of a scale block have 8 dims each
// (two 16-bit words), and the words of the row's NB blocks are interleaved: thread (b, q) of a row
// (block b, quarter q) has words e = 0, 1 of K and of V for block b, and stores or loads the 8 bytes
// that hold word (e', b') of one of them for all blocks.  NB = 4: a 4 x 4 transpose of 16-bit items
// over the lanes b (lane bits 2 and 3), in two exchanges, which is its own inverse.  NB = 2: one.
// kBack: from the row's words to the thread's dims.
template <int NB, bool kBack>
__device__ __forceinline__ void mx_exchange(unsigned mask, int lane, uint32_t& k, uint32_t& v) {
  if constexpr (NB == 2 && kBack) {
    const bool up = (lane >> 2) & 1;  // has V's words, and takes block 1
    const uint32_t mine = prmt(k, v, up ? 0x7632u : 0x5410u);
    const uint32_t got = __shfl_xor_sync(mask, prmt(k, v, up ? 0x5410u : 0x7632u), 4);
    k = up ? got : mine;
    v = up ? mine : got;
    return;
  }
  const bool upper = (lane >> (NB == 4 ? 3 : 2)) & 1;  // takes V
  const uint32_t keep = upper ? v : k;
  const uint32_t got = __shfl_xor_sync(mask, upper ? k : v, NB == 4 ? 8 : 4);
  if constexpr (NB == 4) {
    const bool odd = (lane >> 2) & 1;                  // takes the second words
    const uint32_t mine = prmt(keep, got, odd ? 0x7632u : 0x5410u);
    const uint32_t other =
        __shfl_xor_sync(mask, prmt(keep, got, odd ? 0x5410u : 0x7632u), 4);
    const uint32_t first = odd ? other : mine, second = odd ? mine : other;
    const uint32_t lo = prmt(first, second, 0x5410u), hi = prmt(first, second, 0x7632u);
    k = upper ? hi : lo;
    v = upper ? lo : hi;
  } else {
    const uint32_t first = upper ? got : keep, second = upper ? keep : got;
    k = prmt(first, second, 0x5410u);
    v = prmt(first, second, 0x7632u);
  }
}
// Byte of a row, of K (`upper` false) or V, that the thread's 8 bytes begin at.
template <int NB>
__device__ __forceinline__ int mx_piece(int lane, bool* upper) {
  const int q = lane & 3, b = (lane >> 2) & (NB - 1);
  *upper = b >= NB / 2;
  return NB == 4 ? (2 * q + (b & 1)) * 8 : q * 8;
}

// MXFP4 append.  A block of 32 dims is shared by the scale 2^e with e = floor(log2 max |x|) - 2
// (the exponent of 4, the largest power of two of E2M1), at least -127; a code is x * 2^-e, exact
// in fp32, rounded to nearest even and saturated at 6.  A block that holds a NaN gets the NaN
// scale and zero codes.  A thread quantises 8 dims of K and of V, finds the block's maximum with
// its three neighbours by two exchanges, and stores 8 bytes of a row of one of them.  Bound by HBM,
// with the ALU close behind: 8,191 tokens x 32 heads of 128 dims in 32 us (170 MB, 5.3 TB/s), the
// read back in 31 us.
template <int NB>
__global__ void __launch_bounds__(256) cache_append_mx_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v, const int64_t* __restrict__ slots,
    uint32_t rows, FastDiv heads, int64_t total_slots, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache, uint32_t* __restrict__ err) {
  constexpr int VEC = 4 * NB;  // threads of a row
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t row = blockIdx.x * (256 / VEC) + threadIdx.x / VEC;  // (token, kv head)
  if (row >= rows) return;
  const int64_t gid = static_cast<int64_t>(row) * VEC + threadIdx.x % VEC;
  const uint32_t t = heads(row), h = row - t * heads.d;
  const int lane = threadIdx.x & 31;
  const uint4 kx = __ldg(k + gid), vx = __ldg(v + gid);
  const int64_t slot = __ldg(slots + t);
  if (slot < 0) return;
  if (slot >= total_slots) {
    if (threadIdx.x % VEC == 0 && h == 0) set_error(err, PA_DEVERR_SLOT);
    return;
  }
  // a row's threads leave together: exchanges stay within its lanes
  const unsigned row_mask = ((1u << VEC) - 1u) << (lane & ~(VEC - 1));
  const uint32_t blk = static_cast<uint32_t>(slot / kBlockSize);  // (the pool's rows fit in 31 bits)
  const int off = static_cast<int>(slot % kBlockSize);
  const int64_t tile = static_cast<int64_t>(blk * heads.d + h) * (NB * 32 * 17 / 2);
  auto quantise = [&](uint4 x, uint32_t& byte) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    // largest |x| of the block as bf16 bits, two halves at a time
    uint32_t top2 = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 4; ++i) top2 = __vmaxu2(top2, w[i] & 0x7fff7fffu);
    top2 = __vmaxu2(top2, __shfl_xor_sync(row_mask, top2, 1));
    top2 = __vmaxu2(top2, __shfl_xor_sync(row_mask, top2, 2));
    const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
    const bool nan = top > 0x7f80u;
    byte = nan ? 255u : max(static_cast<int>(top >> 7) - 2, 0);
    const float up = nan ? 0.f : __uint_as_float((254u - byte) << 23);
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = bf16lo_to_f32(w[i]) * up;
      y[2 * i + 1] = bf16hi_to_f32(w[i]) * up;
    }
    const uint32_t codes = f32x8_to_e2m1x8(y);
    return nan ? 0u : codes;
  };
  uint32_t k_byte, v_byte;
  uint32_t w0 = quantise(kx, k_byte), w1 = quantise(vx, v_byte);
  mx_exchange<NB, false>(row_mask, lane, w0, w1);
  bool upper;
  const int at = mx_piece<NB>(lane, &upper);
  *reinterpret_cast<uint2*>((upper ? v_cache : k_cache) + tile + off * (16 * NB) + at) =
      make_uint2(w0, w1);
  const int q = lane & 3;
  if (q < 2)  // the block's scale bytes: K's by its first thread, V's by its second
    ((q ? v_cache : k_cache) + tile)[kBlockSize * 16 * NB + off * NB + ((lane >> 2) & (NB - 1))] =
        static_cast<uint8_t>(q ? v_byte : k_byte);
}

// Reads slots back: [num_tokens][num_kv_heads][D] of the values the pool holds, rounded once to
// the output type (exact for bf16 and MXFP4 pools).  One thread has 8 dims of K and V.
enum class PoolKind { kBf16, kE4m3 };
template <bool kOutBf16>
__device__ __forceinline__ void store_row_piece(const float (&x)[8], void* out, int64_t at) {
  if constexpr (kOutBf16) {
    reinterpret_cast<uint4*>(out)[at] =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
  } else {
    float4* o = reinterpret_cast<float4*>(out) + 2 * at;
    o[0] = make_float4(x[0], x[1], x[2], x[3]);
    o[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// From an MXFP4 pool: the append's exchange backwards.
template <int NB, bool kOutBf16>
__global__ void __launch_bounds__(256) cache_read_mx_kernel(
    const int64_t* __restrict__ slots, uint32_t rows, FastDiv heads, int64_t total_slots,
    const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
    void* __restrict__ k_out, void* __restrict__ v_out, uint32_t* __restrict__ err) {
  constexpr int VEC = 4 * NB;
  grid_dependency_wait();
  const uint32_t row = blockIdx.x * (256 / VEC) + threadIdx.x / VEC;
  if (row >= rows) return;
  const int64_t gid = static_cast<int64_t>(row) * VEC + threadIdx.x % VEC;
  const uint32_t t = heads(row), h = row - t * heads.d;
  const int lane = threadIdx.x & 31;
  const int64_t slot = __ldg(slots + t);
  const bool ok = slot >= 0 && slot < total_slots;
  if (slot >= total_slots && threadIdx.x % VEC == 0 && h == 0) set_error(err, PA_DEVERR_SLOT);
  float kx[8] = {}, vx[8] = {};
  if (ok) {  // (a row's threads take the same way)
    const unsigned row_mask = ((1u << VEC) - 1u) << (lane & ~(VEC - 1));
    const uint32_t blk = static_cast<uint32_t>(slot / kBlockSize);
    const int off = static_cast<int>(slot % kBlockSize);
    const int64_t tile = static_cast<int64_t>(blk * heads.d + h) * (NB * 32 * 17 / 2);
    const int64_t scale_at = tile + kBlockSize * 16 * NB + off * NB + ((lane >> 2) & (NB - 1));
    const float ks = e8m0_to_f32(__ldg(k_cache + scale_at));
    const float vs = e8m0_to_f32(__ldg(v_cache + scale_at));
    bool upper;
    const int at = mx_piece<NB>(lane, &upper);
    uint2 w = __ldg(reinterpret_cast<const uint2*>((upper ? v_cache : k_cache) + tile +
                                                   off * (16 * NB) + at));
    mx_exchange<NB, true>(row_mask, lane, w.x, w.y);
    auto decode = [](uint32_t codes, float s, float (&x)[8]) {
      uint32_t f[4];
      e2m1x8_to_f16x2x4(codes, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
        x[2 * i] = y.x * s;
        x[2 * i + 1] = y.y * s;
      }
    };
    decode(w.x, ks, kx);
    decode(w.y, vs, vx);
  }
  store_row_piece<kOutBf16>(kx, k_out, gid);
  store_row_piece<kOutBf16>(vx, v_out, gid);
}

template <PoolKind kKind, bool kOutBf16>
__global__ void __launch_bounds__(256) cache_read_kernel(
    const int64_t* __restrict__ slots, int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
    int64_t total_slots, const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
    float k_scale, float v_scale, void* __restrict__ k_out, void* __restrict__ v_out,
    uint32_t* __restrict__ err) {
  grid_dependency_wait();
  const int32_t vec = head_dim / 8;
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t row = gid / vec;
  const int c = static_cast<int>(gid - row * vec);
  if (row >= static_cast<int64_t>(num_tokens) * num_kv_heads) return;
  const int64_t t = row / num_kv_heads;
  const int64_t h = row - t * num_kv_heads;
  const int64_t slot = __ldg(slots + t);
  const bool ok = slot >= 0 && slot < total_slots;
  if (slot >= total_slots && c == 0 && h == 0) set_error(err, PA_DEVERR_SLOT);
  const int64_t blk = ok ? slot / kBlockSize : 0;
  const int off = ok ? static_cast<int>(slot - blk * kBlockSize) : 0;
  const int64_t tile = blk * num_kv_heads + h;
  auto load = [&](const uint8_t* pool, float scale, float (&x)[8]) {
    if constexpr (kKind == PoolKind::kBf16) {
      const uint4 w = *reinterpret_cast<const uint4*>(
          pool + ((tile * kBlockSize + off) * head_dim + 8 * c) * 2);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo_to_f32(u[i]);
        x[2 * i + 1] = bf16hi_to_f32(u[i]);
      }
    } else if constexpr (kKind == PoolKind::kE4m3) {
      const uint2 w = *reinterpret_cast<const uint2*>(
          pool + (tile * kBlockSize + off) * head_dim + 8 * c);
      const uint32_t u[2] = {w.x, w.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e4m3x2_to_f32x2(static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1))), x[2 * i], x[2 * i + 1]);
        x[2 * i] *= scale;
        x[2 * i + 1] *= scale;
      }
    }
  };
  float kx[8] = {}, vx[8] = {};
  if (ok) {
    load(k_cache, k_scale, kx);
    load(v_cache, v_scale, vx);
  }
  store_row_piece<kOutBf16>(kx, k_out, gid);
  store_row_piece<kOutBf16>(vx, v_out, gid);
}

// Calls launch(first token, rows) for pieces of at most 2^28 rows of (token, kv head).
template <typename F>
static cudaError_t by_rows(int32_t num_tokens, int32_t num_kv_heads, F launch) {
  const int64_t step = std::max<int64_t>(1, (int64_t(1) << 28) / num_kv_heads);
  cudaError_t e = cudaSuccess;
  for (int64_t t0 = 0; t0 < num_tokens && e == cudaSuccess; t0 += step)
    e = launch(t0, static_cast<uint32_t>(std::min<int64_t>(step, num_tokens - t0) * num_kv_heads));
  return e;
}

cudaError_t launch_cache_read(const int64_t* slots, int32_t num_tokens, const void* k_cache,
                              const void* v_cache, const pa_cache_desc& c, void* k_out,
                              void* v_out, bool out_bf16, uint32_t* err, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(num_tokens) * c.num_kv_heads * (c.head_dim / 8);
  const int64_t grid = (threads + 255) / 256;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const int64_t total_slots = static_cast<int64_t>(c.num_blocks) * c.block_size;
  if (c.cache_dtype == PA_MXFP4) {
    auto kern = c.head_dim == 128
                    ? (out_bf16 ? cache_read_mx_kernel<4, true> : cache_read_mx_kernel<4, false>)
                    : (out_bf16 ? cache_read_mx_kernel<2, true> : cache_read_mx_kernel<2, false>);
    const int64_t row_bytes = int64_t(c.head_dim) * (out_bf16 ? 2 : 4);
    return by_rows(num_tokens, c.num_kv_heads, [&](int64_t t0, uint32_t rows) {
      const int64_t at = t0 * c.num_kv_heads * row_bytes;
      return launch_dependent(kern, dim3((rows * int64_t(c.head_dim / 8) + 255) / 256), dim3(256), 0,
                              stream, slots + t0, rows, FastDiv(c.num_kv_heads), total_slots,
                              static_cast<const uint8_t*>(k_cache),
                              static_cast<const uint8_t*>(v_cache),
                              static_cast<void*>(static_cast<uint8_t*>(k_out) + at),
                              static_cast<void*>(static_cast<uint8_t*>(v_out) + at), err);
    });
  }
  auto kern = c.cache_dtype == PA_BF16
                  ? (out_bf16 ? cache_read_kernel<PoolKind::kBf16, true>
                              : cache_read_kernel<PoolKind::kBf16, false>)
                  : (out_bf16 ? cache_read_kernel<PoolKind::kE4m3, true>
                              : cache_read_kernel<PoolKind::kE4m3, false>);
  return launch_dependent(kern, dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, slots,
                          num_tokens, c.num_kv_heads, c.head_dim, total_slots,
                          static_cast<const uint8_t*>(k_cache),
                          static_cast<const uint8_t*>(v_cache), c.k_scale, c.v_scale, k_out, v_out,
                          err);
}

cudaError_t launch_cache_append(const void* k, const void* v, const int64_t* slots,
                                int32_t num_tokens, void* k_cache, void* v_cache,
                                const pa_cache_desc& c, uint32_t* err, cudaStream_t stream) {
  const int32_t vec_per_row = c.head_dim / 8;
  const int64_t threads = static_cast<int64_t>(num_tokens) * c.num_kv_heads * vec_per_row;
  if (threads == 0) return cudaSuccess;
  const int block = 256;
  const int64_t grid = (threads + block - 1) / block;
  const int64_t total_slots = static_cast<int64_t>(c.num_blocks) * c.block_size;
  if (c.cache_dtype == PA_MXFP4) {
    return by_rows(num_tokens, c.num_kv_heads, [&](int64_t t0, uint32_t rows) {
      const int64_t at = t0 * c.num_kv_heads * vec_per_row;
      return launch_dependent(
          c.head_dim == 128 ? cache_append_mx_kernel<4> : cache_append_mx_kernel<2>,
          dim3((rows * int64_t(vec_per_row) + 255) / 256), dim3(256), 0, stream,
          static_cast<const uint4*>(k) + at, static_cast<const uint4*>(v) + at, slots + t0, rows,
          FastDiv(c.num_kv_heads), total_slots, static_cast<uint8_t*>(k_cache),
          static_cast<uint8_t*>(v_cache), err);
    });
  }
  if (c.cache_dtype == PA_FP8_E4M3) {
    return launch_dependent(cache_append_kernel<true>, dim3(static_cast<unsigned>(grid)),
                            dim3(block), 0, stream, static_cast<const uint4*>(k),
                            static_cast<const uint4*>(v), slots, num_tokens, c.num_kv_heads,
                            vec_per_row, total_slots, k_cache, v_cache, c.k_scale, c.v_scale,
                            err);
  }
  return launch_dependent(cache_append_kernel<false>, dim3(static_cast<unsigned>(grid)),
                          dim3(block), 0, stream, static_cast<const uint4*>(k),
                          static_cast<const uint4*>(v), slots, num_tokens, c.num_kv_heads,
                          vec_per_row, total_slots, k_cache, v_cache, 1.f, 1.f, err);
}

}  // namespace pa
