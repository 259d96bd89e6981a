// Slot-mapped cache append ("Serving LLMs with vLLM: Continuous Batching and PagedAttention
// Explained", section "Growing During Decode": each step appends the new token into the last
// block of its sequence; "Blocks and Block Tables": blocks are fixed-size and found through the
// table, which the caller folds into slot = block * block_size + offset).
//
// One thread moves 8 elements (16 bytes of bf16 input) of one (token, kv head) row for both K
// and V: coalesced 16-byte loads, 16-byte (bf16) or 8-byte (E4M3) stores into
// cache[slot / bs][head][slot % bs][:].  HBM- or launch-bound; no shared memory.
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

// MXFP4 append.  A block of 32 dims is shared by the scale 2^e with e = floor(log2 max |x|) - 2
// (the exponent of 4, the largest power of two of E2M1), at least -127; a code is x * 2^-e, exact
// in fp32, rounded to nearest even and saturated at 6.  A block that holds a NaN gets the NaN
// scale and zero codes.  Four neighbouring threads have a block: 8 dims each, as in the kernel
// above, and the block's maximum by two exchanges.
template <int NB>
__global__ void __launch_bounds__(256) cache_append_mx_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v, const int64_t* __restrict__ slots,
    int32_t num_tokens, int32_t num_kv_heads, int64_t total_slots, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache, uint32_t* __restrict__ err) {
  constexpr int VEC = 4 * NB;  // threads of a row
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t gid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t row = gid / VEC;  // (token, kv head)
  const int c = static_cast<int>(gid - row * VEC);
  if (row >= static_cast<int64_t>(num_tokens) * num_kv_heads) return;
  const int64_t t = row / num_kv_heads;
  const int64_t h = row - t * num_kv_heads;
  const int64_t slot = __ldg(slots + t);
  if (slot < 0) return;
  if (slot >= total_slots) {
    if (c == 0 && h == 0) set_error(err, PA_DEVERR_SLOT);
    return;
  }
  const uint32_t quad_mask = 0xfu << (threadIdx.x & 28);  // the block's threads leave together
  const int64_t blk = slot / kBlockSize;
  const int off = static_cast<int>(slot - blk * kBlockSize);
  const int64_t tile = (blk * num_kv_heads + h) * (NB * 32 * 17 / 2);
  const int b = c >> 2;
  auto quantise = [&](uint4 x, uint8_t* pool) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;  // largest |x| of the block as bf16 bits
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    top = max(top, __shfl_xor_sync(quad_mask, top, 1));
    top = max(top, __shfl_xor_sync(quad_mask, top, 2));
    const bool nan = top > 0x7f80u;
    const uint32_t byte = nan ? 255u : max(static_cast<int>(top >> 7) - 2, 0);
    const float up = nan ? 0.f : __uint_as_float((254u - byte) << 23);
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      codes |= f32x2_to_e2m1x2(bf16lo_to_f32(w[i]) * up, bf16hi_to_f32(w[i]) * up) << (8 * i);
    if (nan) codes = 0;
    uint16_t* dst = reinterpret_cast<uint16_t*>(pool + tile + off * (16 * NB));
    const int g = 2 * (c & 3);
    dst[g * NB + b] = static_cast<uint16_t>(codes);
    dst[(g + 1) * NB + b] = static_cast<uint16_t>(codes >> 16);
    if ((c & 3) == 0) pool[tile + kBlockSize * 16 * NB + off * NB + b] = static_cast<uint8_t>(byte);
  };
  quantise(__ldg(k + gid), k_cache);
  quantise(__ldg(v + gid), v_cache);
}

// Reads slots back: [num_tokens][num_kv_heads][D] of the values the pool holds, rounded once to
// the output type (exact for bf16 and MXFP4 pools).  One thread has 8 dims of K and V.
enum class PoolKind { kBf16, kE4m3, kMx };
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
    } else {
      const int nb = head_dim / 32, b = c >> 2, g = 2 * (c & 3);
      const uint8_t* t0 = pool + tile * (head_dim * 17 / 2);
      const uint16_t* src = reinterpret_cast<const uint16_t*>(t0 + off * (head_dim / 2));
      const uint32_t codes = src[g * nb + b] | (static_cast<uint32_t>(src[(g + 1) * nb + b]) << 16);
      const float s = e8m0_to_f32(t0[kBlockSize * (head_dim / 2) + off * nb + b], 0);
      uint32_t f[4];
      e2m1x8_to_f16x2x4(codes, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
        x[2 * i] = y.x * s;
        x[2 * i + 1] = y.y * s;
      }
    }
  };
  auto store = [&](const float (&x)[8], void* out) {
    if constexpr (kOutBf16) {
      reinterpret_cast<uint4*>(out)[gid] =
          make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                     pack_bf16x2(x[6], x[7]));
    } else {
      float4* o = reinterpret_cast<float4*>(out) + 2 * gid;
      o[0] = make_float4(x[0], x[1], x[2], x[3]);
      o[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  };
  float kx[8] = {}, vx[8] = {};
  if (ok) {
    load(k_cache, k_scale, kx);
    load(v_cache, v_scale, vx);
  }
  store(kx, k_out);
  store(vx, v_out);
}

cudaError_t launch_cache_read(const int64_t* slots, int32_t num_tokens, const void* k_cache,
                              const void* v_cache, const pa_cache_desc& c, void* k_out,
                              void* v_out, bool out_bf16, uint32_t* err, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(num_tokens) * c.num_kv_heads * (c.head_dim / 8);
  const int64_t grid = (threads + 255) / 256;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const int64_t total_slots = static_cast<int64_t>(c.num_blocks) * c.block_size;
  auto kern = c.cache_dtype == PA_BF16
                  ? (out_bf16 ? cache_read_kernel<PoolKind::kBf16, true>
                              : cache_read_kernel<PoolKind::kBf16, false>)
              : c.cache_dtype == PA_FP8_E4M3
                  ? (out_bf16 ? cache_read_kernel<PoolKind::kE4m3, true>
                              : cache_read_kernel<PoolKind::kE4m3, false>)
                  : (out_bf16 ? cache_read_kernel<PoolKind::kMx, true>
                              : cache_read_kernel<PoolKind::kMx, false>);
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
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch_dependent(c.head_dim == 128 ? cache_append_mx_kernel<4> : cache_append_mx_kernel<2>,
                            dim3(static_cast<unsigned>(grid)), dim3(block), 0, stream,
                            static_cast<const uint4*>(k), static_cast<const uint4*>(v), slots,
                            num_tokens, c.num_kv_heads, total_slots,
                            static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), err);
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
