// Keys of E4M3 and MXFP4 pools as bf16, for kernels whose MMAs take bf16 operands.
#pragma once

#include "mxfp4.cuh"
#include "pa_common.cuh"

namespace pa {

enum class Pool { kBf16, kE4m3, kMx };

// 8 dims of a key (32 c + 8 qc ..) of an E4M3 or MXFP4 pool as bf16 pairs, exactly.
template <Pool kPool, int D>
__device__ __forceinline__ void load_dims(const uint8_t* __restrict__ k_cache, int64_t tile,
                                          int off, int c, int qc, uint32_t (&w)[4]) {
  static_assert(kPool != Pool::kBf16, "");
  constexpr int NC = D / 32;
  if constexpr (kPool == Pool::kE4m3) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(
        k_cache + (tile * kBlockSize + off) * D + 32 * c + 8 * qc));
    const uint32_t u[2] = {x.x, x.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f0, f1;
      e4m3x2_to_f32x2(static_cast<uint16_t>(u[j >> 1] >> (16 * (j & 1))), f0, f1);
      w[j] = pack_bf16x2(f0, f1);
    }
  } else {
    const uint8_t* t = k_cache + tile * Mx<D>::kTileBytes;
    const uint16_t* src = reinterpret_cast<const uint16_t*>(t + off * Mx<D>::kRowBytes);
    const uint32_t codes = __ldg(src + 2 * qc * NC + c) |
                           (static_cast<uint32_t>(__ldg(src + (2 * qc + 1) * NC + c)) << 16);
    const float sc = e8m0_to_f32(__ldg(t + Mx<D>::kCodeBytes + off * NC + c));
    uint32_t f[4];
    e2m1x8_to_f16x2x4(codes, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f[j]));
      w[j] = pack_bf16x2(y.x * sc, y.y * sc);
    }
  }
}

}  // namespace pa
