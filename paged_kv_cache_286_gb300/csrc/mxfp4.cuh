// MXFP4 pool tiles: E2M1 codes (sign, two exponent bits, one mantissa bit: 0 .5 1 1.5 2 3 4 6) in
// blocks of 32 dims of a row that share one E8M0 scale byte e, which stands for 2^(e - 127)
// (255: NaN; the codes of such a block are zeros).
//
// One (block, kv head) tile is 16 rows of D / 2 bytes of codes, then 16 rows of D / 32 scale
// bytes: 17 D / 2 bytes, a multiple of 16.  Within a row, 16-bit word g * (D / 32) + b holds
// dims 32 b + 4 g .. 32 b + 4 g + 3, the lowest dim in the lowest four bits: four neighbouring
// words belong to the row's four scale blocks, so that a lane which loads 8 or 16 consecutive
// bytes of a row holds the same few dims of every block, as an MMA fragment per block needs.
#pragma once

#include "pa_common.cuh"

namespace pa {

template <int D>
struct Mx {
  static constexpr int kBlocks = D / 32;              // scale blocks of a row
  static constexpr int kRowBytes = D / 2;             // codes of a row
  static constexpr int kCodeBytes = kBlockSize * kRowBytes;
  static constexpr int kTileBytes = kCodeBytes + kBlockSize * kBlocks;
};

// Eight E2M1 codes to four exact f16 pairs, byte i (low nibble in the low half) to out[i].
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t w, uint32_t (&out)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(w));
}

// Eight fp32 to E2M1 codes, round to nearest even, saturating at 6: x[0] in the lowest nibble.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&x)[8]) {
  uint32_t out;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(out)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return out;
}

// Two neighbouring scale bytes (a half of the word) as a bf16 pair, exactly: byte 0 is the subnormal
// 2^-127 (codes times it are up to 1.5 * 2^-125), byte 255 NaN.
__device__ __forceinline__ uint32_t e8m0x2_to_bf16x2(uint32_t word, int half) {
  uint32_t out;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(out) : "h"(static_cast<uint16_t>(word >> (16 * half))));
  return out;
}

// One scale byte as fp32.
__device__ __forceinline__ float e8m0_to_f32(uint32_t byte) {
  return bf16lo_to_f32(e8m0x2_to_bf16x2(byte, 0));
}

// Transposes the 8 x 8 matrix of 16-bit elements that the warp holds two to a lane.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

}  // namespace pa
