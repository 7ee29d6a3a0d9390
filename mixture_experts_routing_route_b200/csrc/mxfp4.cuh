// MXFP4 (OCP Microscaling Formats, version 1.0): blocks of 32 values share
// one power-of-two scale (E8M0, a byte s: 2^(s - 127), 255: NaN); each value
// is an E2M1 code of four bits (sign; 0, 0.5, 1, 1.5, 2, 3, 4, 6).
//
// Quantising a block with largest magnitude a: s = max(floor(log2 a) - 2 +
// 127, 0) (2 is the exponent of the largest E2M1 value), codes = v 2^(127 - s)
// rounded to the nearest E2M1 value, ties to the even code, magnitudes above 6
// to 6. The scaling is exact, so the codes depend on the inputs alone. A block
// that holds an Inf or a NaN gets s = 255 and reads back as NaN: E2M1 has
// neither, and a saturated Inf would pass for a number.
//
// Two codes to a byte, the earlier value in the low half. Scales are kept as
// the tensor cores read them: tiles of 128 rows x 4 blocks (128 values), 512
// bytes, row r and block b of a tile at byte (r % 32) * 16 + (r / 32) * 4 + b;
// the tiles of one row group lie in the order of the blocks. A weight matrix
// [N, K] has row groups n / 128. Rows sorted by expert have, for expert e, the
// groups seg[e] / 128 + e, ... (each expert's rows start a group of their own,
// whatever seg[e] is; rows_max / 128 + E groups hold them all, because
// floor((a + n) / 128) + 1 >= floor(a / 128) + ceil(n / 128)).
#pragma once
#include "common.cuh"
#include <cuda_fp16.h>

namespace moe {

constexpr int kMxBlock = 32;
constexpr int kScaleTile = 512;  // bytes of one 128-row x 4-block tile of scales

// Scale byte of a block whose largest magnitude has the fp32 bits `abs_bits`.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t abs_bits) {
  if (abs_bits >= 0x7f800000u) return 255u;
  const uint32_t ex = abs_bits >> 23;  // floor(log2) + 127; 0: zero or subnormal
  return ex > 2u ? ex - 2u : 0u;
}

// 2^(127 - s), the factor that scales a block before rounding; 0 for s = 255
// (every code is then 0, the scale alone makes the block NaN).
__device__ __forceinline__ float mx_inv_scale(uint32_t s) {
  return __uint_as_float(s == 255u ? 0u : (254u - s) << 23);
}

// 2^(s - 127); NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7fc00000u : s << 23);
}

// Eight scaled values to eight E2M1 codes, v[0] in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// One scaled value to its code.
__device__ __forceinline__ uint32_t e2m1(float v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b, z;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 z, %2, %2;\n\t"
      "mov.b32 %0, {b, z, z, z};\n\t}"
      : "=r"(r) : "f"(v), "f"(0.0f));
  return r;
}

// Eight codes (the first in the lowest four bits) to their values times f:
// through fp16, which holds every E2M1 value exactly.
__device__ __forceinline__ void e2m1x8_values(uint32_t codes, float f, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = p.x * f;
    v[2 * i + 1] = p.y * f;
  }
}

// Byte offset of the scale of (row group, row in the group, block) among
// groups of K / 128 tiles.
__host__ __device__ __forceinline__ size_t mx_scale_at(long long group, int ktiles, int row, int block) {
  return (static_cast<size_t>(group) * ktiles + (block >> 2)) * kScaleTile + (row & 31) * 16 +
         (row >> 5) * 4 + (block & 3);
}

}  // namespace moe
