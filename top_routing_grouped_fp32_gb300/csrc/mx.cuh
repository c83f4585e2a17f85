// mx.cuh -- microscaled (MX) blocks: 32 consecutive values of a row share one
// power-of-two scale, held as a biased exponent byte b (the scale is 2^(b-127);
// 255 marks a block without values: NaN).  Elements are e2m1 ("mxfp4": +-0,
// 0.5, 1, 1.5, 2, 3, 4, 6; two in a byte, the first in the low half) or e4m3
// ("mxfp8": three mantissa bits, largest value 448).
//
// With a the largest magnitude of a block, 2^p <= a < 2^(p+1), and emax the
// exponent of the largest element (2 or 8), the scale is 2^(p - emax), one step
// more where a would still be clipped by half an element step or more (from
// 1.75 2^p on for e2m1, 1.8125 2^p for e4m3).  Elements are x over the scale,
// exactly, rounded once to nearest even; nothing else is rounded.
#pragma once

#include "common.cuh"

namespace moe {
namespace mx {

constexpr int kBlock = 32;

// largest magnitude as the bits of |x|: NaN orders above inf, inf above the rest
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// scale byte of a block whose largest magnitude has the bits a
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t a) {
  constexpr int emax = FMT == MOE_MXFP4 ? 2 : 8;
  constexpr uint32_t bump = FMT == MOE_MXFP4 ? 0x600000u : 0x680000u;  // significand 1.75, 1.8125
  const int e = (int)(a >> 23);
  if (e == 255) return 255u;
  const int b = e - emax + ((a & 0x7FFFFFu) >= bump ? 1 : 0);
  return (uint32_t)max(b, 0);
}
// 1 / scale, exactly (0 for byte 255, so that its elements become 0 unless NaN)
__device__ __forceinline__ float inverse_scale(uint32_t b) {
  return b == 255u ? 0.f : __uint_as_float((254u - b) << 23);
}
__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7FC00000u : b == 0u ? 0x00400000u : b << 23);
}

// 8 scaled values -> 8 e2m1 elements
__device__ __forceinline__ uint32_t to_e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// 4 scaled values -> 4 e4m3 elements
__device__ __forceinline__ uint32_t to_e4m3x4(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
  return r;
}
// 8 e2m1 elements -> FP32 (unscaled)
__device__ __forceinline__ void from_e2m1x8(uint32_t q, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
// 4 e4m3 elements -> FP32 (unscaled)
__device__ __forceinline__ void from_e4m3x4(uint32_t q, float* v) {
  uint32_t h[2];
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(q));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// ---- scales in the order of the products ---------------------------------------
// The scale bytes of 32 rows by one span of 512 columns (16 blocks) form a
// group: 16 bytes a row, so that lane r of a warp reads row r's four words of
// four bytes at once, as tensor memory wants them (a column a word, 128 columns
// of the row each).  The groups of one span lie together, for an expert's
// weight rows and for 256 activation rows, so that a tile's scales of a span
// are contiguous; the spans follow one another.  Bytes of blocks past a row's
// end are finite scales (their elements are zero).
constexpr int kSpanCols = 512, kGroupRows = 32, kGroupBytes = 512;
constexpr int kUnitRows = 256, kUnitGroups = kUnitRows / kGroupRows;  // activations
__host__ __device__ inline int64_t spans(int64_t C) { return (C + kSpanCols - 1) / kSpanCols; }

}  // namespace mx
}  // namespace moe
