// MXFP4 blocks: 32 elements, one scale 2^(e - 127) with e = floor(log2 max|x|) - 2 + 127 (at least 0;
// 127 if all are 0; 255, a NaN, if one is no finite number), codes of x / scale rounded to the nearest
// E2M1 value, ties to the even code, saturating at 6.
//
// All of it is exact in fp32: the scale is a power of two taken from the largest element's exponent
// bits, so x * 2^(127 - e) is x with another exponent (or so small that its code is 0), and the
// conversion rounds once.
#pragma once

#include "mx.h"

namespace moe {
namespace mxq {

// Scale byte from the bits of the block's largest |x| as fp32.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int e = (int)(amax >> 23);
  return e == 255 ? 255u : amax == 0u ? 127u : (uint32_t)max(e - 2, 0);
}

// 2^(127 - s): s = 254 and 255 give a subnormal and 0 (a NaN block's codes are then 0 or a NaN's).
__device__ __forceinline__ float inverse(uint32_t s) {
  return s < 254u ? __uint_as_float((254u - s) << 23) : s == 254u ? __uint_as_float(0x00400000u) : 0.f;
}

// 2^(s - 127)
__device__ __forceinline__ float value(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7FC00000u)
         : s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
}

// Eight values -> eight E2M1 codes, element i in bits 4 i .. 4 i + 3.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n"
      "  .reg .b8 a, b, c, d;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "  mov.b32 %0, {a, b, c, d};\n"
      "}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The two values of a byte of codes (bits 0 .. 7 of b), as two f16: exact.
__device__ __forceinline__ float2 pair(uint32_t b) {
  uint32_t h;
  asm("{\n"
      "  .reg .b8 c;\n"
      "  .reg .b32 w;\n"
      "  mov.b32 {c, _, _, _}, %1;\n"
      "  cvt.rn.f16x2.e2m1x2 %0, c;\n"
      "}"
      : "=r"(h)
      : "r"(b));
  float2 f;
  asm("{ .reg .f16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi; }"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// The four lanes that hold a block's 8 elements each (a quad of lanes): its scale byte.
__device__ __forceinline__ uint32_t quad_scale(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  // NaNs lie above infinity as bits: both give 255
  return scale_byte(m);
}

__device__ __forceinline__ void bf16x8(const uint4& u, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = bf16x8_elem(u, i);
}

// The codes and the scale of eight elements of a block that a quad of lanes holds.
__device__ __forceinline__ uint32_t quantise8(float (&v)[8], uint32_t& s) {
  s = quad_scale(v);
  const float f = inverse(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= f;
  return s == 255u ? 0u : codes8(v);
}

// Place of row r's scale of 32-block j among tiles of `chunks` chunks a row of tiles.
__device__ __forceinline__ size_t tile_at(long r, int j, int chunks) {
  return ((size_t)(r >> 7) * chunks + (j >> 2)) * kMxTile + (size_t)((r & 31) * 16) +
         (size_t)(((r & 127) >> 5) * 4 + (j & 3));
}

}  // namespace mxq
}  // namespace moe
