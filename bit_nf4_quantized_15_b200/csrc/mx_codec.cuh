// The MXFP4 element and scale codec.
#pragma once

#include "common.cuh"

namespace qnf4 {
namespace {

// Scale byte of a block from the largest |x| bits (Inf and NaN included: their
// exponent field is 255 and their bits compare above every finite value's).
QDEV uint32_t mx_scale_byte(uint32_t maxbits) {
  const uint32_t e = maxbits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - b): exact in fp32 for every b that a finite block has (b <= 252).
QDEV float mx_inv_scale(uint32_t b) { return __uint_as_float((254u - (b > 252u ? 127u : b)) << 23); }

// Codes of eight scaled values, element i in nibble i: nearest, ties to even,
// saturated to 6.
QDEV uint32_t mx_codes8(const float2 (&v)[4]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return w;
}
// The same for eight bf16 in four words, scaled by f here.
QDEV uint32_t mx_codes8(const uint32_t* w, float f) {
  const float2 ff = make_float2(f, f);
  float2 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = __fmul2_rn(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)), ff);
  return mx_codes8(v);
}
// Running maximum of |x| of bf16 pairs, NaN kept; the sign bits are noise.
QDEV uint32_t mx_absmax2(uint32_t m, uint32_t w) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w));
  return r;
}
// The larger of the two as fp32 bits.
QDEV uint32_t mx_absmax_bits(uint32_t m) { return max(m & 0x7FFFu, (m >> 16) & 0x7FFFu) << 16; }

}  // namespace
}  // namespace qnf4
