// The MXFP4 element and scale codec.
#pragma once

#include <cuda_fp4.h>

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

QDEV uint32_t mx_codes(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}
// Codes of two bf16 packed in a word, scaled by f.
QDEV uint32_t mx_codes2(uint32_t w, float f) {
  const float2 v = __fmul2_rn(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)), make_float2(f, f));
  return mx_codes(v.x, v.y);
}

}  // namespace
}  // namespace qnf4
