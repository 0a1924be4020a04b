// Counter-based random bits for dropout: Philox4x32-10 (Salmon, Moraes, Dror
// and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).
//
// Element i of a tensor takes 16 bits: counter (i / 8, offset), both 64 bits
// low word first, key `seed`; of the four output words element i uses word
// (i % 8) / 2, its low half for an even i.  It is kept where those 16 bits
// are at least `threshold` = round(65536 p), so the drop probability is a
// multiple of 2^-16 and eight neighbours share one evaluation (about 50
// integer instructions): cheap enough to recompute wherever the mask is
// needed, so no mask outlives a call.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace qnf4 {

struct PhiloxKey {
  uint32_t k0, k1, o0, o1;  // seed, offset
};

QDEV PhiloxKey philox_key(const DropArgs& d) {
  const uint64_t off = d.offset + (d.offset_dev ? (uint64_t)__ldg(d.offset_dev) : 0ull);
  return PhiloxKey{(uint32_t)d.seed, (uint32_t)(d.seed >> 32), (uint32_t)off, (uint32_t)(off >> 32)};
}

// High and low word of a product.  (As one 32 x 32 -> 64 instruction: a
// 64-bit multiplication of widened operands measured 112 cycles an evaluation
// and scheduler, this 90.)
QDEV void mul_wide(uint32_t a, uint32_t m, uint32_t& hi, uint32_t& lo) {
  uint64_t p;
  asm("mul.wide.u32 %0, %1, %2;" : "=l"(p) : "r"(a), "r"(m));
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(p));
}
// Keeps the evaluation of `w` ahead of the waits that follow in the program:
// without it the compiler sinks the arithmetic behind them, onto the path of
// the data.
QDEV void keep_here(uint4& w) { asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)); }

QDEV uint4 philox4x32_10(uint64_t ctr, const PhiloxKey& key) {
  uint32_t c0 = (uint32_t)ctr, c1 = (uint32_t)(ctr >> 32), c2 = key.o0, c3 = key.o1;
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    uint32_t h0, l0, h1, l1;
    mul_wide(c0, 0xD2511F53u, h0, l0);
    mul_wide(c2, 0xCD9E8D57u, h1, l1);
    c0 = h1 ^ c1 ^ k0;
    c2 = h0 ^ c3 ^ k1;
    c1 = l1;
    c3 = l0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Bit j set: element 8 ctr + j is kept.
QDEV uint32_t keep8(uint64_t ctr, const PhiloxKey& key, uint32_t threshold) {
  const uint4 w = philox4x32_10(ctr, key);
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m |= ((ws[j] & 0xFFFFu) >= threshold ? 1u : 0u) << (2 * j);
    m |= ((ws[j] >> 16) >= threshold ? 1u : 0u) << (2 * j + 1);
  }
  return m;
}

// Zero the dropped of eight bf16 (four words): `w` their random words, `thr`
// the threshold in the high half.  A 16-bit lane is kept where it is >= the
// threshold; for the high lane the whole word compares alike.
QDEV void drop8_bf16(uint32_t* x, const uint4& w, uint32_t thr) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (ws[j] < thr) x[j] &= 0x0000FFFFu;
    if ((ws[j] << 16) < thr) x[j] &= 0xFFFF0000u;
  }
}

}  // namespace qnf4
