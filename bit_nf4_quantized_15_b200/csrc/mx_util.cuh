// Descriptors shared by the block-scaled product kernels.
#pragma once

#include "common.cuh"

namespace qnf4 {
namespace {

// Cluster barrier in two halves, by whole warps (the lanes meet first).  The arrival is a release:
// it orders the reads of the peers' shared memory before it, so that a peer
// that leaves after its wait gives up nothing that is still being read.
QDEV void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
QDEV void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kMxKB = 256;  // reduction elements of a stage: 128 bytes of codes

// Stages of one accumulation of an fp32 product.  The tensor cores truncate
// their sums, toward zero and by the length of the sum: blocks of sizes over
// 2^24 : 1 and 22016 terms in one accumulation were 6.9e-6 off (fp32 arithmetic
// 1.1e-6; blocks of about one size are exact either way).  So an fp32 result is
// accumulated in pieces of 2048 terms that are added with rounding: 0.7e-6,
// whatever the length (8192^3 in 317 us, 302 in one accumulation).  A bf16
// result takes one accumulation: its own rounding is 1.7e-3.
constexpr int kMxPiece = 8;

// Instruction descriptor, kind::mxf4: E2M1 x E2M1, E8M0 scales; the scale ids
// pick bytes 0-1 or 2-3 of each scale column word (two 32-blocks a step).
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, int sf_id) {
  return ((uint32_t)sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 7) << 27) | ((uint32_t)sf_id << 29);
}
// Unswizzled matrix of 16-byte rows, 8-row groups 128 bytes apart.
QDEV uint64_t sdesc_scales(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)8 << 32) | ((uint64_t)1 << 46);
}

// Stores from shared memory by TMA (the issuing thread's bulk group).
QDEV void tma_store_2d(const CUtensorMap* m, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"((uint64_t)m),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}
QDEV void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
QDEV void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
QDEV void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
QDEV void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// One elected lane of a converged warp.  The MMA warps below run their loops
// with all 32 lanes and only predicate the tensor-core instructions with it:
// their addresses and descriptors then stay in uniform registers.  (With a
// loop in a lane == 0 branch every operand is moved there one by one: 100
// cycles an MMA and 62 a scale copy were measured, which made the issuing
// thread the bound, 1140 cycles a stage of 512 cycles of tensor work.)
QDEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// K-major, 128-byte-swizzled operand tile: the descriptor's constant half and
// its address half (advance by 2 for each 32 bytes of K).
constexpr uint32_t kDescHi = (uint32_t)((1024u >> 4) | (1u << 14) | (2u << 29));
QDEV uint64_t kdesc(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }
QDEV uint32_t kdesc_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }

}  // namespace
}  // namespace qnf4
