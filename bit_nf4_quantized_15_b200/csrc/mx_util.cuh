// Descriptors shared by the block-scaled product kernels.
#pragma once

#include "common.cuh"

namespace qnf4 {
namespace {

constexpr int kMxKB = 256;  // reduction elements of a stage: 128 bytes of codes

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

}  // namespace
}  // namespace qnf4
