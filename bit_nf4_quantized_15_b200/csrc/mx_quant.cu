// MXFP4 quantisation and dequantisation, and dropout: the memory-bound
// element passes of the microscaled path.
//
// MXFP4 (OCP Microscaling Formats v1.0): blocks of 32 elements along a row,
// E2M1 codes and one E8M0 scale 2^(b - 127) a block,
//   b    = max(exponent(max |x|) - 2, 0)   (biased fp32 exponent; 255 for a
//                                           block that holds an Inf or NaN)
//   code = E2M1(x 2^(127 - b))   nearest, ties to even, saturated to 6.
// The scaled value is exact (a power of two), so the code is rounded once.
//
// Scales are stored as the block-scaled MMA reads them: tiles of 128 rows x
// 4 blocks (128 columns), 512 bytes, the tiles of one row range consecutive;
// in a tile the scale of row i, block j is byte (i % 32) * 16 + (i / 32) * 4
// + j.  A tile goes from global to tensor memory without being rearranged.
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "mx_codec.cuh"
#include "philox.cuh"

namespace qnf4 {
namespace {

constexpr int kQT = 256;  // threads of the element kernels

// Eight consecutive elements as fp32.
template <int DT>
QDEV void load8(const void* base, int64_t i, float (&v)[8]) {
  if constexpr (DT == QLORA_DTYPE_F32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(base) + i / 4);
    const float4 b = __ldg(reinterpret_cast<const float4*>(base) + i / 4 + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(base) + i / 8);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == QLORA_DTYPE_BF16) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
      }
    }
  }
}

template <int DT>
QDEV float load1(const void* base, int64_t i) {
  if constexpr (DT == QLORA_DTYPE_F32) return reinterpret_cast<const float*>(base)[i];
  else if constexpr (DT == QLORA_DTYPE_BF16)
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[i]);
  else return __half2float(reinterpret_cast<const __half*>(base)[i]);
}

QDEV uint32_t codes8(const float (&v)[8], float f) {
  const float2 ff = make_float2(f, f);
  float2 u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = __fmul2_rn(make_float2(v[2 * j], v[2 * j + 1]), ff);
  return mx_codes8(u);
}

// One CTA per scale tile (128 rows x 128 columns).  16 threads share a row,
// 8 elements (one 16-byte load) each, so a warp reads whole 256-byte row
// pieces; every thread has its 8 rows' loads in flight at once.  The block
// maximum is two shuffles over 4 lanes.  The 512 scale bytes meet in shared
// memory and leave as 16-byte stores, zeros outside the matrix.
template <int DT>
__global__ void __launch_bounds__(kQT) mx_quantize_kernel(const void* __restrict__ X, int64_t rows, int64_t cols,
                                                          uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                          int kt, int* status) {
  __shared__ __align__(16) uint8_t s_sc[512];
  pdl_trigger();
  const int t = threadIdx.x;
  const int64_t rt = blockIdx.x / kt;
  const int ct = (int)(blockIdx.x % kt);
  const int64_t row0 = rt * 128;
  const int64_t col = (int64_t)ct * 128 + (t & 15) * 8;
  const bool cok = col < cols;
  if (t < 32) reinterpret_cast<uint4*>(s_sc)[t] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + (t >> 4) + 16 * i;
    if (cok && row < rows) load8<DT>(X, row * cols + col, v[i]);
    else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rl = (t >> 4) + 16 * i;
    const int64_t row = row0 + rl;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const uint32_t b = mx_scale_byte(m);
    bad |= b == 255u;
    const uint32_t w = codes8(v[i], mx_inv_scale(b));
    if (cok && row < rows) {
      reinterpret_cast<uint32_t*>(codes)[(row * cols + col) >> 3] = w;
      if ((t & 3) == 0) s_sc[(rl & 31) * 16 + (rl >> 5) * 4 + ((t & 15) >> 2)] = (uint8_t)b;
    }
  }
  if (bad) report(status, QLORA_ERR_NONFINITE);
  __syncthreads();
  if (t < 32) reinterpret_cast<uint4*>(scales)[(rt * kt + ct) * 32 + t] = reinterpret_cast<const uint4*>(s_sc)[t];
}

// Transposed: X [R][C], output [C][R] with blocks along R.  One CTA per
// output scale tile: a 128 (r) x 128 (c) piece goes through shared memory as
// fp32 (row pitch 129 words: both the row writes and the column reads are
// free of bank conflicts up to the vector loads' order); a thread then owns
// one c and two blocks of 32 r.
constexpr int kTP = 129;
template <int DT>
__global__ void __launch_bounds__(kQT) mx_quantize_t_kernel(const void* __restrict__ X, int64_t R, int64_t C,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales, int kt, int* status) {
  extern __shared__ float s_x[];
  __shared__ __align__(16) uint8_t s_sc[512];
  const int t = threadIdx.x;
  // consecutive CTAs walk along C, so that their row pieces share DRAM pages
  const int64_t n_ct = (C + 127) / 128;
  const int64_t ct = blockIdx.x % n_ct;      // output row tile
  const int rt = (int)(blockIdx.x / n_ct);   // output scale-tile column
  if (t < 32) reinterpret_cast<uint4*>(s_sc)[t] = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rl = (t >> 4) + 16 * i;
    const int64_t r = (int64_t)rt * 128 + rl, c = ct * 128 + (t & 15) * 8;
    float v[8];
    if (r < R && c < C) load8<DT>(X, r * C + c, v);
    else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s_x[rl * kTP + (t & 15) * 8 + j] = v[j];
  }
  __syncthreads();
  const int cl = t & 127, half = t >> 7;
  const int64_t c = ct * 128 + cl;
  bool bad = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int blk = half * 2 + h;
    const int64_t r0 = (int64_t)rt * 128 + blk * 32;
    if (c >= C || r0 >= R) continue;
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[j] = s_x[(blk * 32 + j) * kTP + cl];
      m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    }
    const uint32_t b = mx_scale_byte(m);
    bad |= b == 255u;
    const float f = mx_inv_scale(b);
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float u[8] = {v[8 * q], v[8 * q + 1], v[8 * q + 2], v[8 * q + 3], v[8 * q + 4], v[8 * q + 5], v[8 * q + 6],
                          v[8 * q + 7]};
      w[q] = codes8(u, f);
    }
    reinterpret_cast<uint4*>(codes)[(c * R + r0) >> 5] = make_uint4(w[0], w[1], w[2], w[3]);
    s_sc[(cl & 31) * 16 + (cl >> 5) * 4 + blk] = (uint8_t)b;
  }
  if (bad) report(status, QLORA_ERR_NONFINITE);
  __syncthreads();
  if (t < 32) reinterpret_cast<uint4*>(scales)[(ct * kt + rt) * 32 + t] = reinterpret_cast<const uint4*>(s_sc)[t];
}

// Value of a code times 2^(b - 127).  The E2M1 value is exact in fp16 and the
// product exact in fp32 (a subnormal one included: at least 2^-128); scale
// byte 255 is NaN.
QDEV float2 values2(uint32_t byte, float lo, float hi) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)byte, __NV_E2M1);
  const float2 f = __half22float2(__half2(h));
  return make_float2(__fmul_rn(__fmul_rn(f.x, lo), hi), __fmul_rn(__fmul_rn(f.y, lo), hi));
}

// Eight elements a thread: a 4-byte code load and one (bf16) or two (fp32)
// 16-byte stores, all coalesced; the four threads of a block read the same
// scale byte.
template <int DT>
__global__ void __launch_bounds__(kQT) mx_dequant_kernel(const uint32_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int64_t n8, int cols8,
                                                         int kt, void* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * kQT + threadIdx.x; i < n8; i += (int64_t)gridDim.x * kQT) {
    const int64_t row = i / cols8;
    const int c8 = (int)(i - row * cols8);
    const int blk = c8 >> 2, rl = (int)(row & 127);
    const uint32_t b = __ldg(scales + ((row >> 7) * kt + (blk >> 2)) * 512 + (rl & 31) * 16 + (rl >> 5) * 4 + (blk & 3));
    const uint32_t w = __ldg(codes + i);
    // 2^(b - 127) as a product of two normal powers of two
    const float lo = b == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((64u + (b >> 1)) << 23);
    const float hi = __uint_as_float((63u + b - (b >> 1)) << 23);
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = values2((w >> (8 * j)) & 255u, lo, hi);
    if constexpr (DT == QLORA_DTYPE_F32) {
      reinterpret_cast<float4*>(out)[2 * i] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
      reinterpret_cast<float4*>(out)[2 * i + 1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    } else {
      reinterpret_cast<uint4*>(out)[i] = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                                    pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
    }
  }
}

template <int DT>
QDEV void store1(void* out, int64_t i, float v) {
  if constexpr (DT == QLORA_DTYPE_F32) reinterpret_cast<float*>(out)[i] = v;
  else if constexpr (DT == QLORA_DTYPE_BF16) reinterpret_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else reinterpret_cast<__half*>(out)[i] = __float2half_rn(v);
}

// out = x inv where kept, else 0 (a selection: a dropped Inf or NaN is 0).
// Eight elements (one generator evaluation) a thread and step.
template <int DT>
__global__ void __launch_bounds__(kQT) dropout_kernel(const void* __restrict__ X, int64_t n, DropArgs d,
                                                      void* __restrict__ out) {
  const PhiloxKey key = philox_key(d);
  const int64_t n8 = n / 8, stride = (int64_t)gridDim.x * kQT;
  for (int64_t i = (int64_t)blockIdx.x * kQT + threadIdx.x; i < n8; i += stride) {
    float v[8];
    load8<DT>(X, i * 8, v);
    const uint32_t keep = keep8((uint64_t)i, key, d.threshold);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (keep >> j) & 1u ? __fmul_rn(v[j], d.inv) : 0.0f;
    if constexpr (DT == QLORA_DTYPE_F32) {
      reinterpret_cast<float4*>(out)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(out)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if constexpr (DT == QLORA_DTYPE_BF16) {
      reinterpret_cast<uint4*>(out)[i] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                    pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      reinterpret_cast<uint4*>(out)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  const int64_t tail = n8 * 8;
  if (blockIdx.x == 0 && threadIdx.x < n - tail) {
    const int64_t i = tail + threadIdx.x;
    const uint32_t keep = keep8((uint64_t)n8, key, d.threshold);
    store1<DT>(out, i, (keep >> threadIdx.x) & 1u ? __fmul_rn(load1<DT>(X, i), d.inv) : 0.0f);
  }
}

int elem_grid(int64_t n) {
  const int64_t want = (n + kQT - 1) / kQT;
  return (int)(want < 148 * 16 ? (want > 0 ? want : 1) : 148 * 16);
}

}  // namespace

cudaError_t launch_mx_quantize(const void* X, int dtype, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                               int* status, cudaStream_t st) {
  const int kt = (int)((cols + 127) / 128);
  const unsigned grid = (unsigned)(((rows + 127) / 128) * kt);
  switch (dtype) {
    case QLORA_DTYPE_BF16:
      mx_quantize_kernel<QLORA_DTYPE_BF16><<<grid, kQT, 0, st>>>(X, rows, cols, codes, scales, kt, status);
      break;
    case QLORA_DTYPE_F16:
      mx_quantize_kernel<QLORA_DTYPE_F16><<<grid, kQT, 0, st>>>(X, rows, cols, codes, scales, kt, status);
      break;
    default:
      mx_quantize_kernel<QLORA_DTYPE_F32><<<grid, kQT, 0, st>>>(X, rows, cols, codes, scales, kt, status);
  }
  count_launches(1);
  return cudaGetLastError();
}

template <int DT>
static cudaError_t quantize_t(const void* X, int64_t R, int64_t C, uint8_t* codes, uint8_t* scales, int* status,
                              cudaStream_t st) {
  const int kt = (int)((R + 127) / 128);
  const unsigned grid = (unsigned)(((C + 127) / 128) * kt);
  const int smem = 128 * kTP * 4;
  cudaError_t err = cudaFuncSetAttribute(mx_quantize_t_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  mx_quantize_t_kernel<DT><<<grid, kQT, smem, st>>>(X, R, C, codes, scales, kt, status);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_mx_quantize_t(const void* X, int dtype, int64_t R, int64_t C, uint8_t* codes, uint8_t* scales,
                                 int* status, cudaStream_t st) {
  switch (dtype) {
    case QLORA_DTYPE_BF16: return quantize_t<QLORA_DTYPE_BF16>(X, R, C, codes, scales, status, st);
    case QLORA_DTYPE_F16: return quantize_t<QLORA_DTYPE_F16>(X, R, C, codes, scales, status, st);
    default: return quantize_t<QLORA_DTYPE_F32>(X, R, C, codes, scales, status, st);
  }
}

cudaError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int dtype,
                              void* out, cudaStream_t st) {
  const int kt = (int)((cols + 127) / 128), cols8 = (int)(cols / 8);
  const int64_t n8 = rows * cols8;
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  if (dtype == QLORA_DTYPE_F32)
    mx_dequant_kernel<QLORA_DTYPE_F32><<<elem_grid(n8), kQT, 0, st>>>(c, scales, n8, cols8, kt, out);
  else
    mx_dequant_kernel<QLORA_DTYPE_BF16><<<elem_grid(n8), kQT, 0, st>>>(c, scales, n8, cols8, kt, out);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_dropout(const void* X, int dtype, int64_t n, const DropArgs& d, void* out, cudaStream_t st) {
  const int grid = elem_grid((n + 7) / 8);
  switch (dtype) {
    case QLORA_DTYPE_BF16: dropout_kernel<QLORA_DTYPE_BF16><<<grid, kQT, 0, st>>>(X, n, d, out); break;
    case QLORA_DTYPE_F16: dropout_kernel<QLORA_DTYPE_F16><<<grid, kQT, 0, st>>>(X, n, d, out); break;
    default: dropout_kernel<QLORA_DTYPE_F32><<<grid, kQT, 0, st>>>(X, n, d, out);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace qnf4
