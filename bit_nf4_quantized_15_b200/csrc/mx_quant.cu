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

#include "engine_util.cuh"
#include "internal.h"
#include "launch.cuh"
#include "mx_codec.cuh"
#include "philox.cuh"

namespace qnf4 {
namespace {

constexpr int kQT = 256;  // threads of the element kernels

template <int DT>
constexpr int kWords = DT == QLORA_DTYPE_F32 ? 8 : 4;  // 32-bit words of eight elements

// Eight consecutive elements as they are stored.  CONST: nothing writes them
// while the kernel runs, so they may come through the read-only path.
template <int DT, bool CONST>
QDEV void load8(const uint4* p, uint32_t* w) {
#pragma unroll
  for (int j = 0; j < kWords<DT>; j += 4) {
    const uint4 r = CONST ? __ldg(p + j / 4) : p[j / 4];
    w[j] = r.x, w[j + 1] = r.y, w[j + 2] = r.z, w[j + 3] = r.w;
  }
}
// ... and as fp32, in pairs.
template <int DT>
QDEV float2 pair_of(const uint32_t* w, int j) {
  if constexpr (DT == QLORA_DTYPE_F32) return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  else if constexpr (DT == QLORA_DTYPE_BF16)
    return make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
}
// Largest |x| as fp32 bits (an Inf or NaN has exponent 255 and compares above).
template <int DT>
QDEV uint32_t absmax8(const uint32_t* w) {
  if constexpr (DT == QLORA_DTYPE_BF16) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = mx_absmax2(m, w[j]);
    return mx_absmax_bits(m);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = pair_of<DT>(w, j);
      m = max(m, max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu));
    }
    return m;
  }
}
template <int DT>
QDEV uint32_t codes8(const uint32_t* w, float f) {
  const float2 ff = make_float2(f, f);
  float2 u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = __fmul2_rn(pair_of<DT>(w, j), ff);
  return mx_codes8(u);
}

template <int DT>
QDEV float load1(const void* base, int64_t i) {
  if constexpr (DT == QLORA_DTYPE_F32) return reinterpret_cast<const float*>(base)[i];
  else if constexpr (DT == QLORA_DTYPE_BF16)
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[i]);
  else return __half2float(reinterpret_cast<const __half*>(base)[i]);
}

// One CTA per scale tile (128 rows x 128 columns).  16 threads share a row, 8
// elements each, so a warp reads whole row pieces; a thread has the loads of
// kRows rows in flight, as stored (fp32 takes twice the registers).  The block
// maximum is two shuffles over 4 lanes.  The 512 scale bytes meet in shared
// memory and leave as 16-byte stores, zeros outside the matrix.
//
// Bound by HBM: 8192 x 8192 bf16, 170 MB, 29 us (5.9 TB/s; 6.7 TB/s by the slope
// over larger ones).
template <int DT>
__global__ void __launch_bounds__(kQT) mx_quantize_kernel(const void* __restrict__ X, int64_t rows, int64_t cols,
                                                          uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                          int kt, int* status) {
  constexpr int kRows = DT == QLORA_DTYPE_F32 ? 4 : 8, kW = kWords<DT>;
  __shared__ __align__(16) uint8_t s_sc[512];
  pdl_trigger();
  const int t = threadIdx.x, rl0 = t >> 4, ch = t & 15;  // this thread's rows rl0 + 16 i, its 8 columns
  const unsigned rt = blockIdx.x / (unsigned)kt, ct = blockIdx.x % (unsigned)kt;
  const int64_t left = rows - (int64_t)rt * 128;
  const int n = (int64_t)ct * 128 + ch * 8 < cols ? (int)(left < 128 ? left : 128) : 0;  // rows to do
  const int64_t e8 = (((int64_t)rt * 128 + rl0) * cols + (int64_t)ct * 128) / 8 + ch;    // first row's 8 elements
  const uint4* px = reinterpret_cast<const uint4*>(X) + e8 * (kW / 4);
  uint32_t* pc = reinterpret_cast<uint32_t*>(codes) + e8;
  const int64_t step = 2 * cols;  // 16 rows, in groups of 8 elements
  bool bad = false;
#pragma unroll
  for (int p = 0; p < 8; p += kRows) {
    uint32_t w[kRows][kW];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (rl0 + 16 * (p + i) < n) {
        load8<DT, true>(px + (p + i) * step * (kW / 4), w[i]);
      } else {
#pragma unroll
        for (int j = 0; j < kW; ++j) w[i][j] = 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int rl = rl0 + 16 * (p + i);
      uint32_t m = absmax8<DT>(w[i]);
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const uint32_t b = mx_scale_byte(m);
      bad |= b == 255u;
      const uint32_t c = codes8<DT>(w[i], mx_inv_scale(b));
      if (rl < n) pc[(p + i) * step] = c;
      if ((t & 3) == 0) s_sc[(rl & 31) * 16 + (rl >> 5) * 4 + (ch >> 2)] = (uint8_t)b;  // 0 outside
    }
  }
  if (bad) report(status, QLORA_ERR_NONFINITE);
  __syncthreads();
  if (t < 32) reinterpret_cast<uint4*>(scales)[(int64_t)blockIdx.x * 32 + t] = reinterpret_cast<const uint4*>(s_sc)[t];
}

// Transposed: X [R][C], output [C][R] with blocks along R.  A tile is 128 r x
// 64 c, half the rows of an output scale tile.  It comes by TMA as it is
// stored, into a ring (the next tiles travel while this one is worked on); a
// thread owns a 32-block of one c, and a warp's reads of a row are consecutive
// words, so the tile needs neither padding nor a swizzle.  The codes meet in
// shared memory too and leave as 64 bytes a row of the output.
//
// Bound by HBM: 11008 x 4096 fp32, 204 MB, 34.4 us (5.9 TB/s); 8192 x 8192 bf16,
// 170 MB, 30 us (5.6).  With loads to registers and a CTA a tile it was 41 and
// 35; with two CTAs an SM and longer rings 34.9 and 32.8, with one or two 35.6
// of fp32, with four CTAs 30.9 of bf16.
template <int DT>
struct QtCfg {
  static constexpr int E = DT == QLORA_DTYPE_F32 ? 4 : 2;  // bytes an element
  static constexpr int TILE = 128 * 64 * E;
  static constexpr int S = E == 4 ? 2 : 3;      // stages
  static constexpr int CTAS = 3;                // that share an SM
  static constexpr int CODES = S * TILE;        // two buffers of 64 rows of 4 x 16 bytes, padded
  static constexpr int SC = CODES + 2 * 64 * 80;  // two of 256: 32 x (2 groups of 32 rows) x 4 blocks
  static constexpr int BAR = SC + 2 * 256;
  static constexpr int TOTAL = BAR + 64 + 128;
  static_assert(CTAS * (TOTAL + 1024) <= 228 * 1024, "budget");
};

template <int DT>
__global__ void __launch_bounds__(kQT, QtCfg<DT>::CTAS)
    mx_quantize_t_kernel(const __grid_constant__ CUtensorMap tm, int64_t R, int64_t C, uint8_t* __restrict__ codes,
                         uint8_t* __restrict__ scales, int kt, int* status) {
  using G = QtCfg<DT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::BAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(full + G::S);
  const int t = threadIdx.x, lane = t & 31;
  // consecutive CTAs walk along C, so that their row pieces share DRAM pages
  const unsigned n_ct = (unsigned)((C + 63) / 64), tiles = n_ct * (unsigned)kt;
  auto load = [&](unsigned tile, int s) {
    mbar_arrive_expect_tx(full + s, (uint32_t)G::TILE);  // zeros outside the matrix
    tma_load_2d(smem + s * G::TILE, &tm, full + s, (int)(tile % n_ct) * 64, (int)(tile / n_ct) * 128);
  };
  if (t == 0) {
    for (int s = 0; s < G::S; ++s) mbar_init(full + s, 1);
    *abort_flag = 0;
    fence_mbar_init();
    unsigned tile = blockIdx.x;
    for (int s = 0; s < G::S && tile < tiles; ++s, tile += gridDim.x) load(tile, s);
  }
  __syncthreads();

  const int cl = t & 63, blk = t >> 6;
  bool bad = false;
  int s = 0, o = 0;  // stage, output buffer
  uint32_t ph = 0;
  for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x, o ^= 1) {
    const unsigned ct = tile % n_ct, rt = tile / n_ct;  // 64 output rows, output scale-tile column
    const int64_t r0 = (int64_t)rt * 128, c0 = (int64_t)ct * 64;
    const int nr = (int)(R - r0 < 128 ? R - r0 : 128), nc = (int)(C - c0 < 64 ? C - c0 : 64);
    uint4(*s_c)[5] = reinterpret_cast<uint4(*)[5]>(smem + G::CODES + o * 64 * 80);
    uint8_t* s_sc = smem + G::SC + o * 256;
    const bool ok = warp_wait(full + s, ph, abort_flag, status, lane);
    if (ok) {
      const uint8_t* x = smem + s * G::TILE + blk * 32 * 64 * G::E;
      float v[32];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        v[j] = load1<DT>(x + j * 64 * G::E, cl);
        m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
      }
      const uint32_t b = mx_scale_byte(m);  // 0 outside the matrix
      const float f = mx_inv_scale(b);
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float2 u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          u[j] = __fmul2_rn(make_float2(v[8 * q + 2 * j], v[8 * q + 2 * j + 1]), make_float2(f, f));
        w[q] = mx_codes8(u);
      }
      s_c[cl][blk] = make_uint4(w[0], w[1], w[2], w[3]);
      s_sc[(cl & 31) * 8 + (cl >> 5) * 4 + blk] = (uint8_t)b;
      bad |= b == 255u;
    }
    // The stage has been read and the codes are in place.  (Those of the tile
    // before last, in the same buffer, were read before the last barrier.)
    if (__syncthreads_or(!ok)) break;
    if (t == 0 && (uint64_t)tile + (uint64_t)G::S * gridDim.x < tiles) load(tile + G::S * gridDim.x, s);
    {
      const int row = t >> 2, q = t & 3;  // 4 lanes a row of codes
      if (row < nc && q * 32 < nr) reinterpret_cast<uint4*>(codes)[((c0 + row) * R + r0) / 32 + q] = s_c[row][q];
    }
    // this tile's half of the scale tile: 8 of every 16 bytes
    uint8_t* sc = scales + ((int64_t)(ct >> 1) * kt + rt) * 512 + t * 16 + (ct & 1) * 8;
    if (t < 32) *reinterpret_cast<uint2*>(sc) = *reinterpret_cast<const uint2*>(s_sc + t * 8);
    // the last half tile of rows has no tile of its own: its padding is zero too
    if (t < 32 && ct + 1 == n_ct && (ct & 1) == 0) *reinterpret_cast<uint2*>(sc + 8) = make_uint2(0u, 0u);
    if (++s == G::S) {
      s = 0;
      ph ^= 1u;
    }
  }
  if (bad) report(status, QLORA_ERR_NONFINITE);
  if (*abort_flag && t == 0) {  // error path: let the loads in flight finish
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
}

// Value of a code times 2^(b - 127).  The E2M1 value is exact in fp16 and the
// product exact in fp32 (a subnormal one included: at least 2^-128), or past
// its range an infinity; scale byte 255 is NaN.
QDEV float2 values2(uint32_t byte, float lo, float hi) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)byte, __NV_E2M1);
  const float2 f = __half22float2(__half2(h));
  return make_float2(__fmul_rn(__fmul_rn(f.x, lo), hi), __fmul_rn(__fmul_rn(f.y, lo), hi));
}

// One CTA per scale tile again, the quantiser's mapping: its 512 scale bytes
// through shared memory, 8 rows' codes in flight a thread, 16-byte stores.
// Bound by HBM: 8192 x 8192 to bf16, 170 MB, 28 us.
template <int DT>
__global__ void __launch_bounds__(kQT) mx_dequant_kernel(const uint32_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int64_t rows,
                                                         int64_t cols, int kt, void* __restrict__ out) {
  __shared__ __align__(16) uint8_t s_sc[512];
  const int t = threadIdx.x, rl0 = t >> 4, ch = t & 15;
  const unsigned rt = blockIdx.x / (unsigned)kt, ct = blockIdx.x % (unsigned)kt;
  const int64_t left = rows - (int64_t)rt * 128;
  const int n = (int64_t)ct * 128 + ch * 8 < cols ? (int)(left < 128 ? left : 128) : 0;
  const int64_t e8 = (((int64_t)rt * 128 + rl0) * cols + (int64_t)ct * 128) / 8 + ch;
  const int64_t step = 2 * cols;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = rl0 + 16 * i < n ? __ldg(codes + e8 + i * step) : 0u;
  if (t < 32)
    reinterpret_cast<uint4*>(s_sc)[t] = __ldg(reinterpret_cast<const uint4*>(scales) + (int64_t)blockIdx.x * 32 + t);
  __syncthreads();
  uint4* po = reinterpret_cast<uint4*>(out) + e8 * (kWords<DT> / 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rl = rl0 + 16 * i;
    if (rl >= n) break;
    const uint32_t b = s_sc[(rl & 31) * 16 + (rl >> 5) * 4 + (ch >> 2)];
    // 2^(b - 127) as a product of two normal powers of two
    const float lo = b == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((64u + (b >> 1)) << 23);
    const float hi = __uint_as_float((63u + b - (b >> 1)) << 23);
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = values2((w[i] >> (8 * j)) & 255u, lo, hi);
    uint4* o = po + i * step * (kWords<DT> / 4);
    if constexpr (DT == QLORA_DTYPE_F32) {
      reinterpret_cast<float4*>(o)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
      reinterpret_cast<float4*>(o)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    } else {
      *o = make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                      pack_bf16x2(v[3].x, v[3].y));
    }
  }
}

template <int DT>
QDEV void store1(void* out, int64_t i, float v) {
  if constexpr (DT == QLORA_DTYPE_F32) reinterpret_cast<float*>(out)[i] = v;
  else if constexpr (DT == QLORA_DTYPE_BF16) reinterpret_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else reinterpret_cast<__half*>(out)[i] = __float2half_rn(v);
}

// Eight elements as stored: dropped ones to zero (a selection: a dropped Inf
// or NaN is 0), the others times inv.
template <int DT>
QDEV void drop_store8(void* out, int64_t i, uint32_t* w, const uint4& rnd, const DropArgs& d) {
  const uint32_t thr = d.threshold << 16;
  if constexpr (DT == QLORA_DTYPE_F32) {
    const uint32_t ws[4] = {rnd.x, rnd.y, rnd.z, rnd.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if ((ws[j] << 16) < thr) w[2 * j] = 0u;
      if (ws[j] < thr) w[2 * j + 1] = 0u;
    }
  } else {
    drop8_bf16(w, rnd, thr);  // two 16-bit elements a word, of either kind
  }
  float2 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = pair_of<DT>(w, j);
    v[j] = make_float2(__fmul_rn(v[j].x, d.inv), __fmul_rn(v[j].y, d.inv));
  }
  if constexpr (DT == QLORA_DTYPE_F32) {
    reinterpret_cast<float4*>(out)[2 * i] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    reinterpret_cast<float4*>(out)[2 * i + 1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  } else {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == QLORA_DTYPE_BF16) {
        o[j] = pack_bf16x2(v[j].x, v[j].y);
      } else {
        const __half2 h = __floats2half2_rn(v[j].x, v[j].y);
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    reinterpret_cast<uint4*>(out)[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// out = x inv where kept, else 0.  Eight elements (one generator evaluation) a
// thread and turn; a step has two turns with their loads in flight.  Bound by
// HBM: 8192 x 8192 bf16, 268 MB, 47 us (5.7 TB/s), fp32 87 us (6.2 TB/s; with
// one turn 93); a copy of the bf16 tensor takes 42.  out may be X: a thread
// reads what it writes, by ordinary loads.
template <int DT>
__global__ void __launch_bounds__(kQT) dropout_kernel(const void* X, int64_t n, DropArgs d, void* out) {
  constexpr int kTurns = 2;
  const PhiloxKey key = philox_key(d);
  const int64_t n8 = n / 8, stride = (int64_t)gridDim.x * kQT;
  for (int64_t i = (int64_t)blockIdx.x * kQT + threadIdx.x; i < n8; i += kTurns * stride) {
    uint32_t w[kTurns][kWords<DT>];
#pragma unroll
    for (int k = 0; k < kTurns; ++k)
      if (i + k * stride < n8)
        load8<DT, false>(reinterpret_cast<const uint4*>(X) + (i + k * stride) * (kWords<DT> / 4), w[k]);
#pragma unroll
    for (int k = 0; k < kTurns; ++k)
      if (i + k * stride < n8)
        drop_store8<DT>(out, i + k * stride, w[k], philox4x32_10((uint64_t)(i + k * stride), key), d);
  }
  const int64_t tail = n8 * 8;
  if (blockIdx.x == 0 && threadIdx.x < n - tail) {
    const int64_t i = tail + threadIdx.x;
    const uint32_t keep = keep8((uint64_t)n8, key, d.threshold);
    store1<DT>(out, i, (keep >> threadIdx.x) & 1u ? __fmul_rn(load1<DT>(X, i), d.inv) : 0.0f);
  }
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
                              int sms, cudaStream_t st) {
  using G = QtCfg<DT>;
  CUtensorMap tm;
  if (make_map(&tm, X, G::E == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, G::E, (uint64_t)C,
               (uint64_t)R, 64, 128, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const int kt = (int)((R + 127) / 128);
  const int64_t tiles = (C + 63) / 64 * kt, most = (int64_t)sms * G::CTAS;
  return launch_kernel<mx_quantize_t_kernel<DT>>(
      {dim3((unsigned)(tiles < most ? tiles : most)), kQT, G::TOTAL, 1, false}, st, tm, R, C, codes, scales, kt,
      status);
}

cudaError_t launch_mx_quantize_t(const void* X, int dtype, int64_t R, int64_t C, uint8_t* codes, uint8_t* scales,
                                 int* status, int sms, cudaStream_t st) {
  switch (dtype) {
    case QLORA_DTYPE_BF16: return quantize_t<QLORA_DTYPE_BF16>(X, R, C, codes, scales, status, sms, st);
    case QLORA_DTYPE_F16: return quantize_t<QLORA_DTYPE_F16>(X, R, C, codes, scales, status, sms, st);
    default: return quantize_t<QLORA_DTYPE_F32>(X, R, C, codes, scales, status, sms, st);
  }
}

cudaError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int dtype,
                              void* out, cudaStream_t st) {
  const int kt = (int)((cols + 127) / 128);
  const unsigned grid = (unsigned)(((rows + 127) / 128) * kt);
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  if (dtype == QLORA_DTYPE_F32)
    mx_dequant_kernel<QLORA_DTYPE_F32><<<grid, kQT, 0, st>>>(c, scales, rows, cols, kt, out);
  else
    mx_dequant_kernel<QLORA_DTYPE_BF16><<<grid, kQT, 0, st>>>(c, scales, rows, cols, kt, out);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_dropout(const void* X, int dtype, int64_t n, const DropArgs& d, void* out, int sms, cudaStream_t st) {
  const int64_t want = ((n + 7) / 8 + kQT - 1) / kQT, most = (int64_t)sms * 16;
  const int grid = (int)(want < most ? want : most);
  switch (dtype) {
    case QLORA_DTYPE_BF16: dropout_kernel<QLORA_DTYPE_BF16><<<grid, kQT, 0, st>>>(X, n, d, out); break;
    case QLORA_DTYPE_F16: dropout_kernel<QLORA_DTYPE_F16><<<grid, kQT, 0, st>>>(X, n, d, out); break;
    default: dropout_kernel<QLORA_DTYPE_F32><<<grid, kQT, 0, st>>>(X, n, d, out);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace qnf4
