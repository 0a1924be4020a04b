// Internal declarations shared by the kernels and the C-ABI layer.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mx_plan.h"

namespace qnf4 {

// ------------------------------------------------- host helpers (api.cu)
struct DevInfo {
  int ok = 0;
  int sms = 148;
};
int current_device_info(DevInfo* out);
// 2-D map over a row-major matrix [outer][inner] of `esize`-byte elements.
int make_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int esize, uint64_t inner, uint64_t outer,
             uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw);
// 3-D map of bf16 with dimensions n0 (contiguous) x n1 x n2, `s1` and `s2` bytes
// apart, 128-byte swizzle.
int make_map3(CUtensorMap* m, const void* base, uint64_t n0, uint64_t n1, uint64_t n2, uint64_t s1, uint64_t s2,
              uint32_t b0, uint32_t b1, uint32_t b2);
// bf16 operand of the engines.  K-major: matrix [mn][k] (k contiguous), box
// 64 k x `rows` mn.  MN-major: matrix [k][mn] (mn contiguous), box 64 x 64.
int map_operand(CUtensorMap* m, const void* base, int mn_major, uint64_t mn_extent, uint64_t k_extent, int rows);
// Takes this thread's pending request of qlora_debug_stall_next_gemm (0: none).
uint64_t take_stall_request();

// NF4 codebook and decision thresholds as the kernels use them.
//   q[i] : the 16 levels (fp32), ascending, q[7] = 0 exactly.
//   t[i] : RD32 of the exact midpoint (q[i] + q[i+1]) / 2; for an fp32 x,
//          x > midpoint  <=>  x > t[i].
struct Nf4Tables {
  float q[16];
  float t[15];
  // Code search used by the quantiser: a degree-5 polynomial f(x) with
  // f(t[i]) in [i + 0.1, i + 0.9], f(-1) >= 0.1, f(1) <= 14.9 and f increasing
  // on [-1, 1], so that k = round(f(x) - 1/2) is the code of x or one less and
  // code = k + (x > t[k]).  poly[0] already includes the -1/2.
  float poly[6];
  bool poly_ok;  // the conditions above were verified when the tables were built
};

// Derived once per process on the host, from the normal quantiles.
const Nf4Tables& nf4_tables();

// Code formats (QLORA_FMT_*): NF4, and the two formats the method is
// compared with, FP4 (E2M1 / 6) and Int4 (k / 7), each with a pad level
// below -1 that is never produced.  Same table layout; only NF4 has a
// code-search polynomial (poly_ok is false for the others, whose quantiser
// searches the thresholds).
constexpr int kNumFormats = 3;
const Nf4Tables& code_tables(int format);  // format in [0, kNumFormats)

// Process-wide count of kernels launched through the library.
void count_launches(uint64_t n);
uint64_t launches_so_far();

// ------------------------------------------------------------------ engine
// Where the UMMA A operand of the main segment comes from.
enum AMode : int {
  A_TMA = 0,     // TMA tile (K- or MN-major per args)
  A_DEQ_K = 1,   // NF4 dequantised on chip, K-major  (A = W^, rows = n, k along K)
  A_DEQ_MN = 2,  // NF4 dequantised on chip, MN-major (A = W^T, rows = k, reduction over n)
};

// Final store of an accumulator element (row, col) of the output tile:
//   out [row*rs  + col*cs ] = alpha  * v   (fp32 or bf16)
//   out2[row*rs2 + col*cs2] = alpha2 * v   (bf16, optional)
struct EpiArgs {
  void* out;
  int out_bf16;
  float alpha;
  int64_t rs, cs;
  void* out2;
  float alpha2;
  int64_t rs2, cs2;
};

struct EngineArgs {
  CUtensorMap tmA;   // main A (A_TMA) or the NF4 code tensor (A_DEQ_*)
  CUtensorMap tmB;   // main B
  CUtensorMap tmAx;  // extension A (LoRA term)
  CUtensorMap tmBx;  // extension B
  const uint8_t* codes;  // NF4 codes [wN][wK/2] (read directly by the pair forward)
  const uint8_t* c2;
  int c2_e5m2;           // c2 holds E5M2 codes instead of E4M3
  int c1_mean;           // mean-centred codec: c1 holds [c1, mean] per group
  const float* c1;
  int64_t wN, wK;    // quantised weight shape (for scale indexing)
  int rows, cols;    // output extent: UMMA-M side, UMMA-N side
  int kb_main;       // 64-wide reduction blocks of the main segment
  int kb_ext;        // 64-wide reduction blocks of the extension (0: none)
  int splits;        // split of the main reduction across grid.z
  int a_mn_main, b_mn_main, a_mn_ext, b_mn_ext;
  float* partial;    // [splits][cols][rows] fp32 when splits > 1
  EpiArgs epi;
  int* status;
  uint64_t wait_ns;  // bound of every internal wait (0: the default, 4 s)
  int stall;         // failure-detection hook: the producer issues no loads
  float q[16];
};

struct GemmPlan {
  int BN;
  int m_tiles, n_tiles, splits;
  size_t partial_bytes;
};

int bn_for_cols(int cols);  // token-tile width: the smallest of 16 ... 256 that holds `cols`, else 256
GemmPlan plan_gemm(int rows, int cols, int kb_main, int num_sms);
size_t engine_smem_bytes(int BN, int amode);
cudaError_t launch_engine(const EngineArgs& a, int amode, const GemmPlan& p, cudaStream_t st);
cudaError_t launch_split_reduce(const float* partial, int splits, int rows, int cols, const EpiArgs& e,
                                cudaStream_t st);

// Forward dequant-GEMM on CTA pairs (cta_group::2, 256 x 256 output tile per
// pair).  Same EngineArgs as A_DEQ_K with these tensor maps: tmA codes (box
// 32 x 128 bytes), tmB X (K-major, box 64 x 128), tmAx L2 (MN-major, 64 x 64),
// tmBx RNbf16(s.T) (K-major, box 64 x 128); bf16 output, no split.
bool pair_fwd_supported(int rows, int cols, int kb_ext);
size_t pair_fwd_smem_bytes();
cudaError_t launch_pair_fwd(const EngineArgs& a, cudaStream_t st);

// ------------------------------------------------------------ small-M GEMV
// Forward for M <= kGemvMaxM tokens: Y = X.W^T + s.(X.L1).L2 with the weight
// streamed once from HBM.  Three kernels:
//   (1) T partials: Tp[p][m][j] = sum_{k in slice p} X[m,k] L1[k,j]
//   (2) stream-K dequant-GEMV: the units (128-row tile, 256-wide k range) of
//       W split in equal runs over three workers per SM; every maximal run
//       inside one row tile (a segment) leaves a 128 x 16 fp32 partial tile;
//       one warp per CTA also sums its share of the T partials (T saved,
//       RNbf16(s.T) for (3));
//   (3) finish: Y = RNbf16(sum of a row tile's partials in worker order
//       + RNbf16(s.T).L2).
constexpr int kGemvMaxM = 16;
constexpr int kGemvTSlices = 128;  // max T partial slices

struct GemvPlan {
  int m_tiles, kbt;   // 128-row tiles of W, 64-wide k blocks per row
  int upr;            // units per row tile (256-wide k ranges)
  int64_t units;      // m_tiles * upr
  int grid, workers;  // CTAs (<= SMs), stream-K workers (3 per CTA)
  int maxc;           // max workers covering one row tile
  int t_slices, bps;  // T partial slices, k blocks per slice
  size_t part_bytes;  // segment partials [m_tiles * maxc][16][128] fp32
  size_t tp_bytes;    // T partials [t_slices][16][128] fp32
  size_t stw_bytes;   // RNbf16(s.T) as fp32 [16][128]
};

struct GemvArgs {
  CUtensorMap tmCodes;  // uint8 [N][K/2], box 128 x 128, 128-byte swizzle
  CUtensorMap tmX;      // bf16 [M][K] as 3-D (64, M, K/64), box 64 x 16 x 4, 128-byte swizzle
  const uint8_t* c2;
  int c2_e5m2;          // c2 holds E5M2 codes instead of E4M3
  int c1_mean;          // mean-centred codec: c1 holds [c1, mean] per group
  const float* c1;
  int64_t N, K;
  int M;
  int kbt, upr, m_tiles, maxc;
  int64_t units;
  float* part;
  // LoRA: T partials in, T (saved) and RNbf16(s.T) out
  const float* tp;
  int t_slices, r;
  float s;
  float* T_save;
  float* sTw;
  int* status;
  uint32_t smem_bytes;
  float q[16];
};

GemvPlan plan_gemv(int64_t M, int64_t N, int64_t K, int num_sms);
cudaError_t launch_gemv(const GemvArgs& a, const GemvPlan& p, const uint16_t* X, const uint16_t* L1,
                        const uint16_t* L2, uint16_t* Y, cudaStream_t st);

// ------------------------------------------------- small-M backward (GEMV)
// Backward for M <= kGemvMaxM tokens with the weight streamed once:
//   (1) lora_bwd_n_kernel: over N slices, dL2 = s.T^T.dY and the slices'
//       partials of dT = dY.L2^T; zeroes the k-range arrival counters;
//   (2) nf4_gemv_t_kernel: dX = dY.W^ by stream-K over units (128-row tile
//       of W, 256-wide k range) ordered by k range; the last worker of a k
//       range adds s.dT.L1^T, rounds dX and forms dL1 = s.X^T.dT there.
struct GemvTPlan {
  int n_tiles, kbt, k_ranges;  // 128-row tiles of W, 64-wide k blocks, 256-wide k ranges
  int64_t units;               // n_tiles * k_ranges
  int grid, workers, maxc;     // CTAs, stream-K workers (3 per CTA), max workers per k range
  int slice, t_slices;         // dT slices over N
  size_t part_bytes;           // [k_ranges][maxc][16][256] fp32
  size_t tp_bytes;             // [t_slices][16][128] fp32
  size_t cnt_bytes;            // [k_ranges] int
};

struct GemvTArgs {
  CUtensorMap tmCodes;  // uint8 [N][K/2], box 128 x 128, 128-byte swizzle
  CUtensorMap tmDY;     // bf16 [M][N], box 64 x 16, 128-byte swizzle
  const uint8_t* c2;
  int c2_e5m2, c1_mean;
  const float* c1;
  int64_t N, K;
  int M, r, kbt, n_tiles, maxc, t_slices;
  int64_t units;
  float s;
  float* part;
  const float* tp;
  int* cnt;
  const uint16_t* L1;
  const uint16_t* X;
  uint16_t* dX;   // may be null
  float* dL1;     // may be null
  int* status;
  uint32_t smem_bytes;
  float q[16];
};

GemvTPlan plan_gemv_t(int64_t M, int64_t N, int64_t K, int num_sms);
cudaError_t launch_gemv_t(const GemvTArgs& a, const GemvTPlan& p, const uint16_t* dY, const uint16_t* L2,
                          const float* T, float* dL2, cudaStream_t st);

// --------------------------------------------------------- quantise kernels
cudaError_t launch_quantize(const uint16_t* W, int64_t n_weights, uint8_t* codes, uint8_t* c2, float* c1,
                            int* status, int format, int scale_codec, cudaStream_t st);
cudaError_t launch_dequant(const uint8_t* codes, const uint8_t* c2, const float* c1, int64_t n_weights,
                           uint16_t* out, int format, int scale_codec, cudaStream_t st);
cudaError_t launch_scale_to_bf16(const float* in, int64_t n, float s, uint16_t* out, cudaStream_t st);

// ------------------------------------------------------- adapter kernels
// W_merged = RNbf16(W^ + s (L1 L2)^T), one CTA per 128 x 128 output tile.
size_t merge_smem_bytes(int r);
cudaError_t launch_adapter_merge(const uint8_t* codes, const uint8_t* c2, const float* c1, int format, int scale_codec,
                                 int64_t N, int64_t K, const uint16_t* L1, const uint16_t* L2, int r, float s,
                                 uint16_t* out, cudaStream_t st);
// AdamW step; sc = lr, b1, 1-b1, b2, 1-b2, eps, wd, 1-b1^t, 1-b2^t (fp32).
cudaError_t launch_adamw(float* p, uint16_t* pb, const float* g, float* m, float* v, int64_t n, const float* sc,
                         cudaStream_t st);

// ------------------------------------------------ MXFP4 and dropout kernels
// Dropout as the kernels take it: keep where the element's 16 random bits are
// at least `threshold`; `inv` = 65536 / (65536 - threshold).
struct DropArgs {
  uint32_t threshold;  // 0: nothing is dropped
  float inv;
  uint64_t seed, offset;
  const uint64_t* offset_dev;  // added to offset when not null
};

cudaError_t launch_mx_quantize(const void* X, int dtype, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                               int* status, cudaStream_t st);
// X [R][C] -> the MXFP4 form of its transpose [C][R].
cudaError_t launch_mx_quantize_t(const void* X, int dtype, int64_t R, int64_t C, uint8_t* codes, uint8_t* scales,
                                 int* status, int sms, cudaStream_t st);
cudaError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int dtype,
                              void* out, cudaStream_t st);
cudaError_t launch_dropout(const void* X, int dtype, int64_t n, const DropArgs& d, void* out, int sms, cudaStream_t st);

// bf16 terms of the LoRA term's token side (s T or the scaled dT) in a product.
// One, its rounding to bf16, would leave an error of up to 2^-8 of the LoRA
// term, as large as the rounding of the result where that term carries it (1.83e-3
// of dX of 1088 x 256 x 64, r = 16, in place of 1.65e-3); two leave 2^-16.
constexpr int kLoraTerms = 2;

// D[col][row] = sum_k A[row, k] B[col, k] (+ the LoRA term, masked when
// drop.threshold > 0), A and B in MXFP4.
struct MxGemmArgs {
  CUtensorMap tmA;   // codes of A, uint8 [rows][K/2], box 128 x 128, 128-byte swizzle
  CUtensorMap tmB;   // codes of B, uint8 [cols][K/2], box 128 x BN
  CUtensorMap tmAx;  // LoRA term: A side, bf16 (K- or MN-major per a_mn_ext)
  CUtensorMap tmBx;  // LoRA term: B side, bf16 (r, kLoraTerms, cols), box 64 x 1 x BN
  const uint8_t* sfA;  // tiled scales
  const uint8_t* sfB;
  int rows, cols;
  int64_t K;
  int kt;            // scale tiles along K
  int kb;            // 256-wide reduction blocks
  int r;             // rank of the LoRA term (0: none)
  int a_mn_ext;
  void* out;         // [cols][ldo]
  int64_t ldo;
  int out_f32;
  DropArgs drop;     // mask of the LoRA term at element col * ldo + row
  int* status;
  uint64_t wait_ns;
  int stall;
};

struct MxGemmPlan {
  int BN;
  int m_tiles, n_tiles, cluster;
};
MxGemmPlan plan_mx_gemm(int64_t rows, int64_t cols, int64_t K, int num_sms);
// dependent: starts while the kernel before it on the stream (which writes
// the tokens' side) still runs.
cudaError_t launch_mx_gemm(const MxGemmArgs& a, const MxGemmPlan& p, bool dependent, cudaStream_t st);

// The same product on persistent CTA pairs, tokens on the lanes:
// out[row][col] = sum_k A[row, k] B[col, k] (+ LoRA term), 256 x 256 tiles.
struct MxPairArgs {
  CUtensorMap tmA;   // codes of A (tokens), box 128 x 128, 128-byte swizzle
  CUtensorMap tmB;   // codes of B (weight), the same
  CUtensorMap tmSA;  // tiled scales as uint32 [row tiles][kt * 128], box 256 x 1
  CUtensorMap tmSB;  // the same, box 256 x 2
  CUtensorMap tmAx;  // LoRA term: bf16 (r, kLoraTerms, rows), box 64 x 1 x 128
  CUtensorMap tmBx;  // LoRA term: B side (K- or MN-major per b_mn_ext)
  CUtensorMap tmOut; // bf16 output [rows][ldo], box 64 x 32, 128-byte swizzle
  int rows, cols;
  int64_t K;
  int kb;            // 256-wide reduction blocks
  int r;             // rank of the LoRA term (0: none)
  int b_mn_ext;
  void* out;         // [rows][ldo]
  int64_t ldo;
  int out_f32;
  DropArgs drop;     // mask of the LoRA term at element row * ldo + col
  uint4* keep;       // if set: its bits, [rows][128-column tiles of ldo], 16 bytes each
  int* status;
};
cudaError_t launch_mx_gemm_pair(const MxPairArgs& a, int num_sms, bool dependent, cudaStream_t st);

// Quantise X and form D = drop(X).L in one pass (mx_prep.cu).
// What becomes of D.
struct MxPrepFinish {
  int64_t M;
  float* T;             // alpha D (may be null)
  float alpha;
  uint16_t* out;        // `terms` bf16 terms of beta D
  int terms;
  float beta;
  const float* T_in;    // when not null: out2 = three bf16 terms of gamma T_in
  uint16_t* out2;
  float gamma;
  const float* part;    // from here filled by the launch
  int r;
  int64_t units;
  int units_per_tile, grid;
};
struct MxPrepArgs {
  CUtensorMap tmX;      // bf16 [M][C], box 64 x 128, 128-byte swizzle
  CUtensorMap tmL;      // L1 [C][r] (l_mn: box 64 x 64) or L2 [r][C] (box 64 x r16)
  CUtensorMap tmCodes;  // codes [M][C / 2], box 128 x 128, 128-byte swizzle
  uint8_t* scales;
  int kt;               // scale tiles along C
  int64_t cols;
  int r, r16, l_mn;     // r16: r rounded up to 16
  int64_t units;
  int units_per_tile;
  int direct;
  float* part;
  MxPrepFinish fin;
  DropArgs drop;
  int* status;
};
int mx_prep_max_cluster();
cudaError_t launch_mx_prep(MxPrepArgs& a, const MxPrepPlan& p, cudaStream_t st);

// Adapter gradients (mx_grad.cu): problem 0 is dL1 = drop(X)^T.u, problem 1
// dL2 = (dY^T.v)^T, either may be absent (cols 0).
struct MxGradProblem {
  CUtensorMap tmZ;  // X or dY, bf16 [M][cols], box 64 x 64, 128-byte swizzle
  CUtensorMap tmV;  // bf16 [M][3r], the same box
  int64_t cols;
  int transposed;   // out is [r][cols], else [cols][r]
  float* out;
};
struct MxGradArgs {
  MxGradProblem p[2];
  int M, r;
  MxGradShare sh;
  int piece, pieces;
  float* part;         // slots, the tiles of problem 0 first
  int n16, nbuf;       // columns of an accumulator (3r up to 16), accumulators
  int vboxes, stages;
  DropArgs drop;       // mask of X
  const uint8_t* keep; // its bits as the product of dX left them, or null: evaluated
  int* status;
};
cudaError_t launch_mx_grad(MxGradArgs& a, const MxGradPlan& p, cudaStream_t st);

// scale * in [M][r] as three bf16 terms [M][3r] (their sum is exact in fp32).
cudaError_t launch_split3(const float* in, int64_t M, int r, float scale, uint16_t* out, int sms, cudaStream_t st);

}  // namespace qnf4
