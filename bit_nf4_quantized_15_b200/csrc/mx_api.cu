// The C ABI of the MXFP4 calls and of dropout (include/qlora_nf4.h):
// argument checks, tensor maps, workspace layout and launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/qlora_nf4.h"
#include "internal.h"

using namespace qnf4;

namespace {

bool ok16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool all16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!ok16(p)) return false;
  return true;
}
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int64_t kMaxDim = 1 << 24;

bool mx_shape_ok(int64_t rows, int64_t cols) {
  return rows >= 1 && cols >= 32 && cols % 32 == 0 && rows <= kMaxDim && cols <= kMaxDim &&
         ((rows + 127) / 128) * ((cols + 127) / 128) <= 0x3FFFFFFF;
}
bool rank_ok(int r) { return r == 0 || (r >= 8 && r <= 128 && r % 8 == 0); }
bool dtype_ok(int d) { return d == QLORA_DTYPE_BF16 || d == QLORA_DTYPE_F16 || d == QLORA_DTYPE_F32; }

size_t codes_bytes(int64_t rows, int64_t cols) { return (size_t)(rows * (cols / 2)); }
size_t scales_bytes(int64_t rows, int64_t cols) {
  return (size_t)((rows + 127) / 128) * (size_t)((cols + 127) / 128) * 512;
}

// Kernel arguments of a dropout configuration (NULL: none).
int drop_args(const qlora_dropout_config* c, DropArgs* d) {
  std::memset(d, 0, sizeof(*d));
  d->inv = 1.0f;
  if (!c) return QLORA_OK;
  if (!(c->p >= 0.0 && c->p < 1.0)) return QLORA_ERR_DROPOUT;
  const long t = std::lrint(c->p * 65536.0);
  if (t >= 65536) return QLORA_ERR_DROPOUT;
  d->threshold = (uint32_t)t;
  d->inv = (float)(65536.0 / (double)(65536 - t));
  d->seed = c->seed;
  d->offset = c->offset;
  d->offset_dev = c->offset_dev;
  if (reinterpret_cast<uintptr_t>(c->offset_dev) & 7u) return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

// The LoRA term of a product: u [M][kLoraTerms of `terms`][r] bf16, whose terms
// add up to the fp32 operand, times the feature side v, MN-major
// ([r][features]) or K-major ([features][r]).
struct LoraTerm {
  const uint16_t* u;
  int terms;
  const uint16_t* v;
  int v_mn, r;
};

// u as (r, kLoraTerms, M); a box is 64 x 1 x `rows`, zeros past r.
int map_terms(CUtensorMap* m, const LoraTerm& l, int64_t M, int rows) {
  return make_map3(m, l.u, (uint64_t)l.r, kLoraTerms, (uint64_t)M, (uint64_t)l.r * 2, (uint64_t)l.r * 2 * l.terms, 64,
                   1, (uint32_t)rows);
}

// Scales as a map of uint32 [row tiles][kt * 128]: a box is two tiles of
// `tiles` row ranges.
int map_scales(CUtensorMap* m, const uint8_t* scales, int64_t rows, int64_t K, int tiles) {
  return make_map(m, scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, (uint64_t)((K + 127) / 128) * 128,
                  (uint64_t)((rows + 127) / 128), 256, (uint32_t)tiles, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// out [M][N] = x w^T (+ the LoRA term), x = (xc, xs) the tokens, w = (wc, ws)
// the features.  *keep, if given: where the mask's bits may be left; null after
// the call if they were not.
//
// CTA pairs when more than a quarter of the SMs would have one of their 256 x
// 256 tiles, else tiles of 128 features split over clusters.  Both measured:
// 1024 x 4096 x 4096 (64 tiles) 14.0 us on pairs, 16.0 on clusters; 256 x
// 11008 x 4096 (43) 15.6 and 16.2; 512 x 4096 x 4096 (32) 13.5 and 12.2; but
// 128 x 22016 x 8192 (86, half of each empty) 36.8 and 34.3.
int product(const uint8_t* xc, const uint8_t* xs, int64_t M, const uint8_t* wc, const uint8_t* ws, int64_t N,
            int64_t K, const LoraTerm* lora, const DropArgs& drop, uint8_t** keep, void* out, int out_f32, int* status,
            int sms, bool dependent, cudaStream_t st) {
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t stall_ns = take_stall_request();
  if (M > 128 && ((M + 255) / 256) * ((N + 255) / 256) > sms / 4 && !stall_ns) {
    MxPairArgs g;
    std::memset(&g, 0, sizeof(g));
    if (make_map(&g.tmA, xc, u8, 1, (uint64_t)K / 2, (uint64_t)M, 128, 128, sw) ||
        make_map(&g.tmB, wc, u8, 1, (uint64_t)K / 2, (uint64_t)N, 128, 128, sw) || map_scales(&g.tmSA, xs, M, K, 1) ||
        map_scales(&g.tmSB, ws, N, K, 2) || (!out_f32 && map_operand(&g.tmOut, out, 0, M, N, 32)))
      return QLORA_ERR_CUDA;
    if (lora) {
      if (map_terms(&g.tmAx, *lora, M, 128) || map_operand(&g.tmBx, lora->v, lora->v_mn, N, lora->r, 128))
        return QLORA_ERR_CUDA;
      g.r = lora->r;
      g.b_mn_ext = lora->v_mn;
      g.drop = drop;
      if (keep && drop.threshold) g.keep = reinterpret_cast<uint4*>(*keep);
    }
    g.rows = (int)M;
    g.cols = (int)N;
    g.K = K;
    g.kb = (int)((K + 255) / 256);
    g.out = out;
    g.ldo = N;
    g.out_f32 = out_f32;
    g.status = status;
    return launch_mx_gemm_pair(g, sms, dependent, st) == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
  }
  if (keep) *keep = nullptr;
  const MxGemmPlan p = plan_mx_gemm(N, M, K, sms);
  MxGemmArgs g;
  std::memset(&g, 0, sizeof(g));
  if (make_map(&g.tmA, wc, u8, 1, (uint64_t)K / 2, (uint64_t)N, 128, 128, sw) ||
      make_map(&g.tmB, xc, u8, 1, (uint64_t)K / 2, (uint64_t)M, 128, (uint32_t)p.BN, sw))
    return QLORA_ERR_CUDA;
  if (lora) {
    if (map_operand(&g.tmAx, lora->v, lora->v_mn, N, lora->r, 128) || map_terms(&g.tmBx, *lora, M, p.BN))
      return QLORA_ERR_CUDA;
    g.r = lora->r;
    g.a_mn_ext = lora->v_mn;
    g.drop = drop;
  }
  g.sfA = ws;
  g.sfB = xs;
  g.rows = (int)N;
  g.cols = (int)M;
  g.K = K;
  g.kt = (int)((K + 127) / 128);
  g.kb = (int)((K + 255) / 256);
  g.out = out;
  g.ldo = N;
  g.out_f32 = out_f32;
  g.status = status;
  g.stall = stall_ns != 0;
  g.wait_ns = stall_ns;
  return launch_mx_gemm(g, p, dependent, st) == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

// Q(X) and the partial sums of D = drop(X).L (L MN-major [C][r] or K-major [r][C]).
int prep(const uint16_t* X, int64_t M, int64_t C, const uint16_t* L, int l_mn, int r, const DropArgs& d,
         uint8_t* codes, uint8_t* scales, float* part, const MxPrepPlan& p, const MxPrepFinish& fin, int* status,
         cudaStream_t st) {
  MxPrepArgs a;
  std::memset(&a, 0, sizeof(a));
  const int r16 = (r + 15) / 16 * 16;
  if (map_operand(&a.tmX, X, 0, M, C, 128) ||
      (l_mn ? map_operand(&a.tmL, L, 1, r, C, 64) : map_operand(&a.tmL, L, 0, r, C, r16)) ||
      make_map(&a.tmCodes, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)C / 2, (uint64_t)M, 128, 128,
               CU_TENSOR_MAP_SWIZZLE_128B))
    return QLORA_ERR_CUDA;
  a.scales = scales;
  a.kt = (int)((C + 127) / 128);
  a.cols = C;
  a.r = r;
  a.l_mn = l_mn;
  a.part = part;
  a.fin = fin;
  a.drop = d;
  a.status = status;
  return launch_mx_prep(a, p, st) == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

// Workspace of the linear layer (offsets in bytes).  Forward and backward use
// the same regions for their own data.  Every region's size only grows with M,
// so a workspace sized for the largest batch holds the smaller ones:
//   q      MXFP4 of X (forward) or dY (backward): codes, then scales
//   u, v   bf16 [M][3r]: the scaled dT (u) and s T (v) in three terms; the
//          forward keeps s T in u, [M][2r], in two
//   keep   bits of the dropout mask, [M][128-column tiles of K], 16 bytes each,
//          from the product of dX to the kernel of dL1
//   part   fp32 partial sums of the adapter products
// The partial sums are those of a device without clusters of 16, the most, so
// that asking for a size makes no context.
struct MxWs {
  size_t q_scales, u, v, keep, part, total;
};

MxWs mx_ws(int64_t M, int64_t N, int64_t K, int r, int sms) {
  MxWs w{};
  const size_t qk = up256(codes_bytes(M, K)), qn = up256(codes_bytes(M, N));
  w.q_scales = qk > qn ? qk : qn;
  const size_t sk = up256(scales_bytes(M, K)), sn = up256(scales_bytes(M, N));
  size_t o = w.q_scales + (sk > sn ? sk : sn);
  if (r) {
    w.u = o;
    o += up256((size_t)M * r * 6);
    w.v = o;
    o += up256((size_t)M * r * 6);
    w.keep = o;
    o += up256((size_t)M * ((K + 127) / 128) * 16);
    w.part = o;
    o += up256(std::max({plan_mx_prep(M, K, r, sms, 8).part_bytes, plan_mx_prep(M, N, r, sms, 8).part_bytes,
                         mx_grad_part_bound(M, K, N, r, sms)}));
  }
  w.total = o;
  return w;
}

bool linear_shape_ok(int64_t M, int64_t N, int64_t K, int64_t n_mult) {
  return M >= 1 && M <= kMaxDim && N >= n_mult && N % n_mult == 0 && N <= kMaxDim && mx_shape_ok(M, K) &&
         mx_shape_ok(N, K);
}

}  // namespace

extern "C" {

int qlora_mx_storage_bytes(int64_t rows, int64_t cols, size_t* cb, size_t* sb) {
  if (!mx_shape_ok(rows, cols)) return QLORA_ERR_MX_SHAPE;
  if (cb) *cb = codes_bytes(rows, cols);
  if (sb) *sb = scales_bytes(rows, cols);
  return QLORA_OK;
}

int qlora_mx_quantize(const void* X, int dtype, int64_t rows, int64_t cols, int transpose,
                      const qlora_mx_tensor* out, int* status_dev, qlora_stream_t stream) {
  if (!X || !out || !out->codes || !out->scales) return QLORA_ERR_NULL;
  if (!dtype_ok(dtype)) return QLORA_ERR_DTYPE;
  if (!(transpose ? mx_shape_ok(cols, rows) && cols % 8 == 0 : mx_shape_ok(rows, cols))) return QLORA_ERR_MX_SHAPE;
  if (!all16({X, out->codes, out->scales})) return QLORA_ERR_ALIGN;
  DevInfo di;
  if (int rc = current_device_info(&di)) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      transpose ? launch_mx_quantize_t(X, dtype, rows, cols, out->codes, out->scales, status_dev, di.sms, st)
                : launch_mx_quantize(X, dtype, rows, cols, out->codes, out->scales, status_dev, st);
  return e == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

int qlora_mx_dequant(const qlora_mx_tensor* t, void* out, int dtype, qlora_stream_t stream) {
  if (!t || !t->codes || !t->scales || !out) return QLORA_ERR_NULL;
  if (dtype != QLORA_DTYPE_BF16 && dtype != QLORA_DTYPE_F32) return QLORA_ERR_DTYPE;
  if (!mx_shape_ok(t->rows, t->cols)) return QLORA_ERR_MX_SHAPE;
  if (!all16({t->codes, t->scales, out})) return QLORA_ERR_ALIGN;
  DevInfo di;
  if (int rc = current_device_info(&di)) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return launch_mx_dequant(t->codes, t->scales, t->rows, t->cols, dtype, out, st) == cudaSuccess ? QLORA_OK
                                                                                                 : QLORA_ERR_CUDA;
}

int qlora_mx_matmul(const qlora_mx_tensor* a, const qlora_mx_tensor* b, void* out, int dtype, int* status_dev,
                    qlora_stream_t stream) {
  if (!a || !b || !a->codes || !a->scales || !b->codes || !b->scales || !out) return QLORA_ERR_NULL;
  if (dtype != QLORA_DTYPE_BF16 && dtype != QLORA_DTYPE_F32) return QLORA_ERR_DTYPE;
  if (a->cols != b->cols || !linear_shape_ok(a->rows, b->rows, a->cols, 8)) return QLORA_ERR_MX_SHAPE;
  if (!all16({a->codes, a->scales, b->codes, b->scales, out})) return QLORA_ERR_ALIGN;
  DevInfo di;
  if (int rc = current_device_info(&di)) return rc;
  return product(a->codes, a->scales, a->rows, b->codes, b->scales, b->rows, a->cols, nullptr, DropArgs{}, nullptr, out,
                 dtype == QLORA_DTYPE_F32, status_dev, di.sms, false, reinterpret_cast<cudaStream_t>(stream));
}

int qlora_dropout(const void* X, int dtype, int64_t n, const qlora_dropout_config* cfg, void* out,
                  qlora_stream_t stream) {
  if (!X || !cfg || !out) return QLORA_ERR_NULL;
  if (!dtype_ok(dtype)) return QLORA_ERR_DTYPE;
  if (n < 0) return QLORA_ERR_SHAPE;
  DropArgs d;
  if (int rc = drop_args(cfg, &d)) return rc;
  if (!all16({X, out})) return QLORA_ERR_ALIGN;
  const size_t bytes = (size_t)n * (dtype == QLORA_DTYPE_F32 ? 4 : 2);
  if (out != X && overlap(X, bytes, out, bytes)) return QLORA_ERR_OVERLAP;
  if (n == 0) return QLORA_OK;
  DevInfo di;
  if (int rc = current_device_info(&di)) return rc;
  return launch_dropout(X, dtype, n, d, out, di.sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? QLORA_OK
             : QLORA_ERR_CUDA;
}

size_t qlora_mx_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int r) {
  if (!linear_shape_ok(M, N, K, 8) || !rank_ok(r)) return 0;
  DevInfo di;
  if (current_device_info(&di)) di.sms = 148;
  return mx_ws(M, N, K, r, di.sms).total;
}

int qlora_mx_linear_fwd(const uint16_t* X, int64_t M, const qlora_mx_tensor* w, const uint16_t* L1,
                        const uint16_t* L2, int r, float s, const qlora_dropout_config* drop, uint16_t* Y,
                        float* T_save, void* ws, size_t ws_bytes, int* status_dev, qlora_stream_t stream) {
  if (!X || !w || !w->codes || !w->scales || !Y || !ws) return QLORA_ERR_NULL;
  if (!rank_ok(r)) return QLORA_ERR_RANK;
  if (r && (!L1 || !L2 || !T_save)) return QLORA_ERR_NULL;
  const int64_t N = w->rows, K = w->cols;
  if (!linear_shape_ok(M, N, K, 8)) return QLORA_ERR_MX_SHAPE;
  DropArgs d;
  if (int rc = drop_args(drop, &d)) return rc;
  if (!all16({X, w->codes, w->scales, L1, L2, Y, T_save, ws})) return QLORA_ERR_ALIGN;
  DevInfo di;
  if (int rc = current_device_info(&di)) return rc;
  const MxWs lay = mx_ws(M, N, K, r, di.sms);
  if (ws_bytes < lay.total) return QLORA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* wb = static_cast<uint8_t*>(ws);
  uint16_t* sT = reinterpret_cast<uint16_t*>(wb + lay.u);

  if (r) {
    float* part = reinterpret_cast<float*>(wb + lay.part);
    MxPrepFinish f;
    std::memset(&f, 0, sizeof(f));
    f.M = M;
    f.T = T_save;
    f.alpha = d.inv;
    f.out = sT;
    f.terms = kLoraTerms;
    f.beta = s * d.inv;
    const MxPrepPlan p = plan_mx_prep(M, K, r, di.sms, mx_prep_max_cluster());
    if (int rc = prep(X, M, K, L1, 1, r, d, wb, wb + lay.q_scales, part, p, f, status_dev, st)) return rc;
  } else if (launch_mx_quantize(X, QLORA_DTYPE_BF16, M, K, wb, wb + lay.q_scales, status_dev, st) != cudaSuccess) {
    return QLORA_ERR_CUDA;
  }
  const LoraTerm lora{sT, kLoraTerms, L2, 1, r};
  return product(wb, wb + lay.q_scales, M, w->codes, w->scales, N, K, r ? &lora : nullptr, DropArgs{}, nullptr, Y, 0,
                 status_dev, di.sms, true, st);
}

int qlora_mx_linear_bwd(const uint16_t* dY, const uint16_t* X, int64_t M, const float* T_saved,
                        const qlora_mx_tensor* wt, int64_t N, int64_t K, const uint16_t* L1, const uint16_t* L2,
                        int r, float s, const qlora_dropout_config* drop, uint16_t* dX, float* dL1, float* dL2,
                        void* ws, size_t ws_bytes, int* status_dev, qlora_stream_t stream) {
  if (!dY || !ws) return QLORA_ERR_NULL;
  if (!rank_ok(r)) return QLORA_ERR_RANK;
  if (dX && (!wt || !wt->codes || !wt->scales)) return QLORA_ERR_NULL;
  if (!r && (dL1 || dL2)) return QLORA_ERR_RANK;
  if (r && (!L1 || !L2 || (dL1 && !X) || (dL2 && !T_saved))) return QLORA_ERR_NULL;
  if (!linear_shape_ok(M, N, K, 32)) return QLORA_ERR_MX_SHAPE;
  if (dX && (wt->rows != K || wt->cols != N)) return QLORA_ERR_MX_SHAPE;
  DropArgs d;
  if (int rc = drop_args(drop, &d)) return rc;
  if (!all16({dY, X, T_saved, L1, L2, dX, dL1, dL2, ws})) return QLORA_ERR_ALIGN;
  if (dX && !all16({wt->codes, wt->scales})) return QLORA_ERR_ALIGN;
  // dX is written before the adapter gradients read X and dY
  const size_t mk = (size_t)M * K * 2, mn = (size_t)M * N * 2;
  if (dX && ((dL1 && overlap(dX, mk, X, mk)) || (dL2 && overlap(dX, mk, dY, mn)))) return QLORA_ERR_OVERLAP;
  DevInfo di;
  if (int rc = current_device_info(&di)) return rc;
  const MxWs lay = mx_ws(M, N, K, r, di.sms);
  if (ws_bytes < lay.total) return QLORA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* wb = static_cast<uint8_t*>(ws);
  uint16_t* sdT = reinterpret_cast<uint16_t*>(wb + lay.u);
  uint16_t* sT = reinterpret_cast<uint16_t*>(wb + lay.v);
  float* part = reinterpret_cast<float*>(wb + lay.part);

  // Q(dY) and dT = dY.L2^T, kept as three bf16 terms of s dT / (1 - p); with
  // them s T in three terms
  if (r && (dX || dL1)) {
    MxPrepFinish f;
    std::memset(&f, 0, sizeof(f));
    f.M = M;
    f.out = sdT;
    f.terms = 3;
    f.beta = s * d.inv;
    f.T_in = dL2 ? T_saved : nullptr;
    f.out2 = sT;
    f.gamma = s;
    const MxPrepPlan p = plan_mx_prep(M, N, r, di.sms, mx_prep_max_cluster());
    if (int rc = prep(dY, M, N, L2, 0, r, DropArgs{}, wb, wb + lay.q_scales, part, p, f, status_dev, st)) return rc;
  } else if (dX &&
             launch_mx_quantize(dY, QLORA_DTYPE_BF16, M, N, wb, wb + lay.q_scales, status_dev, st) != cudaSuccess) {
    return QLORA_ERR_CUDA;
  }
  // the mask's bits, if dX's product leaves them for dL1
  uint8_t* keep = dX && dL1 && d.threshold ? wb + lay.keep : nullptr;
  if (dX) {
    const LoraTerm lora{sdT, 3, L1, 0, r};
    if (int rc = product(wb, wb + lay.q_scales, M, wt->codes, wt->scales, K, N, r ? &lora : nullptr, d,
                         keep ? &keep : nullptr, dX, 0, status_dev, di.sms, true, st))
      return rc;
  }
  if (dL1 || dL2) {
    if (dL2 && !dX && !dL1 && launch_split3(T_saved, M, r, s, sT, di.sms, st) != cudaSuccess) return QLORA_ERR_CUDA;
    const MxGradMask mask = !d.threshold ? kMaskNone : keep ? kMaskBits : kMaskEvaluated;
    const MxGradPlan p = plan_mx_grad(M, dL1 ? K : 0, dL2 ? N : 0, r, mask, di.sms);
    MxGradArgs a;
    std::memset(&a, 0, sizeof(a));
    if (dL1 && (map_operand(&a.p[0].tmZ, X, 1, K, M, 64) || map_operand(&a.p[0].tmV, sdT, 1, 3 * r, M, 64)))
      return QLORA_ERR_CUDA;
    if (dL2 && (map_operand(&a.p[1].tmZ, dY, 1, N, M, 64) || map_operand(&a.p[1].tmV, sT, 1, 3 * r, M, 64)))
      return QLORA_ERR_CUDA;
    a.p[0].cols = K;
    a.p[0].out = dL1;
    a.p[1].cols = N;
    a.p[1].transposed = 1;
    a.p[1].out = dL2;
    a.M = (int)M;
    a.r = r;
    a.part = part;
    a.drop = d;
    a.keep = keep;
    a.status = status_dev;
    if (launch_mx_grad(a, p, st) != cudaSuccess) return QLORA_ERR_CUDA;
  }
  return QLORA_OK;
}

}  // extern "C"
