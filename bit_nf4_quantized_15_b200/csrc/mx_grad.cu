// Adapter gradients of the MXFP4 linear layer:
//
//   dL1 [K][r] = drop(X)^T . u      dL2 [r][N] = (dY^T . v)^T
//
// u and v [M][r] in fp32, held as three bf16 terms side by side ([M][3r]), so
// the tensor cores' products are those of the fp32 values.  Each sum runs
// over the tokens and reads all of X or dY: the bound is those bytes, with
// the terms' 6 r bytes a token read again (from L2) for every 128 columns.
//
// A unit is 128 columns of X or dY x 512 tokens: one accumulation in tensor
// memory (the tensor cores' truncation grows with the length of a sum, see
// mx_prep.cu), three groups of r columns wide; the sum warps add the groups,
// and units of one run to one another, with rounding.  One CTA per SM takes an equal
// run of units; both gradients are one launch, so that a small one fills the
// other's tail.  Runs end in partial slots that a second kernel adds in order.
//
// With dropout the X tile is masked in shared memory before the MMAs read it.
//
// Roles: warp 0 TMA producer, 1 MMA issuer, 4-7 sum, 8-15 mask.
#include "engine_util.cuh"
#include "mx_util.cuh"
#include "pair_util.cuh"
#include "philox.cuh"

namespace qnf4 {
namespace {

constexpr int kGThreads = 16 * 32;
constexpr int kGMaxS = 6;
constexpr int kGBudget = 220 * 1024;  // bytes of the stages
constexpr int kGPiece = 8;            // 64-token stages of a unit

QDEV int grad_owner(int64_t units, int grid, int64_t u) { return (int)(((u + 1) * grid - 1) / units); }

struct UnitAt {
  int prob;      // 0: dL1, 1: dL2
  int tile;      // 128-column tile
  int piece;     // 512-token piece
  bool last;     // no further piece of this tile in the run
};
QDEV UnitAt unit_at(const MxGradArgs& a, int64_t u, int64_t u_hi) {
  UnitAt x;
  x.prob = u >= a.units0;
  const int64_t v = x.prob ? u - a.units0 : u;
  x.tile = (int)(v / a.pieces);
  x.piece = (int)(v % a.pieces);
  x.last = x.piece + 1 == a.pieces || u + 1 == u_hi;
  return x;
}

__global__ void __launch_bounds__(kGThreads, 1) mx_grad_kernel(const __grid_constant__ MxGradArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage = 16384 + args.vboxes * 8192, kS = args.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kS * stage);
  uint64_t* ready = full + kGMaxS;
  uint64_t* empty = ready + kGMaxS;
  uint64_t* wfull = empty + kGMaxS;
  uint64_t* wempty = wfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(wempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const int grid = (int)gridDim.x;
  const int64_t u_lo = blockIdx.x * args.units / grid, u_hi = ((int64_t)blockIdx.x + 1) * args.units / grid;
  const int nbuf = args.nbuf;
  const uint32_t sum_col = (uint32_t)(nbuf * args.n16);

  if (tid == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(ready + s, 8);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(wfull + b, 1);
      mbar_init(wempty + b, 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int64_t u = u_lo; u < u_hi && ok; ++u) {
        const UnitAt x = unit_at(args, u, u_hi);
        const MxGradProblem& p = args.p[x.prob];
        const int t0 = x.piece * 64 * kGPiece, n = min(kGPiece, (args.M - t0 + 63) / 64);
        for (int i = 0; i < n; ++i) {
          if (!(ok = mbar_wait(empty + s, ph ^ 1u, abort_flag, args.status))) break;
          uint8_t* sa = smem + s * stage;
          mbar_arrive_expect_tx(full + s, (uint32_t)stage);
          for (int j = 0; j < 2; ++j) tma_load_2d(sa + 8192 * j, &p.tmZ, full + s, x.tile * 128 + 64 * j, t0 + 64 * i);
          for (int j = 0; j < args.vboxes; ++j) tma_load_2d(sa + 16384 + 8192 * j, &p.tmV, full + s, 64 * j, t0 + 64 * i);
          if (++s == kS) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    const int n1 = min(args.n16, 256), n2 = args.n16 - n1;
    const uint32_t id1 = idesc_bf16(128, 16, 1, 1) + ((uint32_t)((n1 - 16) >> 3) << 17);
    const uint32_t id2 = idesc_bf16(128, 16, 1, 1) + ((uint32_t)((n2 - 16) >> 3) << 17);  // used when n2 > 0
    const bool one = elect_one();
    int s = 0, b = 0;
    uint32_t ph = 0, wph = 0;
    bool ok = true;
    for (int64_t u = u_lo; u < u_hi && ok; ++u) {
      const UnitAt x = unit_at(args, u, u_hi);
      const bool masked = x.prob == 0 && args.drop.threshold;
      const int t0 = x.piece * 64 * kGPiece, n = min(kGPiece, (args.M - t0 + 63) / 64);
      if (!(ok = warp_poll(wempty + b, wph ^ 1u, abort_flag, args.status, lane))) break;
      const uint32_t d = tmem + (uint32_t)(b * args.n16);
      for (int i = 0; i < n; ++i) {
        if (!(ok = warp_poll((masked ? ready : full) + s, ph, abort_flag, args.status, lane))) break;
        tc_fence_after();
        if (one) {
          const uint8_t* sa = smem + s * stage;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            umma_bf16(d, operand_desc(sa, 1, kk), operand_desc(sa + 16384, 1, kk), id1, (i | kk) != 0);
            if (n2 > 0)
              umma_bf16(d + 256, operand_desc(sa, 1, kk), operand_desc(sa + 16384 + 4 * 8192, 1, kk), id2, (i | kk) != 0);
          }
          umma_commit(empty + s);
        }
        __syncwarp();
        if (++s == kS) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      if (one) umma_commit(wfull + b);
      __syncwarp();
      if (++b == nbuf) {
        b = 0;
        wph ^= 1u;
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------------ sum
    const int q4 = warp & 3;
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
    const int r = args.r, r16 = (r + 15) / 16 * 16;
    int b = 0;
    uint32_t wph = 0;
    bool first = true;
    for (int64_t u = u_lo; u < u_hi; ++u) {
      const UnitAt x = unit_at(args, u, u_hi);
      if (!warp_wait(wfull + b, wph, abort_flag, args.status, lane)) break;
      tc_fence_after();
      const MxGradProblem& p = args.p[x.prob];
      // this run's slot of the tile: its ordinal among the CTAs that share it
      const int64_t tile_u = (x.prob ? args.units0 : 0) + (int64_t)x.tile * args.pieces;
      const int ord = (int)blockIdx.x - grad_owner(args.units, grid, tile_u);
      float* slot = p.part + ((int64_t)x.tile * args.maxc + ord) * 128 * r;
      const int row = q4 * 32 + lane;
      for (int c = 0; c < r16; c += 16) {
        uint32_t v[16], w[16], z[16];
        const uint32_t at = tl + (uint32_t)(b * args.n16 + c);
        tmem_ld16(at, v);
        tmem_ld16(at + (uint32_t)r, w);
        tmem_ld16(at + 2u * (uint32_t)r, z);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          v[j] = __float_as_uint(__fadd_rn(__uint_as_float(v[j]), __fadd_rn(__uint_as_float(w[j]), __uint_as_float(z[j]))));
        if (!first) {
          tmem_ld16(tl + sum_col + (uint32_t)c, w);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__fadd_rn(__uint_as_float(v[j]), __uint_as_float(w[j])));
        }
        if (!x.last) {
          tmem_st16(tl + sum_col + (uint32_t)c, v);
        } else if (p.transposed) {  // slot [r][128]
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < r) slot[(c + j) * 128 + row] = __uint_as_float(v[j]);
        } else {  // slot [128][r]
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            if (c + j < r)
              *reinterpret_cast<uint4*>(slot + (int64_t)row * r + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(wempty + b);
      first = x.last;
      if (++b == nbuf) {
        b = 0;
        wph ^= 1u;
      }
    }
  } else if (warp >= 8 && args.drop.threshold) {
    // ----------------------------------------------------------------- mask
    // Units of dL1 come first in a run, so every stage up to the last masked
    // one is masked and the ready barriers' phases follow the ring's.
    const PhiloxKey key = philox_key(args.drop);
    const int t = tid & 255;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int64_t u = u_lo; u < u_hi && u < args.units0 && ok; ++u) {
      const UnitAt x = unit_at(args, u, u_hi);
      const int t0 = x.piece * 64 * kGPiece, n = min(kGPiece, (args.M - t0 + 63) / 64);
      for (int i = 0; i < n; ++i) {
        // 4 evaluations of this thread's chunks before the wait: they need no data
        uint32_t keep[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q = t + 256 * j, tok = (q >> 3) & 63, ch = q & 7, box = q >> 9;
          const int64_t e = (int64_t)(t0 + 64 * i + tok) * args.p[0].cols + x.tile * 128 + 64 * box + 8 * ch;
          keep[j] = keep8((uint64_t)e >> 3, key, args.drop.threshold);
        }
        if (!(ok = warp_wait(full + s, ph, abort_flag, args.status, lane))) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q = t + 256 * j, tok = (q >> 3) & 63, ch = q & 7, box = q >> 9;
          uint4* at = reinterpret_cast<uint4*>(smem + s * stage + 8192 * box + tok * 128 + ((ch ^ (tok & 7)) << 4));
          const uint4 v = *at;
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] &= ((keep[j] >> (2 * k)) & 1u ? 0xFFFFu : 0u) | ((keep[j] >> (2 * k + 1)) & 1u ? 0xFFFF0000u : 0u);
          *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(ready + s);
        if (++s == kS) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (tid == 0) {  // error path: let loads and MMAs still in flight finish
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 2000000ull) {
      }
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Both gradients from the slots of their tiles, in order.
__global__ void __launch_bounds__(256) mx_grad_finish_kernel(const __grid_constant__ MxGradArgs a, int grid) {
  const int64_t n0 = a.units0 ? a.p[0].cols * a.r : 0, n = n0 + (a.units > a.units0 ? a.p[1].cols * a.r : 0);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int prob = i >= n0;
    const MxGradProblem& p = a.p[prob];
    const int64_t k = prob ? i - n0 : i;
    // the outputs' own order: [cols][r], transposed [r][cols]
    const int64_t col = p.transposed ? k % p.cols : k / a.r;
    const int j = (int)(p.transposed ? k / p.cols : k % a.r);
    const int64_t tile = col >> 7, tile_u = (prob ? a.units0 : 0) + tile * a.pieces;
    const int nc = grad_owner(a.units, grid, tile_u + a.pieces - 1) - grad_owner(a.units, grid, tile_u);
    const float* s = p.part + tile * a.maxc * 128 * a.r + (p.transposed ? j * 128 + (col & 127) : (col & 127) * a.r + j);
    float d = s[0];
    for (int c = 1; c <= nc; ++c) d = __fadd_rn(d, s[(int64_t)c * 128 * a.r]);
    p.out[k] = d;
  }
}

}  // namespace

// Partial slots of one problem with `cols` columns in a launch of `units`.
MxGradPlan plan_mx_grad(int64_t M, int64_t cols0, int64_t cols1, int r, int num_sms) {
  MxGradPlan p{};
  p.pieces = (int)((M + 64 * kGPiece - 1) / (64 * kGPiece));
  const int64_t t0 = (cols0 + 127) / 128, t1 = (cols1 + 127) / 128;
  p.units0 = t0 * p.pieces;
  p.units = p.units0 + t1 * p.pieces;
  if (!p.units) return p;
  p.grid = (int)(p.units < num_sms ? p.units : num_sms);
  const int64_t per = p.units / p.grid;
  p.maxc = (int)((p.pieces + per - 1) / per) + 1;
  if (p.maxc > p.grid) p.maxc = p.grid;
  p.part0_bytes = (size_t)t0 * p.maxc * 128 * r * sizeof(float);
  p.part_bytes = p.part0_bytes + (size_t)t1 * p.maxc * 128 * r * sizeof(float);
  p.n16 = (3 * r + 15) / 16 * 16;
  const int r16 = (r + 15) / 16 * 16;
  p.nbuf = 2 * p.n16 + r16 <= 512 ? 2 : 1;
  p.vboxes = (p.n16 + 63) / 64;
  const int stage = 16384 + p.vboxes * 8192;
  p.stages = kGBudget / stage < kGMaxS ? kGBudget / stage : kGMaxS;
  return p;
}

cudaError_t launch_mx_grad(MxGradArgs& a, const MxGradPlan& p, cudaStream_t st) {
  a.units0 = p.units0;
  a.units = p.units;
  a.pieces = p.pieces;
  a.maxc = p.maxc;
  a.n16 = p.n16;
  a.nbuf = p.nbuf;
  a.vboxes = p.vboxes;
  a.stages = p.stages;
  const int smem = p.stages * (16384 + p.vboxes * 8192) + 512 + 1024;
  cudaError_t err = cudaFuncSetAttribute(mx_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kGBudget + 512 + 1024);
  if (err != cudaSuccess) return err;
  mx_grad_kernel<<<p.grid, kGThreads, smem, st>>>(a);
  count_launches(1);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const int64_t n = ((p.units0 ? a.p[0].cols : 0) + (p.units > p.units0 ? a.p[1].cols : 0)) * a.r;
  const int64_t want = (n + 255) / 256;
  mx_grad_finish_kernel<<<(unsigned)(want < 2368 ? want : 2368), 256, 0, st>>>(a, p.grid);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace qnf4
