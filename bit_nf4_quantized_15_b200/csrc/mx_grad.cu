// Adapter gradients of the MXFP4 linear layer:
//
//   dL1 [K][r] = drop(X)^T . u      dL2 [r][N] = (dY^T . v)^T
//
// u and v [M][r] in fp32, held as three bf16 terms side by side ([M][3r]), so
// the tensor cores' products are those of the fp32 values.  Each sum runs
// over the tokens and reads all of X or dY: the bound is those bytes, with
// the terms' 6 r bytes a token read again (from L2) for every 128 columns.
//
// A unit is 128 columns of X or dY x up to 512 tokens: one accumulation in
// tensor memory (the tensor cores' truncation grows with the length of a sum,
// see mx_prep.cu), three groups of r columns wide; the sum warps add the
// groups, and units of one run to one another, with rounding.  One CTA per SM
// takes a run of units of equal cost; both gradients are one launch, so that a
// small one fills the other's tail.  A tile that is one unit is written at
// once; other runs end in partial slots that a second kernel adds in order.
//
// With dropout the X tile is masked in shared memory before the MMAs read it:
// by the bits that the product of dX has left, an eighth of a byte an element,
// or, without them (dL1 alone, few tokens), by evaluating the generator.
//
// Measured, dL2 of 8192 x 8192 with r = 64: 36 us (35 before infinities were told
// apart), 134 MB at 3.8 TB/s (4.5 by the slope over longer ones).  Without the
// loads of the terms the slope is 5.9 TB/s: of a stage's 40 KB the terms are 24,
// and L2 gives them out at about 11 TB/s.  An evaluated mask costs 1024
// evaluations a stage, 90 cycles each for a warp and scheduler, on the pipes of
// the masking: backward of 4096 x 4096 x 4096 with dropout 96 us, with the bits
// 93.5 (95 since dX takes two terms of dT).
//
// Roles: warp 0 TMA producer, 1 MMA issuer, 4-7 sum, 8-23 mask.
#include "engine_util.cuh"
#include "launch.cuh"
#include "mx_util.cuh"
#include "pair_util.cuh"
#include "philox.cuh"

namespace qnf4 {
namespace {

constexpr int kGThreads = 24 * 32;
struct UnitAt {
  int prob;      // 0: dL1, 1: dL2
  int tile;      // 128-column tile
  int piece;     // piece of the tokens
  bool last;     // no further piece of this tile in the run
};
QDEV UnitAt unit_at(const MxGradArgs& a, int64_t u, int64_t u_hi) {
  UnitAt x;
  x.prob = u >= a.sh.units0;
  const int64_t v = x.prob ? u - a.sh.units0 : u;
  x.tile = (int)(v / a.pieces);
  x.piece = (int)(v % a.pieces);
  x.last = x.piece + 1 == a.pieces || u + 1 == u_hi;
  return x;
}

// The sum of the three terms' groups.  Where the first is an Inf or NaN it is
// the sum: the other terms may be zero, and an infinite X or dY makes NaN of
// them.
QDEV float add_groups(uint32_t v, uint32_t w, uint32_t z) {
  const float first = __uint_as_float(v);
  return (v & 0x7F800000u) == 0x7F800000u
             ? first
             : __fadd_rn(first, __fadd_rn(__uint_as_float(w), __uint_as_float(z)));
}

// Eight bf16 of which those with a bit in `b` stay.  The products put four
// bits into the sign bits of four bytes (their copies do not overlap), from
// where a byte permutation spreads them.
QDEV uint4 keep_bits(uint4 v, uint32_t b) {
  const uint32_t lo = (b & 15u) * 0x10204080u, hi = (b >> 4) * 0x10204080u;
  const auto spread = [](uint32_t x, uint32_t sel) {
    uint32_t m;
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(m) : "r"(x), "r"(sel));
    return m;
  };
  return make_uint4(v.x & spread(lo, 0x9988u), v.y & spread(lo, 0xBBAAu), v.z & spread(hi, 0x9988u),
                    v.w & spread(hi, 0xBBAAu));
}

__global__ void __launch_bounds__(kGThreads, 1) mx_grad_kernel(const __grid_constant__ MxGradArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage = 16384 + args.vboxes * 8192, kS = args.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kS * stage);
  uint64_t* ready = full + kGradMaxStages;
  uint64_t* empty = ready + kGradMaxStages;
  uint64_t* wfull = empty + kGradMaxStages;
  uint64_t* wempty = wfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(wempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const int64_t u_lo = grad_first(args.sh, blockIdx.x), u_hi = grad_first(args.sh, (int64_t)blockIdx.x + 1);
  const int nbuf = args.nbuf;
  const uint32_t sum_col = (uint32_t)(nbuf * args.n16);

  if (warp == 0) {  // a barrier a lane
    if (lane < kS) {
      mbar_init(full + lane, 1);
      mbar_init(ready + lane, 8);
      mbar_init(empty + lane, 1);
    } else if (lane < kS + 2) {
      mbar_init(wfull + lane - kS, 1);
      mbar_init(wempty + lane - kS, 4);
    } else if (lane == kS + 2) {
      *abort_flag = 0;
      if (args.sh.units0) {
        tma_prefetch_desc(&args.p[0].tmZ);
        tma_prefetch_desc(&args.p[0].tmV);
      }
      if (args.sh.units > args.sh.units0) {
        tma_prefetch_desc(&args.p[1].tmZ);
        tma_prefetch_desc(&args.p[1].tmV);
      }
    }
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
  pdl_trigger();  // not before this CTA has its tensor memory: a dependent CTA must not take it first

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      pdl_wait();
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int64_t u = u_lo; u < u_hi && ok; ++u) {
        const UnitAt x = unit_at(args, u, u_hi);
        const MxGradProblem& p = args.p[x.prob];
        const int t0 = x.piece * 64 * args.piece, n = min(args.piece, (args.M - t0 + 63) / 64);
        for (int i = 0; i < n; ++i) {
          if (!(ok = mbar_wait_backoff(empty + s, ph ^ 1u, abort_flag, args.status, 20))) break;
          uint8_t* sa = smem + s * stage;
          mbar_arrive_expect_tx(full + s, (uint32_t)stage);
          for (int j = 0; j < 2; ++j) tma_load_2d(sa + 8192 * j, &p.tmZ, full + s, x.tile * 128 + 64 * j, t0 + 64 * i);
          for (int j = 0; j < args.vboxes; ++j)
            tma_load_2d(sa + 16384 + 8192 * j, &p.tmV, full + s, 64 * j, t0 + 64 * i);
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
      const int t0 = x.piece * 64 * args.piece, n = min(args.piece, (args.M - t0 + 63) / 64);
      if (!(ok = warp_poll<40>(wempty + b, wph ^ 1u, abort_flag, args.status, lane))) break;
      const uint32_t d = tmem + (uint32_t)(b * args.n16);
      for (int i = 0; i < n; ++i) {
        if (!(ok = warp_poll<20>((masked ? ready : full) + s, ph, abort_flag, args.status, lane))) break;
        tc_fence_after();
        if (one) {
          const uint8_t* sa = smem + s * stage;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            umma_bf16(d, operand_desc(sa, 1, kk), operand_desc(sa + 16384, 1, kk), id1, (i | kk) != 0);
            if (n2 > 0)
              umma_bf16(d + 256, operand_desc(sa, 1, kk), operand_desc(sa + 16384 + 4 * 8192, 1, kk), id2,
                        (i | kk) != 0);
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
    bool first = true, bad = false;
    for (int64_t u = u_lo; u < u_hi; ++u) {
      const UnitAt x = unit_at(args, u, u_hi);
      if (!warp_wait_backoff(wfull + b, wph, abort_flag, args.status, lane, 100)) break;
      tc_fence_after();
      const MxGradProblem& p = args.p[x.prob];
      float* const out = p.out;
      const int64_t cols = p.cols;
      const bool transposed = p.transposed, whole = args.pieces == 1;
      // this run's slot of the tile (those of dL1 come first)
      float* slot = args.part + mx_slot(u / args.pieces, blockIdx.x) * 128 * r;
      const int row = q4 * 32 + lane;
      const int64_t col = (int64_t)x.tile * 128 + row;
      for (int c = 0; c < r16; c += 16) {
        uint32_t v[16], w[16], z[16];
        const uint32_t at = tl + (uint32_t)(b * args.n16 + c);
        tmem_ld16(at, v);
        tmem_ld16(at + (uint32_t)r, w);
        tmem_ld16(at + 2u * (uint32_t)r, z);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(add_groups(v[j], w[j], z[j]));
        if (!first) {
          tmem_ld16(tl + sum_col + (uint32_t)c, w);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__fadd_rn(__uint_as_float(v[j]), __uint_as_float(w[j])));
        }
        if (x.last) {
#pragma unroll
          for (int j = 0; j < 16; ++j) bad |= c + j < r && (v[j] & 0x7F800000u) == 0x7F800000u;
        }
        if (!x.last) {
          tmem_st16(tl + sum_col + (uint32_t)c, v);
        } else if (whole) {  // this CTA has the whole sum
          if (col < cols && transposed) {
            float* at = out + c * cols + col;
#pragma unroll
            for (int j = 0; j < 16; ++j, at += cols)
              if (c + j < r) *at = __uint_as_float(v[j]);
          } else if (col < cols) {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              if (c + j < r)
                *reinterpret_cast<uint4*>(out + col * r + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          }
        } else if (transposed) {  // slot [r][128]
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < r) slot[(c + j) * 128 + row] = __uint_as_float(v[j]);
        } else {  // slot [128][r]
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            if (c + j < r)
              *reinterpret_cast<uint4*>(slot + (int64_t)row * r + c + j) =
                  make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        __syncwarp();  // the next load takes the whole warp
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
    // dY is looked at where it is quantised, X and T (and dY for dL2 alone) only here
    if (bad) report(args.status, QLORA_ERR_NONFINITE);
  } else if (warp >= 8 && args.drop.threshold) {
    // ----------------------------------------------------------------- mask
    // Units of dL1 come first in a run, so every stage up to the last masked
    // one is masked and the ready barriers' phases follow the ring's.
    const PhiloxKey key = philox_key(args.drop);
    const uint8_t* keep = args.keep;
    if (keep) pdl_wait();
    // two groups of 8 warps take alternate stages; a thread has 8 columns of
    // tokens tok and tok + 32, in both boxes
    const int grp = (warp - 8) >> 3, tok = (tid & 255) >> 3, ch = tid & 7;
    const int64_t c8 = args.p[0].cols >> 3, kt = (args.p[0].cols + 127) / 128 * 16;
    const uint32_t off = (uint32_t)(tok * 128 + ((ch ^ (tok & 7)) << 4)), thr = args.drop.threshold << 16;
    int s = 0, turn = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int64_t u = u_lo; u < u_hi && u < args.sh.units0 && ok; ++u) {
      const UnitAt x = unit_at(args, u, u_hi);
      const int t0 = x.piece * 64 * args.piece, n = min(args.piece, (args.M - t0 + 63) / 64);
      uint64_t ctr = (uint64_t)((t0 + tok) * c8 + x.tile * 16 + ch);
      for (int i = 0; i < n; ++i, turn ^= 1, ctr += 64 * c8) {
        if (turn == grp) {
          if (keep) {
            uint32_t kb[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int m = t0 + 64 * i + tok + 32 * (j & 1);
              kb[j] = m < args.M ? keep[m * kt + x.tile * 16 + ch + 8 * (j >> 1)] : 0u;
            }
            if (!(ok = warp_poll<20>(full + s, ph, abort_flag, args.status, lane))) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint4* at = reinterpret_cast<uint4*>(smem + s * stage + off + 4096 * (j & 1) + 8192 * (j >> 1));
              *at = keep_bits(*at, kb[j]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(ready + s);
          }
        }
        if (turn == grp && !keep) {
          // this thread's evaluations before the wait: they need no data
          uint4 rnd[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) rnd[j] = philox4x32_10(ctr + (j & 1) * 32 * c8 + (j >> 1) * 8, key);
#pragma unroll
          for (int j = 0; j < 4; ++j) keep_here(rnd[j]);
          if (!(ok = warp_poll<20>(full + s, ph, abort_flag, args.status, lane))) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4* at = reinterpret_cast<uint4*>(smem + s * stage + off + 4096 * (j & 1) + 8192 * (j >> 1));
            const uint4 v = *at;
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            drop8_bf16(w, rnd[j], thr);
            *at = make_uint4(w[0], w[1], w[2], w[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(ready + s);
        }
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

// Both gradients from the slots of their tiles, in order.  blockIdx.x is the
// tile (those of dL1 first); a slot is contiguous in the output's order,
// [128][r] of dL1 and, row by row, [r][128] of dL2.
__global__ void __launch_bounds__(256) mx_grad_finish_kernel(const __grid_constant__ MxGradArgs a) {
  pdl_wait();
  const int64_t tiles0 = a.sh.units0 / a.pieces;
  const int prob = blockIdx.x >= tiles0;
  const MxGradProblem& p = a.p[prob];
  const int64_t tile = blockIdx.x - (prob ? tiles0 : 0), tile_u = (int64_t)blockIdx.x * a.pieces;
  const int first = grad_owner(a.sh, tile_u), nc = grad_owner(a.sh, tile_u + a.pieces - 1) - first;
  const int64_t left = p.cols - tile * 128;
  const int ncol = (int)(left < 128 ? left : 128), slot = 128 * a.r;
  const float* s = a.part + mx_slot(blockIdx.x, first) * slot;
  for (int i = ((int)blockIdx.y * 256 + (int)threadIdx.x) * 4; i < slot; i += (int)gridDim.y * 1024) {
    if (p.transposed ? (i & 127) >= ncol : i >= ncol * a.r) continue;
    float4 d = *reinterpret_cast<const float4*>(s + i);
#pragma unroll 4
    for (int c = 1; c <= nc; ++c) {
      const float4 q = *reinterpret_cast<const float4*>(s + (int64_t)c * slot + i);
      d = make_float4(__fadd_rn(d.x, q.x), __fadd_rn(d.y, q.y), __fadd_rn(d.z, q.z), __fadd_rn(d.w, q.w));
    }
    const int64_t o = p.transposed ? (int64_t)(i >> 7) * p.cols + tile * 128 + (i & 127) : tile * slot + i;
    *reinterpret_cast<float4*>(p.out + o) = d;
  }
}

}  // namespace

cudaError_t launch_mx_grad(MxGradArgs& a, const MxGradPlan& p, cudaStream_t st) {
  a.sh = p.sh;
  a.pieces = p.pieces;
  a.piece = p.piece;
  a.n16 = p.n16;
  a.nbuf = p.nbuf;
  a.vboxes = p.vboxes;
  a.stages = p.stages;
  const int smem = p.stages * (16384 + p.vboxes * 8192) + 512 + 1024;
  const cudaError_t err =
      launch_kernel<mx_grad_kernel>({dim3((unsigned)p.sh.grid), kGThreads, (size_t)smem, 1, true}, st, a);
  if (err != cudaSuccess || p.pieces == 1) return err;
  const dim3 grid((unsigned)(p.sh.units / p.pieces), (unsigned)((128 * a.r + 1023) / 1024));
  return launch_kernel<mx_grad_finish_kernel>({grid, 256, 0, 1, true}, st, a);
}

}  // namespace qnf4
