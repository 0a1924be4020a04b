// One pass over the activations (forward) or the upstream gradient
// (backward) of the MXFP4 linear layer:
//
//   Q(X): codes and scales of X [M][C], and
//   D = drop(X) . L  [M][r]  (fp32), L = L1 [C][r] or L2^T with L2 [r][C].
//
// Both read all of X and little else, so the bound is X's bytes (2 a value
// in, 0.53 out); two passes would read it twice, and a dropped copy of X
// would be a third and fourth.  The tile of X comes to shared memory by TMA;
// there the quantise warps read it once, write the codes and scales, and
// zero the dropped elements in place, and the tensor cores take the same
// tile as the A operand of D.
//
// Work is cut into units of 128 rows x 256 columns.  While clusters of up to 8
// CTAs (16 for up to 4 row tiles) for every row tile run at once, a cluster
// takes a row tile, adds its CTAs' sums in rank order through distributed
// shared memory and forms T and the bf16 terms of the scaled D itself (two for
// the products, three where the adapter gradients take them too).  For more rows
// one CTA per SM takes an equal run of units in order (the last units of a row
// tile and the first of the next may share a CTA); a run's rows of D go to a
// partial slot, and a small second kernel adds the slots of a row tile in
// order.
//
// The tensor cores truncate their fp32 sums, an error that grows with their
// length, so D is accumulated in pieces of 512 columns that are added with
// rounding: two work accumulators in tensor memory that take turns, and the
// sum beside them.
//
// Measured, 8192 x 8192 with r = 64: 36 us, 170 MB of X, codes and scales (the
// quantiser alone: 29 us; loads alone: 29 us, whatever the ring's depth from 4
// to 10 stages).  With dropout 61 us: the generator's and the mask's integer
// instructions add to the quantiser's on the same pipes.
//
// Roles: warp 0 TMA producer, 1 MMA issuer, 2 stores codes and scales, 4-7 sum
// D, 8-23 quantise (two groups of 8 warps, alternate 64-column stages; a
// thread has one 32-block of one row).
#include "engine_util.cuh"
#include "launch.cuh"
#include "mx_codec.cuh"
#include "mx_util.cuh"
#include "pair_util.cuh"
#include "philox.cuh"

namespace qnf4 {
namespace {

constexpr int kPieces = 8;  // 64-column stages of a piece of D

template <bool WIDE>  // r > 64
struct PrepCfg {
  static constexpr int S = WIDE ? 5 : 6;
  static constexpr int L = WIDE ? 16384 : 8192;  // tile of L: 64 columns x up to 128 / 64 ranks
  static constexpr int LT = S * 16384;   // the tiles of L, behind those of X
  static constexpr int OUT = LT + S * L;  // two staging buffers: 16 KB of codes, 1 KB of scales
  static constexpr int OUTB = 16384 + 1024;
  static constexpr int BAR = OUT + 2 * OUTB;
  static constexpr int TOTAL = BAR + 512 + 1024;
  static_assert(TOTAL <= 232448 && OUTB % 1024 == 0, "budget");
  static_assert(S * L >= 128 * ((WIDE ? 128 : 64) + 4) * 4, "a cluster's partial sums go over the tiles of L");
};
constexpr int kQGroups = 2;  // quantise groups of 8 warps (3 were a few percent slower)
constexpr int kPrepThreads = (8 + 8 * kQGroups) * 32;
constexpr uint32_t kSumCol = 256;  // tensor memory: work accumulators at 0 and 128, the sum at 256

// The first bf16 term of v: v rounded toward zero (so it never overflows, and
// what is left has v's sign), an Inf or NaN as it is.
QDEV float first_term(float v) {
  const float h = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
  return v != v ? __uint_as_float(0x7FC00000u) : h;
}
// What the other terms stand for.  An Inf or NaN is repeated, and nothing left
// of a number is 2^-126 of its sign: multiplied with an Inf on the other side
// every term then gives what v itself gives, where 0 or Inf - Inf would make
// it NaN.
QDEV float rest_of(float v, float h) {
  if ((__float_as_uint(v) & 0x7F800000u) == 0x7F800000u) return h;
  const float d = __fsub_rn(v, h);  // exact
  return d == 0.0f && fabsf(h) > 0x1p-100f ? copysignf(0x1p-126f, h) : d;
}
// beta v as `terms` bf16 terms, r elements apart; four neighbours at a time.
// Two terms hold 16 bits of it (2^-16 relative), three all of an fp32.
QDEV void store_terms(uint16_t* out, float4 v, float beta, int terms, int r) {
  v = make_float4(__fmul_rn(v.x, beta), __fmul_rn(v.y, beta), __fmul_rn(v.z, beta), __fmul_rn(v.w, beta));
  const float4 h = make_float4(first_term(v.x), first_term(v.y), first_term(v.z), first_term(v.w));
  *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(h.x, h.y), pack_bf16x2(h.z, h.w));
  v = make_float4(rest_of(v.x, h.x), rest_of(v.y, h.y), rest_of(v.z, h.z), rest_of(v.w, h.w));
  for (int t = 1; t < terms; ++t) {
    const uint2 w = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    *reinterpret_cast<uint2*>(out + (int64_t)t * r) = w;
    v = make_float4(__fsub_rn(v.x, __uint_as_float(w.x << 16)), __fsub_rn(v.y, __uint_as_float(w.x & 0xFFFF0000u)),
                    __fsub_rn(v.z, __uint_as_float(w.y << 16)), __fsub_rn(v.w, __uint_as_float(w.y & 0xFFFF0000u)));
  }
}

// Four neighbours D[row][j ..] to T and the bf16 terms.
QDEV void emit4(const MxPrepFinish& a, int64_t row, int j, float4 d) {
  if (a.T)
    *reinterpret_cast<float4*>(a.T + row * a.r + j) =
        make_float4(__fmul_rn(d.x, a.alpha), __fmul_rn(d.y, a.alpha), __fmul_rn(d.z, a.alpha),
                    __fmul_rn(d.w, a.alpha));
  store_terms(a.out + row * a.terms * a.r + j, d, a.beta, a.terms, a.r);
}
// The other operand of the backward's adapter sums rides along: s T in three terms.
QDEV void emit_t4(const MxPrepFinish& a, int64_t row, int j) {
  store_terms(a.out2 + row * 3 * a.r + j, *reinterpret_cast<const float4*>(a.T_in + row * a.r + j), a.gamma, 3, a.r);
}

template <bool WIDE>
__global__ void __launch_bounds__(kPrepThreads, 1) mx_prep_kernel(const __grid_constant__ MxPrepArgs args) {
  using C = PrepCfg<WIDE>;
  constexpr int kS = C::S;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR);  // X and L tiles landed
  uint64_t* ready = full + kS;    // 8 quantise warps have zeroed the dropped elements (dropout only)
  uint64_t* empty = ready + kS;   // MMAs done (1) and 8 quantise warps have read the tile
  uint64_t* ofull = empty + kS;   // staging buffer written: 8 warps x 4 stages
  uint64_t* oempty = ofull + 2;   // ... and stored
  uint64_t* wfull = oempty + 2;   // work accumulator holds a piece
  uint64_t* wempty = wfull + 2;   // ... and has been added (4 warps)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(wempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const int upt = args.units_per_tile;
  const int csize = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int64_t tile0 = blockIdx.x / (unsigned)csize;  // direct: this cluster's row tile
  const int64_t u_lo = args.direct ? tile0 * upt + (int64_t)rank * upt / csize
                                   : prep_unit(args.units, (int)gridDim.x, blockIdx.x);
  const int64_t u_hi = args.direct ? tile0 * upt + (int64_t)(rank + 1) * upt / csize
                                   : prep_unit(args.units, (int)gridDim.x, (int64_t)blockIdx.x + 1);
  const int n_units = (int)(u_hi - u_lo);
  const bool drop = args.drop.threshold != 0;

  if (warp == 0) {  // a barrier a lane
    if (lane < kS) {
      mbar_init(full + lane, 1);
      mbar_init(ready + lane, 8);
      mbar_init(empty + lane, 9);
    } else if (lane < kS + 2) {
      const int b = lane - kS;
      mbar_init(ofull + b, 32);
      mbar_init(oempty + b, 1);
      mbar_init(wfull + b, 1);
      mbar_init(wempty + b, 4);
    } else if (lane == kS + 2) {
      *abort_flag = 0;
      tma_prefetch_desc(&args.tmX);
      tma_prefetch_desc(&args.tmL);
      tma_prefetch_desc(&args.tmCodes);
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
      const int lboxes = (args.r16 + 63) / 64;
      const uint32_t lbytes = args.l_mn ? (uint32_t)lboxes * 8192u : (uint32_t)args.r16 * 128u;
      int s = 0;
      uint32_t ph = 0;
      for (int u = 0; u < n_units; ++u) {
        const int64_t uu = u_lo + u;
        const int row0 = (int)(uu / upt) * 128, c0 = (int)(uu % upt) * 256;
        bool ok = true;
        for (int q = 0; q < 4; ++q) {
          if (!(ok = mbar_wait_backoff(empty + s, ph ^ 1u, abort_flag, args.status, 20))) break;
          uint8_t* sx = smem + s * 16384;
          uint8_t* sl = smem + C::LT + s * C::L;
          const int c = c0 + 64 * q;
          mbar_arrive_expect_tx(full + s, 16384u + lbytes);
          tma_load_2d(sx, &args.tmX, full + s, c, row0);
          if (args.l_mn) {
            for (int j = 0; j < lboxes; ++j) tma_load_2d(sl + 8192 * j, &args.tmL, full + s, 64 * j, c);
          } else {
            tma_load_2d(sl, &args.tmL, full + s, c, 0);
          }
          if (++s == kS) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    const uint32_t idesc = idesc_bf16(128, 16, 0, args.l_mn) + ((uint32_t)((args.r16 - 16) >> 3) << 17);
    const bool one = elect_one();
    int s = 0, piece = 0, in_piece = 0;
    uint32_t ph = 0;
    for (int u = 0; u < n_units; ++u) {
      const bool last = u + 1 == n_units || (int)((u_lo + u + 1) % upt) == 0;  // ends a row tile's run
      bool ok = true;
      for (int q = 0; q < 4; ++q) {
        const int b = piece & 1;
        if (in_piece == 0) {
          if (!(ok = warp_poll<40>(wempty + b, ((uint32_t)(piece >> 1) & 1u) ^ 1u, abort_flag, args.status, lane)))
            break;
        }
        if (!(ok = warp_poll<40>((drop ? ready : full) + s, ph, abort_flag, args.status, lane))) break;
        tc_fence_after();
        if (one) {
          const uint8_t* sx = smem + s * 16384;
          const uint8_t* sl = smem + C::LT + s * C::L;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem + 128u * (uint32_t)b, operand_desc(sx, 0, kk), operand_desc(sl, args.l_mn, kk), idesc,
                      (in_piece | kk) != 0);
          umma_commit(empty + s);
        }
        __syncwarp();
        ++in_piece;
        if (in_piece == kPieces || (last && q == 3)) {
          if (one) umma_commit(wfull + b);
          __syncwarp();
          in_piece = 0;
          ++piece;
        }
        if (++s == kS) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
    }
  } else if (warp == 2) {
    // --------------------------------------------------- codes and scales out
    if (lane == 0) {
      for (int u = 0; u < n_units; ++u) {
        const int b = u & 1;
        if (!mbar_wait_backoff(ofull + b, (uint32_t)(u >> 1) & 1u, abort_flag, args.status, 40)) break;
        const int64_t uu = u_lo + u;
        const int64_t rt = uu / upt;
        const int kb = (int)(uu % upt);
        const uint8_t* so = smem + C::OUT + b * C::OUTB;
        tma_store_2d(&args.tmCodes, so, kb * 128, (int)(rt * 128));
        bulk_store(args.scales + (rt * args.kt + 2 * kb) * 512, so + 16384, 512u * (uint32_t)min(2, args.kt - 2 * kb));
        bulk_commit();
        bulk_wait_read<0>();
        mbar_arrive(oempty + b);
      }
      bulk_wait_all();
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------- sum of the pieces
    const int q4 = warp & 3;
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
    int piece = 0, in_piece = 0;
    bool first = true;
    for (int u = 0; u < n_units; ++u) {
      const bool last = u + 1 == n_units || (int)((u_lo + u + 1) % upt) == 0;
      in_piece += 4;
      if (in_piece < kPieces && !last) continue;
      const int b = piece & 1;
      if (!warp_wait_backoff(wfull + b, (uint32_t)(piece >> 1) & 1u, abort_flag, args.status, lane, 100)) break;
      tc_fence_after();
      float* dst = nullptr;
      if (last && args.direct) {  // for the cluster, over the tiles of L: all of them have been multiplied
        dst = reinterpret_cast<float*>(smem + C::LT) + (q4 * 32 + lane) * (args.r + 4);
      } else if (last) {  // this run's rows of D
        const int64_t tile = (u_lo + u) / upt;
        dst = args.part + (mx_slot(tile, blockIdx.x) * 128 + q4 * 32 + lane) * args.r;
      }
      for (int c = 0; c < args.r16; c += 16) {
        uint32_t v[16];
        tmem_ld16(tl + 128u * (uint32_t)b + (uint32_t)c, v);
        if (!first) {
          uint32_t m[16];
          tmem_ld16(tl + kSumCol + (uint32_t)c, m);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__fadd_rn(__uint_as_float(v[j]), __uint_as_float(m[j])));
        } else {
          tmem_wait_ld();
        }
        if (!last) {
          tmem_st16(tl + kSumCol + (uint32_t)c, v);
        } else {
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            if (c + j < args.r)
              *reinterpret_cast<uint4*>(dst + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(wempty + b);
      first = last;
      in_piece = 0;
      ++piece;
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ quantise
    const int grp = (warp - 8) >> 3, t = tid & 255;
    const int rl = t & 127, half = t >> 7;
    const PhiloxKey key = drop ? philox_key(args.drop) : PhiloxKey{0, 0, 0, 0};
    const uint32_t thr = args.drop.threshold << 16;
    if (args.direct && args.fin.T_in) {  // while the first tiles are on their way
      const int rows = 128 / csize, r4 = args.r / 4;
      for (int i = tid - 256; i < rows * r4; i += kPrepThreads - 256) {
        const int64_t row = tile0 * 128 + rank * rows + i / r4;
        if (row < args.fin.M) emit_t4(args.fin, row, (i % r4) * 4);
      }
      __syncwarp();
    }
    bool bad = false;
    int s = grp;  // ring stage of iteration `it` (grp < kS)
    uint32_t ph = 0;
    int64_t tile = u_lo / upt;  // of the unit
    int kb = (int)(u_lo % upt);
    for (int it = grp, u = 0; it < 4 * n_units; it += kQGroups) {
      for (; u < it >> 2; ++u)  // the unit of this stage
        if (++kb == upt) {
          kb = 0;
          ++tile;
        }
      const int q = it & 3, ob = u & 1;
      uint8_t* so = smem + C::OUT + ob * C::OUTB;
      // a warp whose 32 rows are all past the last one only zeroes their scales
      const bool live = tile * 128 + (rl & 96) < args.fin.M;
      uint4 rnd[4];
      if (drop && live) {  // the generator needs no data: evaluated before the wait
        const uint64_t e8 = (uint64_t)((tile * 128 + rl) * args.cols + kb * 256 + 64 * q + 32 * half) >> 3;
#pragma unroll
        for (int j = 0; j < 4; ++j) rnd[j] = philox4x32_10(e8 | j, key);  // e8 is a multiple of 4
#pragma unroll
        for (int j = 0; j < 4; ++j) keep_here(rnd[j]);
      }
      if (!warp_poll<20>(full + s, ph, abort_flag, args.status, lane)) break;
      uint8_t* sx = smem + s * 16384 + rl * 128;
      uint32_t c[4], b = 0;
      if (live) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 v = *reinterpret_cast<const uint4*>(sx + (((4 * half + j) ^ (rl & 7)) << 4));
          w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
        }
        if (drop) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t z[4] = {w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]};
            drop8_bf16(z, rnd[j], thr);
            *reinterpret_cast<uint4*>(sx + (((4 * half + j) ^ (rl & 7)) << 4)) = make_uint4(z[0], z[1], z[2], z[3]);
          }
          fence_proxy_async_smem();  // before the MMAs read the tile
          __syncwarp();
          if (lane == 0) mbar_arrive(ready + s);
        }
        uint32_t m2 = 0, m3 = 0;  // largest |x|, two lanes each
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m2 = mx_absmax2(m2, w[j]);
          m3 = mx_absmax2(m3, w[8 + j]);
        }
        b = mx_scale_byte(mx_absmax_bits(mx_absmax2(m2, m3)));
        bad |= b == 255u;
        const float f = mx_inv_scale(b);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = mx_codes8(w + 4 * j, f);
      } else if (drop && lane == 0) {
        mbar_arrive(ready + s);
      }
      if (!warp_poll<20>(oempty + ob, ((uint32_t)(u >> 1) & 1u) ^ 1u, abort_flag, args.status, lane)) break;
      const int blk = 2 * q + half;  // 32-block of the unit
      if (live)
        *reinterpret_cast<uint4*>(so + rl * 128 + ((blk ^ (rl & 7)) << 4)) = make_uint4(c[0], c[1], c[2], c[3]);
      so[16384 + (blk >> 2) * 512 + (rl & 31) * 16 + (rl >> 5) * 4 + (blk & 3)] = (uint8_t)b;
      // the tile's reads before the TMA refills it, the codes before the TMA stores them
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(empty + s);
        mbar_arrive(ofull + ob);
      }
      s += kQGroups;
      if (s >= kS) {
        s -= kS;
        ph ^= 1u;
      }
    }
    if (bad) report(args.status, QLORA_ERR_NONFINITE);
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
  if (args.direct) {
    // The cluster holds its row tile's D: the partial sums are added in rank
    // order, 128 / csize rows a CTA.  Eight of a peer's loads are in flight at
    // once, and the CTA tells its peers that it has read them before it stores.
    const int r = args.r, pitch = r + 4;
    const float* red = reinterpret_cast<const float*>(smem + C::LT);
    cluster_sync_all();
    const MxPrepFinish& f = args.fin;
    const int rows = 128 / csize, r4 = r / 4, n = rows * r4;
    const bool good = !*abort_flag;
    for (int i0 = 0; i0 < n; i0 += kPrepThreads) {
      const int i = i0 + tid;
      const int lr = rank * rows + i / r4, j = (i % r4) * 4;
      const int64_t row = tile0 * 128 + lr;
      const bool mine = good && i < n && row < f.M;
      float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
      if (mine) {
        const uint32_t at = smem_u32(red + lr * pitch + j);
        d = ld_peer_f4(at, 0);
        int c = 1;
        for (; c + 7 <= csize; c += 7) {
          float4 q[7];
#pragma unroll
          for (int k = 0; k < 7; ++k) q[k] = ld_peer_f4(at, (uint32_t)(c + k));
#pragma unroll
          for (int k = 0; k < 7; ++k)
            d = make_float4(__fadd_rn(d.x, q[k].x), __fadd_rn(d.y, q[k].y), __fadd_rn(d.z, q[k].z),
                            __fadd_rn(d.w, q[k].w));
        }
        for (; c < csize; ++c) {
          const float4 q = ld_peer_f4(at, (uint32_t)c);
          d = make_float4(__fadd_rn(d.x, q.x), __fadd_rn(d.y, q.y), __fadd_rn(d.z, q.z), __fadd_rn(d.w, q.w));
        }
      }
      if (i0 + kPrepThreads >= n) cluster_arrive();  // the last rows are read
      if (mine) emit4(f, row, j, d);
    }
    cluster_wait();  // peers may still be reading this CTA's rows
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// D from the partial slots of its row tile, in order: T = alpha D (fp32, when
// asked for) and `terms` bf16 terms of beta D, [M][terms * r].  blockIdx.x is
// the row tile; a slot [128][r] is contiguous in D's own order.
__global__ void __launch_bounds__(256) mx_prep_finish_kernel(const __grid_constant__ MxPrepFinish a) {
  pdl_trigger();
  pdl_wait();
  const int64_t tile = blockIdx.x;
  const int first = prep_owner(a.units, a.grid, tile * a.units_per_tile);
  const int nc = prep_owner(a.units, a.grid, (tile + 1) * a.units_per_tile - 1) - first;
  const int64_t left = (a.M - tile * 128) * a.r;
  const int n = (int)(left < 128 * a.r ? left : 128 * a.r);
  const float* p = a.part + mx_slot(tile, first) * 128 * a.r;
  for (int i = ((int)blockIdx.y * 256 + (int)threadIdx.x) * 4; i < n; i += (int)gridDim.y * 1024) {
    float4 d = *reinterpret_cast<const float4*>(p + i);
#pragma unroll 4
    for (int c = 1; c <= nc; ++c) {
      const float4 q = *reinterpret_cast<const float4*>(p + (int64_t)c * 128 * a.r + i);
      d = make_float4(__fadd_rn(d.x, q.x), __fadd_rn(d.y, q.y), __fadd_rn(d.z, q.z), __fadd_rn(d.w, q.w));
    }
    const int row = i / a.r, j = i - row * a.r;
    emit4(a, tile * 128 + row, j, d);
    if (a.T_in) emit_t4(a, tile * 128 + row, j);
  }
}

__global__ void __launch_bounds__(256) split3_kernel(const float* __restrict__ in, int64_t n4, int r, float scale,
                                                      uint16_t* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i * 4 / r;
    store_terms(out + i * 4 + 2 * r * m, reinterpret_cast<const float4*>(in)[i], scale, 3, r);
  }
}

}  // namespace

// Largest cluster that the current device can hold: 16, else the portable 8.
int mx_prep_max_cluster() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 8;
  int most = known[dev].load(std::memory_order_relaxed);
  if (most) return most;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 16;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(kPrepThreads);
  cfg.dynamicSmemBytes = std::max(PrepCfg<true>::TOTAL, PrepCfg<false>::TOTAL);
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int clusters = 0;
  most = allow_big<mx_prep_kernel<true>>(false) == cudaSuccess &&
                 cudaOccupancyMaxActiveClusters(&clusters, mx_prep_kernel<true>, &cfg) == cudaSuccess && clusters > 0
             ? 16
             : 8;
  (void)cudaGetLastError();
  known[dev].store(most, std::memory_order_relaxed);
  return most;
}

cudaError_t launch_mx_prep(MxPrepArgs& a, const MxPrepPlan& p, cudaStream_t st) {
  a.units = p.units;
  a.units_per_tile = p.units_per_tile;
  a.direct = p.direct;
  a.r16 = (a.r + 15) / 16 * 16;
  a.fin.part = a.part;
  a.fin.r = a.r;
  a.fin.units = p.units;
  a.fin.units_per_tile = p.units_per_tile;
  a.fin.grid = p.grid;
  const LaunchShape narrow{dim3((unsigned)p.grid), kPrepThreads, PrepCfg<false>::TOTAL, (unsigned)p.cluster, false};
  const LaunchShape wide{dim3((unsigned)p.grid), kPrepThreads, PrepCfg<true>::TOTAL, (unsigned)p.cluster, false};
  const cudaError_t e = a.r > 64 ? launch_kernel<mx_prep_kernel<true>>(wide, st, a)
                                 : launch_kernel<mx_prep_kernel<false>>(narrow, st, a);
  if (e != cudaSuccess || p.direct) return e;
  const int64_t tiles = (a.fin.M + 127) / 128;
  return launch_kernel<mx_prep_finish_kernel>(
      {dim3((unsigned)tiles, (unsigned)((128 * a.r + 1023) / 1024)), 256, 0, 1, true}, st, a.fin);
}

cudaError_t launch_split3(const float* in, int64_t M, int r, float scale, uint16_t* out, int sms, cudaStream_t st) {
  const int64_t n4 = M * r / 4, want = (n4 + 255) / 256, most = (int64_t)sms * 8;
  split3_kernel<<<(unsigned)(want < most ? want : most), 256, 0, st>>>(in, n4, r, scale, out);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace qnf4
