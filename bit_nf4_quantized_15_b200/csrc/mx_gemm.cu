// Product of two MXFP4 matrices on the block-scaled tensor cores.
//
//   out[col, row] = RN( sum_k A^[row, k] B^[col, k] + mask sum_j Ax[row, j] Bx[col, j] )
//
// tcgen05.mma kind::mxf4 takes the 4-bit codes as they are stored, 64 of them
// a step, and multiplies each 32-block's exact product sum by both E8M0
// scales in the MMA; the accumulator is fp32 in tensor memory.  So nothing is
// dequantised: codes and scales go HBM -> shared memory by TMA, the scales
// on to tensor memory by tcgen05.cp, and the loop has no arithmetic of its
// own.  The optional second sum is the LoRA term (bf16, kind::f16, the token
// side in two terms) of the linear layer; it is formed first, so that it can be
// masked by the dropout of the adapter path in tensor memory before the main
// sum is added to it.
//
// This kernel gives a 128 (rows) x BN (cols) tile to a cluster of 1, 2, 4 or
// 8 CTAs that split the reduction; the partial tiles meet through distributed
// shared memory and are added in rank order, so results do not depend on
// timing and no workspace is needed.  A is the side with more rows to give
// (the weight), B the tokens: with few tokens BN shrinks to 16 and a call
// streams the weight once through all SMs.
//
// Measured in a graph: one token through 4096 x 4096 5.7 us; 16 tokens through
// 22016 x 8192 19.6 us, where its 96 MB take 14.6 at the measured copy bandwidth
// (15.4 with the weight in L2); 1000 x 2056 x 1568 7.8 us.  The small ones are launch, tensor memory, one round trip
// to HBM and the epilogue, one after another.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer, then 4 epilogue warps (8 for
// BN >= 128).
#include "engine_util.cuh"
#include "launch.cuh"
#include "mx_util.cuh"
#include "pair_util.cuh"
#include "philox.cuh"

namespace qnf4 {
namespace {

template <int BN>
struct MxCfg {
  static constexpr int S = BN >= 256 ? 4 : BN >= 128 ? 6 : BN >= 64 ? 4 : 5;  // stages
  static constexpr int EW = BN >= 128 ? 8 : 4;                                 // epilogue warps
  static constexpr int THREADS = 64 + 32 * EW;
  static constexpr int A = 16384;                      // 128 rows x 128 bytes
  static constexpr int B = BN * 128;
  static constexpr int FB = BN > 128 ? 2 : 1;          // B scale tiles (128 rows each)
  static constexpr int STAGE = A + B + 1024 + FB * 1024;
  static constexpr int BAR = S * STAGE;
  static constexpr int TOTAL = BAR + 256 + 1024;       // barriers + alignment slack
  static constexpr uint32_t ACC = BN < 32 ? 32 : BN;   // accumulator columns
  static constexpr uint32_t SF = 8 + 8 * FB;           // scale columns of a stage: A, then B
  static constexpr uint32_t NEED = ACC + S * SF;
  static constexpr uint32_t COLS = NEED <= 128 ? 128 : NEED <= 256 ? 256 : 512;
  static_assert(NEED <= 512 && STAGE % 1024 == 0 && TOTAL <= 232448 && BN * 512 <= S * STAGE, "budget");
};

QDEV void umma_mxf4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
      : "memory");
}
// One scale tile (512 bytes: 32 lanes x 16 bytes, repeated to the four lane
// quarters) from shared to tensor memory: 4 columns.
QDEV void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
QDEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
// Zero the dropped entries of this warp's 32 lanes x 16 columns of the LoRA
// term.  Lanes are consecutive output rows (elements), so 8 lanes share one
// generator evaluation per column: lane l evaluates column c + (l & 7) for
// its group of 8 and the byte is shuffled to the lane that needs it.
QDEV void mask_chunk(uint32_t (&v)[16], const MxGemmArgs& a, const PhiloxKey& key, int row_base, int col, int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t m = (int64_t)col + 8 * h + (lane & 7);
    const uint32_t byte = keep8((uint64_t)(m * a.ldo + row_base + (lane & ~7)) >> 3, key, a.drop.threshold);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = __shfl_sync(0xFFFFFFFFu, byte, (lane & ~7) | j);
      if (!((b >> (lane & 7)) & 1u)) v[8 * h + j] = 0u;
    }
  }
}

// F32: fp32 output (no LoRA term), in pieces of the reduction.
template <int BN, bool F32>
__global__ void __launch_bounds__(MxCfg<BN>::THREADS, 1) mx_gemm_kernel(const __grid_constant__ MxGemmArgs args) {
  using C = MxCfg<BN>;
  constexpr int kS = C::S;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR);
  uint64_t* empty = full + kS;
  uint64_t* ext_done = empty + kS;    // the LoRA term is in tensor memory
  uint64_t* ext_masked = ext_done + 1;  // ... and masked
  uint64_t* accum = ext_masked + 1;     // the sum (F32: of a piece) is in tensor memory
  uint64_t* drained = accum + 1;        // F32: ... and in registers
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const int rank = (int)cluster_ctarank(), csize = (int)cluster_nctarank();
  const int id = (int)(blockIdx.x / (unsigned)csize);
  const int n_tiles = (args.cols + BN - 1) / BN;
  const int row_tile = id / n_tiles, col_tile = id % n_tiles;
  const int row0 = row_tile * 128, col0 = col_tile * BN;
  const int kb_lo = (int)((int64_t)rank * args.kb / csize), kb_hi = (int)((int64_t)(rank + 1) * args.kb / csize);
  const int rb = (args.r + 63) / 64;                      // 64-wide blocks of the rank
  const int n_ext = !F32 && rank == 0 ? kLoraTerms * rb : 0;  // term by term
  const int n_iters = n_ext + kb_hi - kb_lo;
  const bool masked = n_ext && args.drop.threshold;
  const int pieces = F32 ? (n_iters + kMxPiece - 1) / kMxPiece : 1;
  const uint64_t lim = args.wait_ns ? args.wait_ns : QNF4_WAIT_NS;

  if (tid == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(ext_done, 1);
    mbar_init(ext_masked, C::EW);
    mbar_init(accum, 1);
    mbar_init(drained, C::EW);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&args.tmA);
    tma_prefetch_desc(&args.tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  pdl_trigger();  // not before this CTA has its tensor memory: a dependent CTA must not take it first
  bool committed = false;
  uint32_t last_ph = 0;  // of accum

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The weight side (A) is not written by the kernel before this one, so its
    // first stages are loaded before that has finished; the tokens' side waits.
    if (lane == 0 && !args.stall) {
      const int nb = C::FB == 2 && col0 + 128 < args.cols ? 2 : 1;  // token scale tiles
      auto load_a = [&](int it, int s) {
        uint8_t* sa = smem + s * C::STAGE;
        if (it < n_ext) {
          mbar_arrive_expect_tx(full + s, tx_bytes(args.a_mn_ext, 128) + tx_bytes(0, BN));
          load_operand(sa, &args.tmAx, full + s, args.a_mn_ext, row0, it % rb * 64, 128);
        } else {
          const int kb = kb_lo + it - n_ext;
          const uint32_t sbytes = 512u * (uint32_t)min(2, args.kt - 2 * kb);  // scale tiles along K
          mbar_arrive_expect_tx(full + s, (uint32_t)C::A + (uint32_t)C::B + sbytes * (1u + (uint32_t)nb));
          tma_load_2d(sa, &args.tmA, full + s, kb * 128, row0);
          bulk_load(sa + C::A + C::B, args.sfA + ((int64_t)(row0 >> 7) * args.kt + 2 * kb) * 512, sbytes, full + s);
        }
      };
      auto load_b = [&](int it, int s) {
        uint8_t* sb = smem + s * C::STAGE + C::A;
        if (it < n_ext) {
          tma_load_3d(sb, &args.tmBx, full + s, it % rb * 64, it / rb, col0);
        } else {
          const int kb = kb_lo + it - n_ext;
          const uint32_t sbytes = 512u * (uint32_t)min(2, args.kt - 2 * kb);
          tma_load_2d(sb, &args.tmB, full + s, kb * 128, col0);
          for (int j = 0; j < nb; ++j)
            bulk_load(sb + C::B + 1024 + 1024 * j, args.sfB + ((int64_t)((col0 >> 7) + j) * args.kt + 2 * kb) * 512,
                      sbytes, full + s);
        }
      };
      const int ahead = min(kS, n_iters);
      for (int it = 0; it < ahead; ++it) load_a(it, it);
      pdl_wait();
      for (int it = 0; it < ahead; ++it) load_b(it, it);
      for (int it = ahead; it < n_iters; ++it) {
        const int s = it % kS;
        if (!mbar_wait(empty + s, ((uint32_t)(it / kS) & 1u) ^ 1u, abort_flag, args.status, lim)) break;
        load_a(it, s);
        load_b(it, s);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    const uint32_t id_ext = idesc_bf16(128, BN, args.a_mn_ext, 0);
    const int64_t tail = args.K - (int64_t)(args.kb - 1) * kMxKB;
    const int tail_steps = (int)((tail + 63) / 64);
    const uint32_t base = smem_u32(smem), a0 = kdesc_lo(base), f0 = (uint32_t)sdesc_scales(base + C::A + C::B);
    const uint32_t fhi = (uint32_t)(sdesc_scales(0) >> 32);
    // a tile of 64 tokens may begin inside a scale tile: 32 rows a column
    const uint32_t sfb0 = (uint32_t)(col0 & 127) >> 5;
    const bool one = elect_one();
    int s = 0;
    uint32_t ph = 0;
    for (int it = 0; it < n_iters; ++it) {
      if (!warp_poll(full + s, ph, abort_flag, args.status, lane, lim)) break;
      tc_fence_after();
      if (it < n_ext) {
        const uint8_t* sa = smem + s * C::STAGE;
        if (one) {
          const int steps = (min(64, args.r - it % rb * 64) + 15) / 16;  // zeros past r
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (kk < steps)
              umma_bf16(tmem, operand_desc(sa, args.a_mn_ext, kk), operand_desc(sa + C::A, 0, kk), id_ext,
                        (it | kk) != 0);
          umma_commit(empty + s);
          if (it == n_ext - 1) umma_commit(ext_done);
        }
        __syncwarp();
        // MMAs of another kind follow: let these finish (and be masked)
        if (it == n_ext - 1) {
          if (!warp_poll(masked ? ext_masked : ext_done, 0, abort_flag, args.status, lane, lim)) break;
          tc_fence_after();
        }
      } else if (one) {
        const int steps = kb_lo + it - n_ext == args.kb - 1 ? tail_steps : 4;
        const uint32_t so = (uint32_t)s * (C::STAGE >> 4);
        const uint32_t sf = tmem + C::ACC + (uint32_t)s * C::SF;  // this stage's scale columns
        // A stage's scale columns are free again with the stage: its barrier
        // says that the MMAs that read them have finished.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (2 * h < steps) {
            const uint64_t f = ((uint64_t)fhi << 32) | (f0 + so + 32 * h);
            tmem_cp_scales(sf + 4 * h, f);
#pragma unroll
            for (int j = 0; j < C::FB; ++j) tmem_cp_scales(sf + 8 + 4 * (C::FB * h + j), f + 64 + 64 * j);
          }
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk < steps)
            umma_mxf4(tmem, kdesc(a0 + so + 2 * kk), kdesc(a0 + so + (C::A >> 4) + 2 * kk),
                      idesc_mxf4(128, BN, 2 * (kk & 1)), sf + 4 * (kk >> 1), sfb0 + sf + 8 + 4 * C::FB * (kk >> 1),
                      ((F32 ? it % kMxPiece : it) | kk) != 0);
        }
        umma_commit(empty + s);
      }
      __syncwarp();
      if (F32 && (it + 1) % kMxPiece == 0 && it + 1 < n_iters) {
        if (one) umma_commit(accum);
        committed = true;
        __syncwarp();
        if (!warp_poll(drained, last_ph, abort_flag, args.status, lane, lim)) break;
        tc_fence_after();
        last_ph ^= 1u;
      }
      if (++s == kS) {
        s = 0;
        ph ^= 1u;
      }
    }
    if (one) umma_commit(accum);
    committed = true;
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q4 = warp & 3, grp = (warp - 2) >> 2;
    constexpr int G = C::EW / 4;
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
    const int row = row0 + q4 * 32 + lane;
    if (masked) {
      const PhiloxKey key = philox_key(args.drop);
      if (warp_wait(ext_done, 0, abort_flag, args.status, lane, lim)) {
        tc_fence_after();
        for (int c = grp * 16; c < BN; c += G * 16) {
          uint32_t v[16];
          tmem_ld16(tl + (uint32_t)c, v);
          tmem_wait_ld();
          mask_chunk(v, args, key, row0 + q4 * 32, col0 + c, lane);
          tmem_st16(tl + (uint32_t)c, v);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ext_masked);
    }
    constexpr int kChunks = BN / (16 * G);
    float sum[F32 ? kChunks : 1][16] = {};
    bool ok = true;
#pragma unroll 1
    for (int p = 0; p < pieces && ok; ++p) {
      ok = warp_wait(accum, (uint32_t)p & 1u, abort_flag, args.status, lane, lim);
      tc_fence_after();
      if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          uint32_t v[16];
          tmem_ld16(tl + (uint32_t)((grp + i * G) * 16), v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[i][j] = __fadd_rn(sum[i][j], __uint_as_float(v[j]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(drained);
      }
    }
#pragma unroll(F32 ? kChunks : 1)
    for (int i = 0; i < kChunks; ++i) {
      const int c = (grp + i * G) * 16;
      uint32_t v[16];
      if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(sum[i][j]);
      } else {
        tmem_ld16(tl + (uint32_t)c, v);
        tmem_wait_ld();
      }
      if (csize > 1) {  // this CTA's partial tile, over the stages (all read by now)
        float* red = reinterpret_cast<float*>(smem) + c * 128 + q4 * 32 + lane;
#pragma unroll
        for (int j = 0; j < 16; ++j) red[j * 128] = __uint_as_float(v[j]);
        continue;
      }
      if (ok && !*abort_flag && row < args.rows) {
        const int ncol = min(16, args.cols - (col0 + c));
        const int64_t o = (int64_t)(col0 + c) * args.ldo + row;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (j >= ncol) continue;
          if (F32) reinterpret_cast<float*>(args.out)[o + j * args.ldo] = __uint_as_float(v[j]);
          else reinterpret_cast<__nv_bfloat16*>(args.out)[o + j * args.ldo] = __float2bfloat16_rn(__uint_as_float(v[j]));
        }
      }
      __syncwarp();  // the next load takes the whole warp
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // Error path: let MMAs and loads still in flight finish before shared and
    // tensor memory are given back.
    if (warp == 1 && lane == 0 && committed) mbar_wait_drain(accum, last_ph, 10000000ull);
    if (tid == 0) {
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 2000000ull) {
      }
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
  if (csize > 1) {
    cluster_sync_all();  // every partial tile is in place
    const int per = (BN + csize - 1) / csize;
    const int c0 = rank * per, nc = min(per, BN - c0);
    const uint32_t red = smem_u32(smem);
    const bool good = !*abort_flag;
    for (int i = tid; i < nc * 64; i += C::THREADS) {
      const int c = c0 + (i >> 6), rp = (i & 63) * 2;
      if (!good || col0 + c >= args.cols || row0 + rp >= args.rows) continue;
      const uint32_t at = red + (uint32_t)(c * 128 + rp) * 4u;
      float2 v[8];  // all loads in flight
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (p < csize) v[p] = ld_peer_f2(at, (uint32_t)p);
      float2 acc = v[0];
#pragma unroll
      for (int p = 1; p < 8; ++p)
        if (p < csize) acc = make_float2(acc.x + v[p].x, acc.y + v[p].y);
      const int64_t o = (int64_t)(col0 + c) * args.ldo + row0 + rp;
      if (F32) *reinterpret_cast<float2*>(reinterpret_cast<float*>(args.out) + o) = acc;
      else *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(args.out) + o) = pack_bf16x2(acc.x, acc.y);
    }
    cluster_sync_all();  // peers may still be reading this CTA's tile
  }
}

template <int BN>
cudaError_t launch_bn(const MxGemmArgs& a, const MxGemmPlan& p, bool dependent, cudaStream_t st) {
  using C = MxCfg<BN>;
  const dim3 grid((unsigned)(p.m_tiles * p.n_tiles * p.cluster));
  const LaunchShape shape{grid, C::THREADS, C::TOTAL, (unsigned)p.cluster, dependent};
  return a.out_f32 ? launch_kernel<mx_gemm_kernel<BN, true>>(shape, st, a)
                   : launch_kernel<mx_gemm_kernel<BN, false>>(shape, st, a);
}

}  // namespace

// Tile width and reduction split: the most CTAs that still run at once (one
// an SM), the smaller split among equals; a rank keeps two reduction blocks
// at least.  A second wave costs more than any split gains: 1000 x 2056 x 1568
// took 9.0 us on 136 CTAs of 128 columns, 10.6 on 272 of 64 and 15.2 on 136
// of 256 columns in two ranks; one token through 4096 x 4096 5.9 us on 32 x 4
// CTAs, 7.0 on 32 x 2 and 7.3 on 32 x 8.
MxGemmPlan plan_mx_gemm(int64_t rows, int64_t cols, int64_t K, int num_sms) {
  MxGemmPlan p{};
  const int kb = (int)((K + kMxKB - 1) / kMxKB);
  const int64_t m_tiles = (rows + 127) / 128;
  const int widest = bn_for_cols((int)(cols < 256 ? cols : 256));
  int64_t best = 0;
  for (int cl = 1; cl <= 8 && (cl == 1 || kb >= 2 * cl); cl *= 2)
    for (int bn = widest; bn >= (widest < 64 ? widest : 64); bn /= 2) {
      const int64_t n = m_tiles * ((cols + bn - 1) / bn) * cl;
      if (p.BN && (n <= best || n > num_sms)) continue;
      best = n;
      p.BN = bn;
      p.cluster = cl;
    }
  p.m_tiles = (int)m_tiles;
  p.n_tiles = (int)((cols + p.BN - 1) / p.BN);
  return p;
}

cudaError_t launch_mx_gemm(const MxGemmArgs& a, const MxGemmPlan& p, bool dependent, cudaStream_t st) {
  switch (p.BN) {
    case 16: return launch_bn<16>(a, p, dependent, st);
    case 32: return launch_bn<32>(a, p, dependent, st);
    case 64: return launch_bn<64>(a, p, dependent, st);
    case 128: return launch_bn<128>(a, p, dependent, st);
    case 256: return launch_bn<256>(a, p, dependent, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qnf4
