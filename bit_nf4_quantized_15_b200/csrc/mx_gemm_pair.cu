// Large products of two MXFP4 matrices: persistent CTA pairs (tcgen05
// cta_group::2), one 256 x 256 output tile at a time.
//
//   out[row, col] = RN( sum_k A^[row, k] B^[col, k] + mask sum_j Ax[row, j] Bx[col, j] )
//
// rows are tokens, cols weight rows (features).  Each CTA of a pair loads 128
// of the tile's token rows, 128 of its weight rows, the scales of its tokens
// and the scales of all 256 weight rows; the even CTA's MMA thread issues
// 256 x 256 x 64 kind::mxf4 MMAs that read both CTAs' shared memory, and each
// CTA ends with 128 rows x 256 columns of fp32 in its tensor memory.  A CTA
// pulls 35 KB from L2 for 256 reduction steps of 128 x 256 outputs, where the
// single-CTA kernel pulls 51 KB: at the 4-bit rate L2 bandwidth is what a tile
// shape has to spare.
//
// Tensor memory: the accumulator (256 columns), then the scales of each ring
// stage (8 columns of A, 16 of B).  It has no room for two accumulators of
// this size, so the epilogue drains the tile into registers (128 a thread),
// releases the accumulator, and rounds and stores while the next tile's MMAs
// run.  The LoRA term comes first in a tile, see mx_gemm.cu; with dropout
// the epilogue warps have the tile's mask ready (128 bits a thread, evaluated
// during the previous tile's main loop).
//
// Measured, 8192^3: 201 us in a burst (5.47 PFLOP/s), 235 us sustained, where
// the 1000 W cap holds the SM clock down.  (What follows was measured when the
// burst was 213 us.)  A stage of 256 reduction steps takes about 640 cycles of
// which the MMAs need 512: with half of the MMA work taken out (N = 128
// instructions) the kernel was 9 % faster, so the loads, 11 TB/s out of L2,
// weigh as much as the tensor cores.  A tile ends with some 3000 cycles in
// which the MMAs wait: 2300 are the drain itself (128 KB of tensor memory at 57
// bytes a cycle, whatever the load width).  Two accumulators of 192 columns hide it but pull 15 % more bytes per FLOP:
// 262 us against 213.
//
// Barriers (same offsets in both CTAs; "even" ones are used in the even CTA):
//   full[s]   even: both CTAs' bytes of stage s
//   empty[s]  each: the MMAs that read stage s have finished
//   ext       each: the LoRA term of the tile is in tensor memory
//   masked    even: 16 epilogue warps have masked it
//   accum     each: the tile's accumulator is final (fp32 output: a piece of it)
//   drained   even: 16 epilogue warps hold it in registers
// Every wait is bounded; the pair meets at a cluster barrier before tensor
// memory is freed.
#include "engine_util.cuh"
#include "launch.cuh"
#include "mx_util.cuh"
#include "pair_util.cuh"
#include "philox.cuh"

namespace qnf4 {
namespace {

constexpr int kXS = 5;                                  // stages
constexpr int kXA = 16384, kXB = 16384;                 // 128 rows x 128 bytes of codes each
constexpr int kXStage = kXA + kXB + 1024 + 2048;        // + scales of 128 token rows, 256 weight rows
constexpr int kXEpi = 8;                                // epilogue warps: 2 (column halves) x 4 lane quarters
constexpr int kXOut = kXS * kXStage;                    // output staging, 32 rows x 64 bf16 a warp
constexpr int kXBar = kXOut + kXEpi * 4096;
constexpr int kXTotal = kXBar + 256 + 1024;
constexpr int kXThreads = 64 + 32 * kXEpi;
constexpr uint32_t kXAcc = 256, kXSf = 24;              // accumulator columns, scale columns of a stage
constexpr int kXGroup = 8;                              // row tiles of a raster group
static_assert(kXTotal <= 232448 && kXStage % 1024 == 0 && kXAcc + kXS * kXSf <= 512, "budget");

QDEV void umma_mxf4_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                         uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
      : "memory");
}
// One scale tile of each CTA's shared memory to its own tensor memory.
QDEV void tmem_cp_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

struct TileXY {
  int m, n;
};
// Grouped raster: the pairs that run at a time share a few token and weight
// tiles in L2.
QDEV TileXY tile_of(int id, int m_tiles, int n_tiles) {
  const int per = kXGroup * n_tiles, g = id / per, local = id % per;
  const int gs = min(kXGroup, m_tiles - g * kXGroup);
  return TileXY{g * kXGroup + local % gs, local / gs};
}

// Keep bits of 128 consecutive columns of one row, 32 a word; also left in
// memory for the kernel that masks X for dL1, when that is to come.
QDEV void mask_row(uint32_t (&w)[4], const MxPairArgs& a, const PhiloxKey& key, int64_t row, int col) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[i] |= keep8((uint64_t)(row * a.ldo + col + 32 * i + 8 * j) >> 3, key, a.drop.threshold) << (8 * j);
  }
  if (a.keep && row < a.rows && col < a.cols)
    a.keep[row * ((a.ldo + 127) / 128) + col / 128] = make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kXThreads, 1)
    mx_gemm_pair_kernel(const __grid_constant__ MxPairArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kXBar);
  uint64_t* empty = full + kXS;
  uint64_t* ext = empty + kXS;
  uint64_t* masked = ext + 1;
  uint64_t* accum = masked + 1;
  uint64_t* drained = accum + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const int pair = (int)(blockIdx.x >> 1), n_pairs = (int)(gridDim.x >> 1);
  const int m_tiles = (args.rows + 255) / 256, n_tiles = (args.cols + 255) / 256, tiles = m_tiles * n_tiles;
  const int rb = (args.r + 63) / 64;  // 64-wide blocks of the rank
  const int n_ext = F32 ? 0 : kLoraTerms * rb, n_main = args.kb;  // fp32 output: no LoRA term
  const bool use_mask = n_ext && args.drop.threshold;

  if (tid == 0) {
    for (int s = 0; s < kXS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(ext, 1);
    mbar_init(masked, 2 * kXEpi);
    mbar_init(accum, 1);
    mbar_init(drained, 2 * kXEpi);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&args.tmA);
    tma_prefetch_desc(&args.tmB);
    tma_prefetch_desc(&args.tmSA);
    tma_prefetch_desc(&args.tmSB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers and tensor memory exist from here on
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  pdl_trigger();  // not before this CTA has its tensor memory: a dependent CTA must not take it first
  const uint32_t full0 = mapa_shared(smem_u32(full), 0);
  const uint32_t masked0 = mapa_shared(smem_u32(masked), 0);
  const uint32_t drained0 = mapa_shared(smem_u32(drained), 0);
  bool committed = false;
  uint32_t last_ph = 0;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The weight side (B) is not written by the kernel before this one, so its
    // first stages are loaded before that has finished; the tokens' side waits.
    if (lane == 0) {
      auto load_b = [&](int i, int s, const TileXY& xy) {
        const int col0 = xy.n * 256, bcol0 = col0 + (int)rank * 128;
        uint8_t* sb = smem + s * kXStage + kXA;
        const uint32_t bar = full0 + 8u * (uint32_t)s;
        if (i < n_ext) {
          if (leader) mbar_arrive_expect_tx(full + s, 2u * (kXA + kXB));
          if (args.b_mn_ext) {
            tma_load_2d_pair(sb, &args.tmBx, bar, bcol0, i % rb * 64);
            tma_load_2d_pair(sb + 8192, &args.tmBx, bar, bcol0 + 64, i % rb * 64);
          } else {
            tma_load_2d_pair(sb, &args.tmBx, bar, i % rb * 64, bcol0);
          }
        } else {
          if (leader) mbar_arrive_expect_tx(full + s, 2u * kXStage);
          tma_load_2d_pair(sb, &args.tmB, bar, (i - n_ext) * 128, bcol0);
          tma_load_2d_pair(sb + kXB + 1024, &args.tmSB, bar, (i - n_ext) * 256, col0 >> 7);
        }
      };
      auto load_a = [&](int i, int s, const TileXY& xy) {
        const int row0 = xy.m * 256 + (int)rank * 128;
        uint8_t* sa = smem + s * kXStage;
        const uint32_t bar = full0 + 8u * (uint32_t)s;
        if (i < n_ext) {
          tma_load_3d_pair(sa, &args.tmAx, bar, i % rb * 64, i / rb, row0);
        } else {
          tma_load_2d_pair(sa, &args.tmA, bar, (i - n_ext) * 128, row0);
          tma_load_2d_pair(sa + kXA + kXB, &args.tmSA, bar, (i - n_ext) * 256, row0 >> 7);
        }
      };
      const int ahead = min(kXS, n_ext + n_main);  // of the first tile (every pair has one)
      const TileXY first = tile_of(pair, m_tiles, n_tiles);
      for (int i = 0; i < ahead; ++i) load_b(i, i, first);
      pdl_wait();
      for (int i = 0; i < ahead; ++i) load_a(i, i, first);
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += n_pairs) {
        const TileXY xy = tile_of(t, m_tiles, n_tiles);
        for (int i = 0; i < n_ext + n_main; ++i) {
          if (t != pair || i >= ahead) {
            if (!(ok = mbar_wait(empty + s, ph ^ 1u, abort_flag, args.status))) break;
            load_b(i, s, xy);
            load_a(i, s, xy);
          }
          if (++s == kXS) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA (even CTA)
    if (leader) {
      const uint32_t id_ext = idesc_bf16(256, 256, 0, args.b_mn_ext);
      const int64_t tail = args.K - (int64_t)(n_main - 1) * kMxKB;
      const int tail_steps = (int)((tail + 63) / 64);
      const uint32_t base = smem_u32(smem), a0 = kdesc_lo(base), f0 = (uint32_t)sdesc_scales(base + kXA + kXB);
      const uint32_t fhi = (uint32_t)(sdesc_scales(0) >> 32);
      const bool one = elect_one();
      int s = 0;
      uint32_t sph = 0, ph = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += n_pairs) {
        for (int i = 0; i < n_ext + n_main; ++i) {
          const int in_sum = F32 ? i % kMxPiece : i;  // stage of this accumulation
          if (in_sum == 0) {
            if (!(ok = warp_poll(drained, ph ^ 1u, abort_flag, args.status, lane))) break;
            tc_fence_after();
          }
          if (!(ok = warp_poll(full + s, sph, abort_flag, args.status, lane))) break;
          tc_fence_after();
          if (i < n_ext) {
            const uint8_t* sa = smem + s * kXStage;
            if (one) {
              const int steps = (min(64, args.r - i % rb * 64) + 15) / 16;  // zeros past r
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (kk < steps)
                  umma_pair(tmem, operand_desc(sa, 0, kk), operand_desc(sa + kXA, args.b_mn_ext, kk), id_ext,
                            (i | kk) != 0);
              umma_commit_both(empty + s);
              if (i == n_ext - 1) umma_commit_both(ext);
            }
            // MMAs of another kind follow: let these finish (and be masked)
            if (i == n_ext - 1) {
              if (!(ok = warp_poll(use_mask ? masked : ext, ph, abort_flag, args.status, lane))) break;
              tc_fence_after();
            }
          } else if (one) {
            const int steps = i == n_ext + n_main - 1 ? tail_steps : 4;
            const uint32_t so = (uint32_t)s * (kXStage >> 4);
            const uint32_t sf = tmem + kXAcc + (uint32_t)s * kXSf;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint64_t f = ((uint64_t)fhi << 32) | (f0 + so + 32 * h);
              tmem_cp_scales_pair(sf + 4 * h, f);
              tmem_cp_scales_pair(sf + 8 + 8 * h, f + 64);
              tmem_cp_scales_pair(sf + 12 + 8 * h, f + 128);
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk < steps)
                umma_mxf4_pair(tmem, kdesc(a0 + so + 2 * kk), kdesc(a0 + so + (kXA >> 4) + 2 * kk),
                               idesc_mxf4(256, 256, 2 * (kk & 1)), sf + 4 * (kk >> 1), sf + 8 + 8 * (kk >> 1),
                               (in_sum | kk) != 0);
            }
            umma_commit_both(empty + s);
          }
          __syncwarp();
          if (++s == kXS) {
            s = 0;
            sph ^= 1u;
          }
          if (i + 1 == n_ext + n_main || (F32 && in_sum + 1 == kMxPiece)) {
            if (one) umma_commit_both(accum);
            committed = true;
            last_ph = ph;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {  // what has been issued, for the error path to wait for
        if (one) umma_commit_both(accum);
        committed = true;
        last_ph = ph;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q4 = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16) + (uint32_t)(half * 128);
    const int rl = (int)rank * 128 + q4 * 32 + lane;
    const PhiloxKey key = use_mask ? philox_key(args.drop) : PhiloxKey{0, 0, 0, 0};
    uint32_t mw[4] = {0, 0, 0, 0};
    if (use_mask && pair < tiles) {
      const TileXY xy = tile_of(pair, m_tiles, n_tiles);
      mask_row(mw, args, key, (int64_t)xy.m * 256 + rl, xy.n * 256 + half * 128);
    }
    uint32_t ph = 0;
    for (int t = pair; t < tiles; t += n_pairs) {
      const TileXY xy = tile_of(t, m_tiles, n_tiles);
      if (use_mask) {
        if (!warp_wait(ext, ph, abort_flag, args.status, lane)) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[16];
            tmem_ld16(tl + 32 * i + 16 * h, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (!((mw[i] >> (16 * h + j)) & 1u)) v[j] = 0u;
            tmem_st16(tl + 32 * i + 16 * h, v);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(masked0);
        if (t + n_pairs < tiles) {  // the next tile's mask, while this one's MMAs run
          const TileXY nx = tile_of(t + n_pairs, m_tiles, n_tiles);
          mask_row(mw, args, key, (int64_t)nx.m * 256 + rl, nx.n * 256 + half * 128);
        }
      }
      const int col = xy.n * 256 + half * 128;
      if constexpr (F32) {
        float sum[8][16] = {};  // of the pieces so far
        bool ok = true;
#pragma unroll 1
        for (int i = 0; i < n_main && ok; i += kMxPiece, ph ^= 1u) {
          ok = warp_wait(accum, ph, abort_flag, args.status, lane);
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t v[16];
            tmem_ld16(tl + (uint32_t)(16 * q), v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[q][j] = __fadd_rn(sum[q][j], __uint_as_float(v[j]));
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(drained0);
        }
        if (!ok) break;
        const int64_t row = (int64_t)xy.m * 256 + rl;
        float* dst = reinterpret_cast<float*>(args.out) + row * args.ldo + col;
        if (row < args.rows) {
#pragma unroll
          for (int c = 0; c < 128; c += 4)
            if (col + c < args.cols)
              *reinterpret_cast<float4*>(dst + c) = make_float4(sum[c / 16][c % 16], sum[c / 16][c % 16 + 1],
                                                                sum[c / 16][c % 16 + 2], sum[c / 16][c % 16 + 3]);
        }
        __syncwarp();
      } else {
        if (!warp_wait(accum, ph, abort_flag, args.status, lane)) break;
        tc_fence_after();
        uint32_t v[8][16];  // the whole row half, loads all in flight; packed once the accumulator is released
#pragma unroll
        for (int q = 0; q < 8; ++q) tmem_ld16(tl + (uint32_t)(16 * q), v[q]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(drained0);
        // Out by TMA in two halves of 64 columns, through this warp's buffer: a
        // thread has one row, and its own 16-byte stores would each touch half
        // a sector of another row.
        uint8_t* buf = smem + kXOut + (warp - 2) * 4096;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (lane == 0) bulk_wait_read<0>();  // the buffer's last store has read it
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t* w = v[4 * h + (c >> 1)] + 8 * (c & 1);
            const auto two = [&](int j) { return pack_bf16x2(__uint_as_float(w[j]), __uint_as_float(w[j + 1])); };
            *reinterpret_cast<uint4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                make_uint4(two(0), two(2), two(4), two(6));
          }
          fence_proxy_async_smem();
          __syncwarp();
          const int r0 = xy.m * 256 + (int)rank * 128 + q4 * 32, c0 = col + 64 * h;
          if (lane == 0 && r0 < args.rows && c0 < args.cols) {
            tma_store_2d(&args.tmOut, buf, c0, r0);
            bulk_commit();
          }
        }
        ph ^= 1u;
      }
    }
    if (!F32 && lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // Error path: let MMAs and loads still in flight finish before the pair
    // meets and frees its memory.
    if (warp == 1 && lane == 0 && committed) mbar_wait_drain(accum, last_ph, 10000000ull);
    if (tid == 0) {
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 2000000ull) {
      }
    }
    __syncthreads();
  }
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_mx_gemm_pair(const MxPairArgs& a, int num_sms, bool dependent, cudaStream_t st) {
  const int64_t tiles = (int64_t)((a.rows + 255) / 256) * ((a.cols + 255) / 256);
  const int pairs = num_sms / 2;
  const LaunchShape shape{dim3(2u * (unsigned)(tiles < pairs ? tiles : pairs)), kXThreads, kXTotal, 1, dependent};
  return a.out_f32 ? launch_kernel<mx_gemm_pair_kernel<true>>(shape, st, a)
                   : launch_kernel<mx_gemm_pair_kernel<false>>(shape, st, a);
}

}  // namespace qnf4
