// How the MXFP4 linear layer's kernels share out their work: integer
// arithmetic that the host (plans, workspace sizes) and the kernels use alike.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#ifdef __CUDACC__
#define QPLAN __host__ __device__ inline
#else
#define QPLAN inline
#endif

namespace qnf4 {

// A tile whose units several CTAs share leaves its partial sums in slots of
// 128 x r fp32, one for each pair of a tile and a CTA.  Tiles and CTAs both take
// the units in order, so along the units a new pair raises the tile's number,
// the CTA's or both, and tile + CTA is a number of its own for every pair;
// a tile's slots follow one another in the order of its CTAs.
QPLAN int64_t mx_slot(int64_t tile, int64_t cta) { return tile + cta; }
inline size_t mx_slot_bytes(int64_t tiles, int64_t ctas, int r) {
  return (size_t)(tiles + ctas) * 128 * (size_t)r * sizeof(float);
}

// ------------------------------------------------- Q(X) and D (mx_prep.cu)
struct MxPrepPlan {
  int units_per_tile;   // units (128 rows x 256 columns) of a row tile
  int64_t units;
  bool direct;          // a cluster of `cluster` CTAs finishes a row tile
  int cluster;
  int grid;             // CTAs
  size_t part_bytes;    // partial slots (not direct); never less for more rows
};

// Units [lo, hi) of CTA c.
QPLAN int64_t prep_unit(int64_t units, int grid, int64_t c) { return c * units / grid; }
// CTA that owns unit u.
QPLAN int prep_owner(int64_t units, int grid, int64_t u) { return (int)(((u + 1) * grid - 1) / units); }

// Up to 8 row tiles of up to two units a CTA go to clusters of 8 (16 for up to
// 4 tiles) that finish their tile alone, and so do tiles of one unit; the rest
// is cut into equal runs of units, with a second kernel for what the runs
// share.  Forward with 1024 features, both measured: 1 x 8192 13.6 us on a
// cluster, 15.1 in runs; 600 x 4096 22.9 and 22.6 (and a launch less); 2000 x
// 4096 30.2 and 24.7 (16 clusters of 8 do not all fit at once).  max_cluster: 16,
// or 8 on a device (a partition of one) that has no room for one of 16.
inline MxPrepPlan plan_mx_prep(int64_t M, int64_t C, int r, int num_sms, int max_cluster) {
  MxPrepPlan p{};
  p.units_per_tile = (int)((C + 255) / 256);
  const int64_t tiles = (M + 127) / 128;
  p.units = tiles * p.units_per_tile;
  p.cluster = 1;
  while (p.cluster < (tiles <= 4 ? max_cluster : 8) && 2 * p.cluster <= p.units_per_tile) p.cluster *= 2;
  p.direct = (tiles <= 8 && p.units_per_tile <= 2 * p.cluster) || p.units_per_tile == 1;
  if (p.direct) {
    p.grid = (int)(tiles * p.cluster);
    return p;
  }
  p.cluster = 1;
  p.grid = (int)(p.units < num_sms ? p.units : num_sms);
  p.part_bytes = mx_slot_bytes(tiles, p.grid, r);
  return p;
}

// ------------------------------------------- adapter gradients (mx_grad.cu)
constexpr int kGradPiece = 8;              // 64-token stages of a unit, at most
constexpr int kGradMaxStages = 6;          // of the ring
constexpr int kGradBudget = 220 * 1024;    // bytes of the ring

struct MxGradShare {  // how the units are shared out
  int64_t units0, units;  // 128 columns x a piece of the tokens: of problem 0, of both
  int w0, grid;           // cost of a unit of problem 0 (the other's: 2), CTAs
};
struct MxGradPlan {
  MxGradShare sh;
  int piece, pieces;      // 64-token stages of a unit, units of a tile
  int n16, nbuf, vboxes, stages;
  size_t part_bytes;      // partial slots, the tiles of dL1 first
};
enum MxGradMask { kMaskNone, kMaskEvaluated, kMaskBits };

// Runs are equal in cost: a masked unit of dL1 may count 3, others 2 (the mask
// takes about as long as half a unit's loads).  CTA of a unit, and the
// first unit of a CTA.
QPLAN int64_t grad_cost(const MxGradShare& a, int64_t u) {
  return u < a.units0 ? u * a.w0 : a.units0 * a.w0 + (u - a.units0) * 2;
}
QPLAN int grad_owner(const MxGradShare& a, int64_t u) {
  return (int)(grad_cost(a, u) * a.grid / grad_cost(a, a.units));
}
QPLAN int64_t grad_first(const MxGradShare& a, int64_t c) {
  const int64_t x = (c * grad_cost(a, a.units) + a.grid - 1) / a.grid, x0 = a.units0 * a.w0;
  return x <= x0 ? (x + a.w0 - 1) / a.w0 : a.units0 + (x - x0 + 1) / 2;
}

inline MxGradPlan plan_mx_grad(int64_t M, int64_t cols0, int64_t cols1, int r, MxGradMask mask, int num_sms) {
  MxGradPlan p{};
  const int64_t t0 = (cols0 + 127) / 128, t1 = (cols1 + 127) / 128;
  if (!t0 && !t1) return p;
  if (!t0) mask = kMaskNone;
  // As few pieces of the tokens as their greatest length allows, cut evenly.  The
  // masked stages of a unit follow one another at 1.2 us, so with dropout pieces
  // of about half that length are worth their second kernel and balance the
  // CTAs while those do not have a longer unit each (gradients of 512 x 512 x
  // 512, r = 64: 21 us in two pieces, 27 in one, but without dropout 17.8 and
  // 16.3; backward of 1024 x 4096 x 4096: 44 us in four, 49 in two).
  const int64_t stages = (M + 63) / 64;
  int64_t n = (stages + kGradPiece - 1) / kGradPiece;
  if (mask == kMaskEvaluated && (t0 + t1) * n < num_sms)
    n = std::max(n, (stages + kGradPiece / 4) / (kGradPiece / 2));
  p.piece = (int)((stages + n - 1) / n);
  p.pieces = (int)((stages + p.piece - 1) / p.piece);
  p.sh.units0 = t0 * p.pieces;
  p.sh.units = p.sh.units0 + t1 * p.pieces;
  // (with the bits at hand a CTA alone with its unit has no use for the weight:
  // backward of 1024 x 4096 x 4096 40 us, 44 with it; 4096 x 11008 x 4096 167 us
  // without, 162 with it)
  p.sh.w0 = mask == kMaskEvaluated || (mask == kMaskBits && p.sh.units > num_sms) ? 3 : 2;
  // no more CTAs than leave each the cost of a unit, so that none is empty
  // (the slots of a tile's CTAs are then all written)
  const int64_t cost = grad_cost(p.sh, p.sh.units), fit = cost / p.sh.w0;
  p.sh.grid = (int)(fit < num_sms ? fit : num_sms);
  if (p.pieces > 1) p.part_bytes = mx_slot_bytes(t0 + t1, p.sh.grid, r);
  p.n16 = (3 * r + 15) / 16 * 16;
  const int r16 = (r + 15) / 16 * 16;
  p.nbuf = 2 * p.n16 + r16 <= 512 ? 2 : 1;
  p.vboxes = (p.n16 + 63) / 64;
  const int stage = 16384 + p.vboxes * 8192;
  p.stages = kGradBudget / stage < kGradMaxStages ? kGradBudget / stage : kGradMaxStages;
  return p;
}

// The most that any plan for up to M tokens takes (with dropout or without, one
// gradient or both): none while the tokens are a single piece in all of them.
inline size_t mx_grad_part_bound(int64_t M, int64_t K, int64_t N, int r, int num_sms) {
  const int64_t stages = (M + 63) / 64;
  if ((stages + kGradPiece / 4) / (kGradPiece / 2) <= 1 && stages <= kGradPiece) return 0;
  return mx_slot_bytes((K + 127) / 128 + (N + 127) / 128, num_sms, r);
}

}  // namespace qnf4
