// Host check of how the MXFP4 linear layer's kernels share out their work
// (csrc/mx_plan.h), run by tests/test_mx_host.py: every unit has one CTA, a
// partial slot belongs to one (tile, CTA) and lies inside the workspace, the
// slots that the second kernel adds are those that were written, and no
// workspace region falls with the number of tokens.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "mx_plan.h"

using namespace qnf4;

static long failures = 0, plans = 0;
#define NEED(c)                                             \
  do {                                                      \
    if (!(c) && ++failures < 10) std::printf("line %d: %s\n", __LINE__, #c); \
  } while (0)

// units [first(c), first(c + 1)) of CTA c; `per` consecutive units are a tile
template <class First, class Owner>
static void check_slots(int64_t units, int64_t per, int grid, size_t bytes, int r, First first, Owner owner) {
  const int64_t tiles = units / per, n = (int64_t)(bytes / (128 * sizeof(float) * r));
  std::vector<int64_t> of(n, -1);  // tile of a slot
  NEED(first(0) == 0 && first(grid) == units);
  for (int c = 0; c < grid; ++c) {
    NEED(first(c) < first(c + 1));
    for (int64_t u = first(c); u < first(c + 1); ++u) {
      NEED(owner(u) == c);
      const int64_t tile = u / per, s = mx_slot(tile, c);
      NEED(s >= 0 && s < n);
      if (s < 0 || s >= n) return;
      NEED(of[s] == -1 || (of[s] == tile && u > first(c)));
      of[s] = tile;
    }
  }
  for (int64_t t = 0; t < tiles; ++t)
    for (int c = owner(t * per); c <= owner(t * per + per - 1); ++c) NEED(of[mx_slot(t, c)] == t);
  ++plans;
}

int main() {
  std::srand(1);
  const auto log_rand = [](int lo, int hi) {
    double x = lo;
    while (x < hi && std::rand() % 8) x *= 1.0 + (std::rand() % 1000) / 900.0;
    return (int64_t)(x < hi ? x : hi);
  };
  for (int i = 0; i < 20000; ++i) {
    const int64_t M = log_rand(1, 9000), C = log_rand(1, 900) * 32, N = log_rand(1, 900) * 32;
    const int r = 8 * (1 + std::rand() % 16), sms = std::rand() % 4 ? 148 : 1 + std::rand() % 160;
    const int most = std::rand() % 2 ? 16 : 8;  // largest cluster of the device
    const MxPrepPlan p = plan_mx_prep(M, C, r, sms, most);
    const int64_t tiles = (M + 127) / 128;
    NEED(p.units == tiles * ((C + 255) / 256) && p.grid >= 1);
    if (p.direct) {
      NEED(p.grid == tiles * p.cluster && p.part_bytes == 0);
      NEED(p.cluster <= most && p.cluster <= p.units_per_tile && 128 % p.cluster == 0);
    } else {
      NEED(p.grid <= sms && p.cluster == 1);
      check_slots(p.units, p.units_per_tile, p.grid, p.part_bytes, r,
                  [&](int64_t c) { return prep_unit(p.units, p.grid, c); },
                  [&](int64_t u) { return prep_owner(p.units, p.grid, u); });
    }
    NEED(plan_mx_prep(M, C, r, sms, 8).part_bytes >= p.part_bytes);  // the workspace holds either
    NEED(plan_mx_prep(M + 1 + std::rand() % 300, C, r, sms, most).part_bytes >= p.part_bytes);
    for (int k = 0; k < 9; ++k) {
      const int64_t c0 = k % 3 == 2 ? 0 : C, c1 = k % 3 == 1 ? 0 : N;
      const MxGradPlan g = plan_mx_grad(M, c0, c1, r, (MxGradMask)(k / 3), sms);
      NEED((int64_t)g.piece * g.pieces * 64 >= M && (int64_t)g.piece * (g.pieces - 1) * 64 < M);
      NEED(g.piece <= kGradPiece && g.sh.grid >= 1 && g.sh.grid <= sms);
      NEED(g.part_bytes <= mx_grad_part_bound(M, C, N, r, sms));
      if (g.pieces > 1)
        check_slots(g.sh.units, g.pieces, g.sh.grid, g.part_bytes, r, [&](int64_t c) { return grad_first(g.sh, c); },
                    [&](int64_t u) { return (int64_t)grad_owner(g.sh, u); });
    }
    NEED(mx_grad_part_bound(M + 1 + std::rand() % 300, C, N, r, sms) >= mx_grad_part_bound(M, C, N, r, sms));
  }
  std::printf("plans=%ld failures=%ld\n", plans, failures);
  return failures ? 1 : 0;
}
