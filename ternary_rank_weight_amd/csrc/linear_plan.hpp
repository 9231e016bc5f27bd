// How the linear layer's products are run.  Host code without HIP.
#pragma once
#include "gated_plan.hpp"

namespace externd {

inline bool linear_takes_rows(int64_t tokens, int64_t cols, int64_t rows, bool aligned, int cus) {
  return tokens <= kRowsMostTokens;
}

// The least of an estimate in microseconds, as plan_of; a tile of 256 x 192 (mid) and one of 256 x 256
// may be split in every product.
inline GatedPlan plan_linear(int mode, int64_t m, int64_t n, int64_t steps, int cus) {
  GatedPlan best = {kPair, 1};
  double least = 1e300;
  for (const GatedKind kind : {kBig, kMid, kPair, kDeep}) {
    const int64_t bm = kind == kBig || kind == kMid ? 256 : 128, bn = kind == kBig ? 256 : kind == kMid ? 192 : 128;
    const int64_t tiles = ceil_div64(m, bm) * ceil_div64(n, bn);
    const int64_t most = kind == kPair ? 1 : 16;
    for (int64_t splits = 1; splits <= most && splits <= std::max<int64_t>(1, steps / 4); ++splits) {
      const int64_t units = tiles * splits;
      if (kind == kDeep && units > cus) break;
      const double per = (double)ceil_div64(std::max<int64_t>(steps, 1), splits);
      const double rounds = (double)ceil_div64(units, (int64_t)cus * (kind == kPair ? 2 : 1));
      double us = kind == kBig    ? rounds * (per * 1.4 + 6.0)
                  : kind == kMid  ? rounds * (per * 1.2 + 6.0)
                  : kind == kPair ? rounds * (per * 0.95 + 4.0)
                                  : per * 0.45 + 8.0;
      if (splits > 1) us += 4.0 + (double)m * (double)n * 4.0 * (double)(splits * 2) / 4e6;
      if (us < least) {
        least = us;
        best = {kind, splits};
      }
    }
  }
  return best;
}

// dx from dz in one part or two.  For few tokens the two are stacked as twice the rows, as in the
// gated block.
inline GatedPlan plan_linear_dx(int64_t tokens, int64_t cols, int64_t rows, bool parts, int cus) {
  const bool stack = parts && tokens <= 64 && tiles_of(kDx, 2 * tokens, cols, false) <= cus;
  GatedPlan p = plan_linear(kDx, stack ? 2 * tokens : tokens, cols, (parts && !stack ? 2 : 1) * steps_of(rows), cus);
  if (stack) {
    if (p.kind != kDeep) p = {kDeep, 1};
    p.stacked = 2;
  }
  return p;
}
inline GatedPlan plan_linear_dw(int64_t tokens, int64_t cols, int64_t rows, bool parts, int cus) {
  return plan_linear(kLinDw, rows, cols, (parts ? 2 : 1) * steps_of(tokens), cus);
}

}  // namespace externd
