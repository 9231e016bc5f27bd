// How the linear layer's products are run.  Host code without HIP.
#pragma once
#include "gated_plan.hpp"

namespace externd {

// Most tokens of the forward's few-token kernel (linear_rows.hip).  Its time grows with the tokens, whose entries each
// tile of weight rows reads again, and with what one CU reads, the columns times its tiles; the tiled product's hardly does.
// Aligned operands, that kernel and the tiled product, in us:
//   cols x rows      1 token     4           16          17          32
//   4096 x 4096      9.3 15.3    8.6 15.3    10.1 15.3   11.6 15.6   14.4 15.9
//   2560 x 9728      13.6 17.0   13.1 17.1   17.2 17.7   18.6 17.8   23.6 18.7
//   9728 x 2560      14.4 18.6   14.9 19.2   19.5 19.7   22.5 19.3   28.9 20.0
//   9728 x 9728      40.3 39.9   45.2 39.1   57.7 39.9   63.6 40.0   78.7 40.5
//   9728 x 300       12.4 12.0   14.0 12.4   18.7 12.4   21.1 12.8   27.3 12.8
// Rows that are not aligned, 2559 x 9728: 14.8 37.4, 16.2 36.7, 23.9 37.1, 27.4 37.2, 38.9 37.6.
inline int64_t linear_rows_most(int64_t cols, int64_t rows, bool aligned, int cus) {
  const int64_t tiles = ceil_div64(rows, 16), read = cols * std::max<int64_t>(tiles, cus);
  if (!aligned || read <= (int64_t)5000 * cus) return 32;
  return read <= (int64_t)10000 * cus && 2 * tiles >= cus ? 16 : 3;
}
inline bool linear_takes_rows(int64_t tokens, int64_t cols, int64_t rows, bool aligned, int cus) {
  return tokens <= linear_rows_most(cols, rows, aligned, cus);
}

// The least of an estimate in microseconds, as plan_of; a tile of 256 x 192 (mid) and one of 256 x 256
// may be split in every product.
inline GatedPlan plan_linear(int mode, int64_t m, int64_t n, int64_t steps, int cus, double* estimate = nullptr) {
  GatedPlan best = {kPair, 1};
  double least = 1e300;
  for (const GatedKind kind : {kBig, kMid, kPair, kDeep, kSlim}) {
    const int64_t bm = kind == kBig || kind == kMid ? 256 : 128, bn = kind == kBig ? 256 : kind == kMid ? 192 : kind == kSlim ? 64 : 128;
    const int64_t tiles = ceil_div64(m, bm) * ceil_div64(n, bn);
    const int64_t most = kind == kPair ? 1 : 16;
    for (int64_t splits = 1; splits <= most && splits <= std::max<int64_t>(1, steps / 4); ++splits) {
      const int64_t units = tiles * splits;
      if ((kind == kDeep || kind == kSlim) && units > cus) break;
      const double per = (double)ceil_div64(std::max<int64_t>(steps, 1), splits);
      const double rounds = (double)ceil_div64(units, (int64_t)cus * (kind == kPair ? 2 : 1));
      double us = kind == kBig    ? rounds * (per * 1.5 + 8.0)
                  : kind == kMid  ? rounds * (per * 1.2 + 6.0)
                  : kind == kPair ? rounds * (per * 0.95 + 4.0)
                  : kind == kSlim ? per * 0.33 + 8.0
                                  : per * 0.45 + 8.0;
      if (splits > 1) us += 4.0 + (double)m * (double)n * 4.0 * (double)(splits * 2) / 4e6;
      if (us < least) {
        least = us;
        best = {kind, splits};
      }
    }
  }
  if (estimate) *estimate = least;
  return best;
}

// dx from dz in one part or two.  For few tokens the two are stacked as twice the rows, as in the
// gated block.
inline GatedPlan plan_linear_dx(int64_t tokens, int64_t cols, int64_t rows, bool parts, int cus, double* estimate = nullptr) {
  const bool stack = parts && tokens <= 64 && tiles_of(kDx, 2 * tokens, cols, false) <= cus;
  GatedPlan p = plan_linear(kDx, stack ? 2 * tokens : tokens, cols, (parts && !stack ? 2 : 1) * steps_of(rows), cus, estimate);
  if (stack) {
    if (p.kind != kDeep && p.kind != kSlim) p = {kDeep, 1};
    p.stacked = 2;
  }
  return p;
}
inline GatedPlan plan_linear_dw(int64_t tokens, int64_t cols, int64_t rows, bool parts, int cus, double* estimate = nullptr) {
  return plan_linear(kLinDw, rows, cols, (parts ? 2 : 1) * steps_of(tokens), cus, estimate);
}

// dx and dW in one launch, the first `dx` workgroups for dx and `dw` for dW; dx = 0: in two.  Either both in whole 128 x 64
// tiles, where each has no more of them than CUs; or both in 256 x 192 tiles, where the product of fewer tiles has a
// workgroup for each and the other takes the rest of the CUs, if the longer of them is estimated to end before
// one after the other would.  bf16, tokens, cols x rows, dx and dW apart and in one launch, us:
//   2264, 2296 x 2872: 52 + 40, 62    2656, 1880 x 2488: 47 + 43, 55    2206, 2968 x 1704: 34 + 37, 50
//   2048, 2560 x 9728: 109 + 105, 221   512, 9728 x 2560: 38 + 37, 68   1106, 1872 x 912: 14 + 12, 27
// (the first of the lower row, and the last, the estimate takes wrongly, by 3 in 100).
struct LinearJoin {
  int64_t dx, dw;
  GatedKind kind;
};
inline LinearJoin linear_join(int64_t tokens, int64_t cols, int64_t rows, bool parts, int cus) {
  double ux, uw;
  const GatedPlan px = plan_linear_dx(tokens, cols, rows, parts, cus, &ux), pw = plan_linear_dw(tokens, cols, rows, parts, cus, &uw);
  const LinearJoin none = {0, 0, kSlim};
  if (px.stacked != 1) return none;
  auto tiles = [&](int64_t m, int64_t bm, int64_t bn) { return ceil_div64(m, bm) * ceil_div64(cols, bn); };
  if (px.kind == kSlim && pw.kind == kSlim && px.splits == 1 && pw.splits == 1)
    return {tiles(tokens, 128, 64), tiles(rows, 128, 64), kSlim};
  const int64_t x = tiles(tokens, 256, 192), w = tiles(rows, 256, 192), least = std::min(x, w), rest = (cus - least) / 8 * 8;
  if (rest <= 0) return none;
  auto time = [&](int64_t t, int64_t inner) {   // of a product of t tiles
    return (t == least ? 1.0 : (double)ceil_div64(t, rest)) * ((double)((parts ? 2 : 1) * steps_of(inner)) * 1.2 + 6.0);
  };
  if (std::max(time(x, rows), time(w, tokens)) > 0.95 * (ux + uw)) return none;
  const int64_t most = std::min(std::max(x, w), rest);
  return x <= w ? LinearJoin{x, most, kMid} : LinearJoin{most, w, kMid};
}

}  // namespace externd
