// How the products of the gated block and of the linear layer are run: which kernel, which tiles, how
// many splits.  Host code without HIP.
#pragma once
#include <stdint.h>

#include <algorithm>

namespace externd {

// The gated block's forward, dx and both dW; the linear layer's forward and dW (its dx is kDx).
enum GatedProduct { kFwd = 0, kDx = 1, kDw = 2, kLin = 3, kLinDw = 4 };
constexpr int kBK = 64;   // contraction entries per step: two 16x16x32 products, 128 bytes of a row

// How a product is run: 256 x 256 tiles, 128 x 128 tiles two to a CU, or one to a CU
// with loads three steps ahead; and the splits of its contraction.  The linear layer's also
// in 256 x 192 tiles, and in 128 x 64 with loads three steps ahead.
enum GatedKind { kBig, kPair, kDeep, kMid, kSlim };
struct GatedPlan {
  GatedKind kind;
  int64_t splits;
  int64_t stacked = 1;   // 2 (kDeep only): output rows are the sums of the first and the second half of a's
};

inline int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t padded(int64_t n, int64_t to) { return ceil_div64(n, to) * to; }

// Most tokens of the forward's few-token kernel (gated_rows.hip).  Past 16 tokens a workgroup
// of it reads two tiles of x for its one tile of each weight matrix, and time grows with what
// it reads, the columns times the tiles that one CU takes in turn.  Aligned operands (a product
// that needs no copies) go to the tiled product where that is long: 32 tokens in that
// kernel against 33 in the tiled product, in us,
//   9728 x 9728: 121, 86   300 x 9728: 36, 19   9728 x 2560: 35, 30   4096 x 4096: 19, 20
//   9728 x 1024: 14, 13    1024 x 2560: 13, 17  4096 x 2048: 11, 16
// Rows that are not aligned, 32 tokens at 9728 x 2559: 53 and 58.
constexpr int kRowsMostTokens = 32, kRowsShortTokens = 16;
constexpr int64_t kRowsMostColumns = 5000;

inline bool gated_takes_rows(int64_t tokens, int64_t cols, int64_t rows, bool aligned, int cus) {
  if (tokens <= kRowsShortTokens || tokens > kRowsMostTokens) return tokens <= kRowsShortTokens;
  return !aligned || cols * std::max<int64_t>((rows + 15) / 16, cus) <= kRowsMostColumns * cus;
}

// How a product of m x n outputs (forward: n hidden units; dW: m rows of each of
// the two gradients) over `steps` steps is run: the least of an estimate in
// microseconds, from K = 2560 and F = 9728.
//   big   256 x 256 tiles, one workgroup a CU: 1.4 us a step and 6 a tile;
//   pair  128 x 128 tiles, two a CU: 0.95 us a step and 4 a tile each;
//   deep  128 x 128 tiles, one a CU with loads three steps ahead, where there are
//         no more units than CUs: 0.45 us a step and 8 in all.
// A split costs its sums' way to memory and back.  (Low by a quarter for few steps on
// ragged rows: 777 tokens at 1001 x 1237, 17, 27 and 19 us against 24, 33 and 26 measured.)
inline int64_t tiles_of(int mode, int64_t m, int64_t n, bool big) {
  const int64_t b = big ? 256 : 128;
  return (mode == kDw ? 2 : 1) * ceil_div64(m, b) * ceil_div64(n, mode == kFwd ? b / 2 : b);
}
inline GatedPlan plan_of(int mode, int64_t m, int64_t n, int64_t steps, int cus) {
  GatedPlan best = {kPair, 1};
  double least = 1e300;
  for (const GatedKind kind : {kBig, kPair, kDeep}) {
    const int64_t tiles = tiles_of(mode, m, n, kind == kBig);
    // (dx is split at 256 x 256 too: its contraction is the longest and its tiles the fewest)
    const int64_t most = kind == kDeep || (kind == kBig && mode == kDx) ? 16 : 1;
    for (int64_t splits = 1; splits <= most && splits <= std::max<int64_t>(1, steps / 4); ++splits) {
      const int64_t units = tiles * splits;
      if (kind == kDeep && units > cus) break;
      const double per = (double)ceil_div64(std::max<int64_t>(steps, 1), splits);
      const double rounds = (double)ceil_div64(units, (int64_t)cus * (kind == kPair ? 2 : 1));
      double us = kind == kBig ? rounds * (per * 1.4 + 6.0) : kind == kPair ? rounds * (per * 0.95 + 4.0) : per * 0.45 + 8.0;
      if (splits > 1) us += 4.0 + (double)(mode == kDx ? 1 : 2) * (double)m * (double)n * 4.0 * (double)(splits * 2) / 4e6;
      if (us < least) {
        least = us;
        best = {kind, splits};
      }
    }
  }
  return best;
}
inline int64_t steps_of(int64_t inner) { return inner / kBK; }

// dx.  For few tokens the two parts of dg and du are stacked as twice the rows, which are
// added at the end: a 128-row tile has room for both, so the second costs no matrix
// instruction.  Otherwise they follow each other in the contraction.
inline GatedPlan plan_dx(int64_t tokens, int64_t cols, int64_t rows, int cus) {
  const bool stack = tokens <= 64 && tiles_of(kDx, 2 * tokens, cols, false) <= cus;
  GatedPlan p = plan_of(kDx, stack ? 2 * tokens : tokens, cols, (stack ? 2 : 4) * steps_of(rows), cus);
  if (stack) {
    if (p.kind != kDeep) p = {kDeep, 1};
    p.stacked = 2;
  }
  return p;
}
inline GatedPlan plan_dw(int64_t tokens, int64_t cols, int64_t rows, int cus) {
  return plan_of(kDw, rows, cols, 2 * steps_of(tokens), cus);
}
inline int64_t part_floats(int mode, int64_t m, int64_t n, const GatedPlan& p) {
  return p.splits * p.stacked > 1 ? p.splits * p.stacked * (mode == kFwd || mode == kDw ? 2 : 1) * m * n : 0;
}

}  // namespace externd
