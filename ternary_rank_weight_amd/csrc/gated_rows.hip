// The gated block's forward pass for a few tokens (up to 32):
// h = act(x Wg^T) (x Wu^T) with every weight read once from memory, which is
// what bounds it: 2 F K 16-bit weights against one product each per token.
// F = 9728, K = 2560, one token: 20 us, 5.0 TB/s (a large copy: 5.16).
//
// A workgroup takes 16 hidden units.  Its waves take every WV-th stretch of 64
// columns; a lane reads 16 bytes of its row (lane % 16) of each matrix per 32
// columns straight into the layout of the matrix instruction's second operand,
// so weights pass through neither LDS nor a shuffle.  Tokens are the first
// operand's rows, 16 per tile (a missing token repeats the last one, and its
// row is dropped).  The waves' fp32 sums are joined in LDS in wave order.
#include <algorithm>

#include "activation.hpp"
#include "device_common.hpp"
#include "frag.hpp"
#include "kernels.hpp"

namespace externd {

namespace {

// Most tokens of this form.  Past 16 tokens a workgroup reads two tiles of x for its one
// tile of each weight matrix, and time grows with what it reads, the columns times the
// tiles that one CU takes in turn.  Aligned operands (a product that needs no copies) go
// to the tiled product where that is long: 32 tokens here against 33 there, in us,
//   9728 x 9728: 121, 86   300 x 9728: 36, 19   9728 x 2560: 35, 30   4096 x 4096: 19, 20
//   9728 x 1024: 14, 13    1024 x 2560: 13, 17  4096 x 2048: 11, 16
// Rows that are not aligned (9728 x 2559): 61 here, 67 there.
constexpr int kRowsMostTokens = 32, kRowsShortTokens = 16;
constexpr int64_t kRowsMostColumns = 5000;

struct RowsArgs {
  const uint16_t *x, *w[2];
  int64_t tokens, cols, rows, ldx, ldw;
  uint16_t* h;
  float* save[2];
  int act;
};

// AL: every row starts 16-byte aligned and cols is a multiple of 8.
template <bool BF, int NT, int WV, bool AL>
__global__ __launch_bounds__(WV * kWave) void k_gated_rows(RowsArgs a) {
  constexpr int S = 2;   // 32-column slices per stretch
  __shared__ float red[WV][2][256];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int r = lane & 15, p = lane >> 4;
  const int64_t row0 = (int64_t)blockIdx.x * 16;
  const int64_t row = min(row0 + r, a.rows - 1);   // (a row past the end repeats the last)
  const uint16_t* wp[2] = {a.w[0] + row * a.ldw + 8 * p, a.w[1] + row * a.ldw + 8 * p};
  const uint16_t* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xp[n] = a.x + min<int64_t>(n * 16 + r, a.tokens - 1) * a.ldx + 8 * p;
  f32x4 acc[2][NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[0][n] = acc[1][n] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Stage {
    u32x4 w[2][S];
  };
  const int64_t stretches = (a.cols + 32 * S - 1) / (32 * S), full = a.cols / (32 * S);
  auto fetch = [&](int64_t c, Stage& st) {   // a whole stretch
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < S; ++i) st.w[q][i] = load8<AL>(wp[q] + 32 * (S * c + i));
  };
  auto multiply = [&](const u32x4 (&w)[2][S], const u32x4 (&x)[S], int n) {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) acc[q][n] = mfma16<BF>(x[i], w[q][i], acc[q][n]);
  };
  auto work = [&](int64_t c, const Stage& st) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      u32x4 xf[S];
#pragma unroll
      for (int i = 0; i < S; ++i) xf[i] = load8<AL>(xp[n] + 32 * (S * c + i));
      multiply(st.w, xf, n);
    }
  };
  // two stretches ahead of the one that is worked on
  Stage st[3];
  int64_t c = wave;
  if (c < full) fetch(c, st[0]);
  if (c + WV < full) fetch(c + WV, st[1]);
  while (c < full) {
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      if (c < full) {
        if (c + 2 * WV < full) fetch(c + 2 * WV, st[(u + 2) % 3]);
        work(c, st[u]);
        c += WV;
      }
    }
  }
  if (c < stretches) {   // the last, partial stretch
    u32x4 w[2][S];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < S; ++i) w[q][i] = load8_part(wp[q] + 32 * (S * c + i), a.cols - 32 * (S * c + i) - 8 * p);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      u32x4 xf[S];
#pragma unroll
      for (int i = 0; i < S; ++i) xf[i] = load8_part(xp[n] + 32 * (S * c + i), a.cols - 32 * (S * c + i) - 8 * p);
      multiply(w, xf, n);
    }
  }

#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n) __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][q][(4 * p + e) * 16 + r] = acc[q][n][e];
    __syncthreads();
    for (int o = threadIdx.x; o < 256; o += WV * kWave) {
      const int64_t t = n * 16 + (o >> 4), unit = row0 + (o & 15);
      if (t >= a.tokens || unit >= a.rows) continue;
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int w = 0; w < WV; ++w) v[q] += red[w][q][o];
      const int64_t at = t * a.rows + unit;
      a.h[at] = (uint16_t)f32_to_16<BF>(act_value(a.act, v[0]) * v[1]);
      if (a.save[0]) {
        a.save[0][at] = v[0];
        a.save[1][at] = v[1];
      }
    }
  }
}

template <bool BF, int NT, bool AL>
hipError_t launch(const RowsArgs& q, hipStream_t s) {
  const int64_t tiles = (q.rows + 15) / 16;
  // few row tiles: twice the waves on each, to have the whole matrix on its way at once
  if (tiles < 512) {
    hipLaunchKernelGGL((k_gated_rows<BF, NT, 16, AL>), dim3((unsigned)tiles), dim3(16 * kWave), 0, s, q);
  } else {
    hipLaunchKernelGGL((k_gated_rows<BF, NT, 8, AL>), dim3((unsigned)tiles), dim3(8 * kWave), 0, s, q);
  }
  return hipGetLastError();
}

template <bool BF, bool AL>
hipError_t pick(const RowsArgs& q, hipStream_t s) {
  if (q.tokens <= 16) return launch<BF, 1, AL>(q, s);
  return launch<BF, 2, AL>(q, s);
}

}  // namespace

bool gated_takes_rows(int64_t tokens, int64_t cols, int64_t rows, bool aligned, int cus) {
  if (tokens <= kRowsShortTokens || tokens > kRowsMostTokens) return tokens <= kRowsShortTokens;
  return !aligned || cols * std::max<int64_t>((rows + 15) / 16, cus) <= kRowsMostColumns * cus;
}

hipError_t run_gated_rows(const GatedArgs& a, hipStream_t s) {
  RowsArgs q;
  q.x = static_cast<const uint16_t*>(a.x);
  q.w[0] = static_cast<const uint16_t*>(a.wg);
  q.w[1] = static_cast<const uint16_t*>(a.wu);
  q.tokens = a.tokens;
  q.cols = a.cols;
  q.rows = a.rows;
  q.ldx = a.ldx;
  q.ldw = a.ldw;
  q.h = static_cast<uint16_t*>(a.h);
  q.save[0] = a.g;
  q.save[1] = a.u;
  q.act = a.act;
  const bool al = gated_is_aligned(a);
  if (a.dtype == EXTERND_BF16) return al ? pick<true, true>(q, s) : pick<true, false>(q, s);
  return al ? pick<false, true>(q, s) : pick<false, false>(q, s);
}

}  // namespace externd
