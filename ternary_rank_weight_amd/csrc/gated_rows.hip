// The gated block's forward pass for a few tokens (up to 32):
// h = act(x Wg^T) (x Wu^T) with every weight read once from memory, which is
// what bounds it: 2 F K 16-bit weights against one product each per token.
// F = 9728, K = 2560, one token: 22 us where the weights come from memory, 4.5 TB/s (reading
// 1 GiB: 5.3), 20 where one layer's 100 MB stay in the last-level cache; K = 2559: 27 and 22.
// (Nontemporal loads: 27 and 26; 36 and 34: a line is taken by two of them.)
//
// A workgroup takes 16 hidden units (neighbours, where rows are aligned).  Its waves
// take every WV-th stretch of 64 columns; a lane reads 16 bytes of its row (lane % 16) of each matrix per 32
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

struct RowsArgs {
  const uint16_t *x, *w[2];
  int64_t tokens, cols, rows, ldx, ldw;
  int apart_bits;   // rows 2^apart_bits apart start at the same place between multiples of 16 bytes
  uint16_t* h;
  float* save[2];
  int act;
};

// The eight entries of a row from column c on, in a row of cols entries; those outside
// are some entry of the row.
__device__ __forceinline__ void load8_near(const uint16_t* row, int64_t c, int64_t cols, uint16_t (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = row[max<int64_t>(0, min(c + j, cols - 1))];
}

// The weights are read in whole aligned 16-byte pieces, wherever their rows start.  Rows
// `apart` rows apart, at most 8, start at the same place between two multiples of 16
// bytes, whatever the stride, so a workgroup takes sixteen of those, reads them from the
// multiple at or before their start, and x as many columns earlier.  (Whole 128-byte
// lines, from rows up to 64 apart: 26.4 us against 28.6 at 2560 x 9727, one token, 25.5
// against 23.8 at 9728 x 2568.)
// AL: no operand is shifted, and x is read in aligned pieces too.  NX = 1: Wg and Wu are
// shifted alike; 2: each has its own shift, and its own reading of x.
template <bool BF, int NT, int WV, bool AL, int NX>
__global__ __launch_bounds__(WV * kWave) void k_gated_rows(RowsArgs a) {
  constexpr int S = 2;   // 32-column slices per stretch
  __shared__ float red[WV][2][256];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int r = lane & 15, p = lane >> 4;
  const int64_t apart = (int64_t)1 << a.apart_bits;
  const int64_t row0 = ((int64_t)(blockIdx.x >> a.apart_bits) << (4 + a.apart_bits)) + (blockIdx.x & (apart - 1));
  if (row0 >= a.rows) return;
  const int64_t row = row0 + apart * r < a.rows ? row0 + apart * r : row0;   // (past the end: the first again)
  const uint16_t* wr[2] = {a.w[0] + row * a.ldw, a.w[1] + row * a.ldw};
  // the columns that would lie before each matrix's rows in their first piece
  int64_t shift[2] = {0, 0};
  if constexpr (!AL) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      shift[q] = (int64_t)((reinterpret_cast<uintptr_t>(a.w[q < NX ? q : 0] + row0 * a.ldw) >> 1) & 7);
  }
  const uint16_t* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xr[n] = a.x + min<int64_t>(n * 16 + r, a.tokens - 1) * a.ldx;
  f32x4 acc[2][NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[0][n] = acc[1][n] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Stage {
    u32x4 w[2][S];
  };
  const int64_t most = max(shift[0], shift[1]);
  const int64_t stretches = (a.cols + most + 32 * S - 1) / (32 * S);
  // whole ones, first to full - 1: not the first where there is a shift, nor what
  // reaches past the end
  const int64_t first = most > 0 ? 1 : 0;
  const int64_t full = max(first, (a.cols + min(shift[0], shift[1])) / (32 * S));
  auto fetch = [&](int64_t c, Stage& st) {   // a whole stretch
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < S; ++i) st.w[q][i] = load8<true>(wr[q] + 32 * (S * c + i) + 8 * p - shift[q]);
  };
  auto multiply = [&](const u32x4 (&w)[2][S], const u32x4 (&x)[NX][S], int n) {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) acc[q][n] = mfma16<BF>(x[q % NX][i], w[q][i], acc[q][n]);
  };
  auto work = [&](int64_t c, const Stage& st) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      u32x4 xf[NX][S];
#pragma unroll
      for (int q = 0; q < NX; ++q)
#pragma unroll
        for (int i = 0; i < S; ++i) xf[q][i] = load8<AL>(xr[n] + 32 * (S * c + i) + 8 * p - shift[q]);
      multiply(st.w, xf, n);
    }
  };
  // two stretches ahead of the one that is worked on
  Stage st[3];
  int64_t c = first + wave;
  if (c < full) fetch(c, st[0]);
  if (c + WV < full) fetch(c + WV, st[1]);
  // The stretches that are not whole, three at most: a wave each.  (With each narrow load
  // waiting for the one before it, these took 14 us.)
  if (wave < first + stretches - full) {
    const int64_t e = wave < first ? 0 : full + wave - first;
#pragma unroll 1
    for (int i = 0; i < S; ++i) {
      const int64_t col = 32 * (S * e + i) + 8 * p;
      uint16_t wv[2][8], xv[NX][NT][8];
#pragma unroll
      for (int q = 0; q < 2; ++q) load8_near(wr[q], col - shift[q], a.cols, wv[q]);
#pragma unroll
      for (int q = 0; q < NX; ++q)
#pragma unroll
        for (int n = 0; n < NT; ++n) load8_near(xr[n], col - shift[q], a.cols, xv[q][n]);
      loads_made();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t from = shift[q] - col, to = a.cols + from;
        const u32x4 w = pack8(wv[q], from, to);
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[q][n] = mfma16<BF>(pack8(xv[q % NX][n], from, to), w, acc[q][n]);
      }
    }
  }
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

#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n) __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][q][(4 * p + e) * 16 + r] = acc[q][n][e];
    __syncthreads();
    for (int o = threadIdx.x; o < 256; o += WV * kWave) {
      const int64_t t = n * 16 + (o >> 4), unit = row0 + apart * (o & 15);
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

template <bool BF, int NT, bool AL, int NX>
hipError_t launch(const RowsArgs& q, hipStream_t s) {
  const int64_t group = (int64_t)16 << q.apart_bits, tiles = ((q.rows + group - 1) / group) << q.apart_bits;
  // few row tiles: twice the waves on each, to have the whole matrix on its way at once
  // (not where a wave needs more than the 128 registers that sixteen waves leave it).  Weights
  // from memory, one token, in us with 8 and 16 waves: 1024 x 2560 (64 tiles) 8.7, 8.0;
  // 4096 x 4096 (256) 15.5, 14.5; 6144 x 2560 (384) 16.0, 16.8; 8000 x 2560 (500) 17.9, 17.9;
  // 9728 x 2560 (608) 23.2, 24.0; 16384 x 2560 (1024) 32.6, 33.8.
  constexpr int most = NX == 2 && NT == 2 ? 8 : 16;
  if (tiles < 512) {
    hipLaunchKernelGGL((k_gated_rows<BF, NT, most, AL, NX>), dim3((unsigned)tiles), dim3(most * kWave), 0, s, q);
  } else {
    hipLaunchKernelGGL((k_gated_rows<BF, NT, 8, AL, NX>), dim3((unsigned)tiles), dim3(8 * kWave), 0, s, q);
  }
  return hipGetLastError();
}

template <bool BF, bool AL, int NX>
hipError_t pick(const RowsArgs& q, hipStream_t s) {
  if (q.tokens <= 16) return launch<BF, 1, AL, NX>(q, s);
  return launch<BF, 2, AL, NX>(q, s);
}

template <bool BF>
hipError_t any(const RowsArgs& q, bool aligned, hipStream_t s) {
  const bool alike = ((reinterpret_cast<uintptr_t>(q.w[0]) ^ reinterpret_cast<uintptr_t>(q.w[1])) & 15) == 0;
  if (aligned) return pick<BF, true, 1>(q, s);
  return alike ? pick<BF, false, 1>(q, s) : pick<BF, false, 2>(q, s);
}

}  // namespace

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
  q.apart_bits = 3;
  while (q.apart_bits > 0 && a.ldw % ((int64_t)16 >> q.apart_bits) == 0) --q.apart_bits;
  q.h = static_cast<uint16_t*>(a.h);
  q.save[0] = a.g;
  q.save[1] = a.u;
  q.act = a.act;
  const bool al = gated_is_aligned(a);
  return a.dtype == EXTERND_BF16 ? any<true>(q, al, s) : any<false>(q, al, s);
}

}  // namespace externd
