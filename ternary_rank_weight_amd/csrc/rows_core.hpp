// Products of 16 weight rows with a few vectors, for kernels that the weights' way from
// memory bounds: every weight is read once, straight into the layout of the matrix instruction's second
// operand (through neither LDS nor a shuffle).  The vectors are the first operand's rows, 16 a tile.
//
// The weights are read in whole aligned 16-byte pieces wherever their rows start: rows 2^apart_bits
// rows apart, at most 8, start at the same place between two multiples of 16 bytes whatever the
// stride, so a workgroup takes sixteen of those, reads them from the multiple at or before their
// start, and the vectors as many columns earlier.
#pragma once
#include "device_common.hpp"
#include "frag.hpp"

namespace externd {

// The bits of how far apart a tile's rows are taken, for rows of ldw entries.
inline int rows_apart_bits(int64_t ldw) {
  int bits = 3;
  while (bits > 0 && ldw % ((int64_t)16 >> bits) == 0) --bits;
  return bits;
}
inline int64_t rows_tiles(int64_t rows, int apart_bits) {
  const int64_t group = (int64_t)16 << apart_bits;
  return ((rows + group - 1) / group) << apart_bits;
}

namespace {

// First row of a tile; its row i is first + (i << apart_bits).  (It may lie past the end.)
__device__ __forceinline__ int64_t tile_row0(int64_t tile, int apart_bits) {
  return ((tile >> apart_bits) << (4 + apart_bits)) + (tile & (((int64_t)1 << apart_bits) - 1));
}
// Entries from the multiple of 16 bytes at or before p up to it.
__device__ __forceinline__ int shift_of(const uint16_t* p) { return (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 7; }

// The eight entries of a row from column c on, in a row of cols entries; those outside
// are some entry of the row.
template <typename T>
__device__ __forceinline__ void load8_around(const T* row, int64_t c, int64_t cols, T (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = row[max<int64_t>(0, min(c + j, cols - 1))];
}

// Vectors of 16-bit entries.  AL: whole pieces of them start on 16 bytes.
template <int NT, bool AL>
struct Rows16 {
  static constexpr int kParts = 1;
  const uint16_t* row[NT];   // the lane's row of each tile
  struct Raw {
    uint16_t v[8];
  };
  __device__ void whole(int n, int64_t c, u32x4 (&f)[1]) const { f[0] = load8<AL>(row[n] + c); }
  __device__ void around(int n, int64_t c, int64_t cols, Raw& raw) const { load8_around(row[n], c, cols, raw.v); }
  __device__ static void pack(const Raw& raw, int64_t from, int64_t to, u32x4 (&f)[1]) { f[0] = pack8(raw.v, from, to); }
};

// Vectors of fp32 entries, entered in two 16-bit parts: the rounded value and what the rounding
// took away.  fp16: after a multiplication by `scale`, a power of two that brings the lane's row into its range.
template <bool BF, int NT>
struct Rows32 {
  static constexpr int kParts = 2;
  const float* row[NT];
  float scale[NT];
  struct Raw {
    float v[8];
    float scale;
  };
  __device__ static void split(const float (&v)[8], float scale, u32x4 (&f)[2]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = BF ? v[j + e] : v[j + e] * scale;
        hi[e] = f32_to_16<BF>(x);
        const float rest = x - f32_from_16<BF>(hi[e]);
        lo[e] = __builtin_isfinite(rest) ? f32_to_16<BF>(rest) : 0u;   // (infinite and NaN are in the first part)
      }
      f[0][j / 2] = hi[0] | (hi[1] << 16);
      f[1][j / 2] = lo[0] | (lo[1] << 16);
    }
  }
  __device__ void whole(int n, int64_t c, u32x4 (&f)[2]) const {
    const u32x4_a4 a = *reinterpret_cast<const u32x4_a4*>(row[n] + c), b = *reinterpret_cast<const u32x4_a4*>(row[n] + c + 4);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(a[j]);
      v[4 + j] = __uint_as_float(b[j]);
    }
    split(v, scale[n], f);
  }
  __device__ void around(int n, int64_t c, int64_t cols, Raw& raw) const {
    load8_around(row[n], c, cols, raw.v);
    raw.scale = scale[n];
  }
  __device__ static void pack(const Raw& raw, int64_t from, int64_t to, u32x4 (&f)[2]) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j >= from && j < to ? raw.v[j] : 0.f;
    split(v, raw.scale, f);
  }
};

// acc[q][n] += the products of matrix q's 16 rows (w[q]: the lane's) with tile n's vectors, over the stretches
// of 64 columns wave, wave + WV, ...; the waves' sums together are the whole product.  shift[q]: as
// shift_of gives it for the matrix (0 with AL).  NX = 1: all matrices are shifted alike; MATS: each has its own
// reading of the vectors.  DEPTH - 1 stretches are on their way ahead of the one that is worked on.
template <bool BF, int MATS, int NT, int WV, bool AL, int NX, int DEPTH, typename X>
__device__ __forceinline__ void rows_product(const uint16_t* const (&w)[MATS], const int (&shift)[MATS], int64_t cols, int wave,
                                             const X& x, f32x4 (&acc)[MATS][NT]) {
  constexpr int S = 2, P = X::kParts;   // 32-column slices per stretch
  const int p = (threadIdx.x & (kWave - 1)) >> 4;
  struct Stage {
    u32x4 w[MATS][S];
  };
  int most = 0, least = 0;
  if constexpr (!AL) {
    most = least = shift[0];
#pragma unroll
    for (int q = 1; q < NX; ++q) {
      most = max(most, shift[q]);
      least = min(least, shift[q]);
    }
  }
  auto shifted = [&](int q) -> int { return AL ? 0 : shift[q % NX]; };
  const int64_t stretches = (cols + most + 32 * S - 1) / (32 * S);
  // whole ones, first to full - 1: not the first where there is a shift, nor what reaches past the end
  const int64_t first = most > 0 ? 1 : 0;
  const int64_t full = max(first, (cols + least) / (32 * S));
  auto fetch = [&](int64_t c, Stage& st) {
#pragma unroll
    for (int q = 0; q < MATS; ++q)
#pragma unroll
      for (int i = 0; i < S; ++i) st.w[q][i] = load8<true>(w[q] + 32 * (S * c + i) + 8 * p - shifted(q));
  };
  auto work = [&](int64_t c, const Stage& st) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      u32x4 f[NX][S][P];
#pragma unroll
      for (int q = 0; q < NX; ++q)
#pragma unroll
        for (int i = 0; i < S; ++i) x.whole(n, 32 * (S * c + i) + 8 * p - shifted(q), f[q][i]);
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e)
#pragma unroll
          for (int q = 0; q < MATS; ++q) acc[q][n] = mfma16<BF>(f[q % NX][i][e], st.w[q][i], acc[q][n]);
    }
  };
  Stage st[DEPTH];
  int64_t c = first + wave;
#pragma unroll
  for (int d = 0; d + 1 < DEPTH; ++d)
    if (c + d * WV < full) fetch(c + d * WV, st[d]);
  // The stretches that are not whole, three at most: a wave each, their narrow loads together.
  for (int64_t odd = wave; odd < first + stretches - full; odd += WV) {
    const int64_t e = odd < first ? 0 : full + odd - first;
#pragma unroll 1
    for (int i = 0; i < S; ++i) {
      const int64_t col = 32 * (S * e + i) + 8 * p;
      uint16_t wv[MATS][8];
      typename X::Raw raw[NX][NT];
#pragma unroll
      for (int q = 0; q < MATS; ++q) load8_around(w[q], col - shifted(q), cols, wv[q]);
#pragma unroll
      for (int q = 0; q < NX; ++q)
#pragma unroll
        for (int n = 0; n < NT; ++n) x.around(n, col - shifted(q), cols, raw[q][n]);
      loads_made();
#pragma unroll
      for (int q = 0; q < MATS; ++q) {
        const int64_t from = shifted(q) - col, to = cols + from;
        const u32x4 wf = pack8(wv[q], from, to);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          u32x4 f[P];
          X::pack(raw[q % NX][n], from, to, f);
#pragma unroll
          for (int e = 0; e < P; ++e) acc[q][n] = mfma16<BF>(f[e], wf, acc[q][n]);
        }
      }
    }
  }
  while (c < full) {
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) {
      if (c < full) {
        if (c + (DEPTH - 1) * WV < full) fetch(c + (DEPTH - 1) * WV, st[(u + DEPTH - 1) % DEPTH]);
        work(c, st[u]);
        c += WV;
      }
    }
  }
}

}  // namespace

}  // namespace externd
