// Products of 16 weight rows with a few vectors, for kernels that the weights' way from
// memory bounds: every weight is read once, straight into the layout of the matrix instruction's second
// operand (through neither LDS nor a shuffle).  The vectors are the first operand's rows, 16 a tile.
//
// The weights are read in whole aligned 16-byte pieces wherever their rows start: rows 2^apart_bits
// rows apart, at most 8, start at the same place between two multiples of 16 bytes whatever the
// stride, so a workgroup takes sixteen of those, reads them from the multiple at or before their
// start, and the vectors as many columns earlier.
#pragma once
#include <type_traits>

#include "device_common.hpp"
#include "frag.hpp"
#include "rows_plan.hpp"

namespace externd {

namespace {

// A value as three of 16 bits whose sum it is: 24 bits of fp32, as 3 x 8 of bf16 (cut off: a rounding up might leave the
// range) or 3 x 11 of fp16.  Infinite and NaN are in the first; fp16 ends at its smallest step, 2^-24.
template <bool BF>
__device__ __forceinline__ void split16(float v, uint32_t (&part)[3]) {
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    part[e] = BF ? __float_as_uint(v) >> 16 : f32_to_16<BF>(v);
    v -= f32_from_16<BF>(part[e]);
    if (e == 0 && !__builtin_isfinite(v)) v = 0.f;
  }
}

// First row of a tile; its row i is first + (i << apart_bits).  (It may lie past the end.)
__device__ __forceinline__ int64_t tile_row0(int64_t tile, int apart_bits) {
  return ((tile >> apart_bits) << (4 + apart_bits)) + (tile & (((int64_t)1 << apart_bits) - 1));
}
// Entries from the multiple of 16 bytes at or before p up to it.
__device__ __forceinline__ int shift_of(const uint16_t* p) { return (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 7; }

// Eight entries from a place of any alignment, as they are read: the dwords that hold them (as load8<false>).
struct Any8 {
  u32x4 v;
  uint32_t w;
  __device__ void load(const uint16_t* q) {
    const uint32_t odd = (uint32_t)(reinterpret_cast<uintptr_t>(q) >> 1) & 1u;
    v = *reinterpret_cast<const u32x4_a4*>(q - odd);
    w = *reinterpret_cast<const uint32_t*>(q - odd + (odd ? 8 : 6));
  }
  __device__ u32x4 get(const uint16_t* q) const {
    const uint32_t sh = ((uint32_t)(reinterpret_cast<uintptr_t>(q) >> 1) & 1u) * 16u;
    u32x4 r;
    r.x = __builtin_amdgcn_alignbit(v.y, v.x, sh);
    r.y = __builtin_amdgcn_alignbit(v.z, v.y, sh);
    r.z = __builtin_amdgcn_alignbit(v.w, v.z, sh);
    r.w = __builtin_amdgcn_alignbit(w, v.w, sh);
    return r;
  }
};

// The eight entries of a row from column c on, in a row of cols entries; those outside are 0.  They are read where
// they are nearest and still inside, at column `at`, and what lies there before c or past its eight is masked: so two
// edges of the same c and cols have the same entry of their row in each place.  AL: c and cols are multiples of 8.
// A row of fewer than eight entries is read entry by entry.
template <bool AL>
struct Edge8 {
  typename std::conditional<AL, u32x4, Any8>::type v;
  __device__ static int nearest(int c, int cols) { return max(0, min(c, cols - 8)); }
  __device__ void load(const uint16_t* row, int c, int cols) {
    if constexpr (AL) {
      v = load8<true>(row + nearest(c, cols));
    } else if (cols >= 8) {
      v.load(row + nearest(c, cols));
    } else {
      uint16_t e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = row[max(0, min(c + j, cols - 1))];
      v.v = pack8(e, -c, cols - c);
    }
  }
  __device__ u32x4 get(const uint16_t* row, int c, int cols) const {
    const int at = nearest(c, cols), from = c - at, to = from + 8;   // entries of `at` that are wanted
    if constexpr (AL) {
      return from == 0 ? v : u32x4{0u, 0u, 0u, 0u};
    } else {
      if (cols < 8) return v.v;
      u32x4 r = v.get(row + at);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        r[k] &= (2 * k >= from && 2 * k < to ? 0xffffu : 0u) | (2 * k + 1 >= from && 2 * k + 1 < to ? 0xffff0000u : 0u);
      return r;
    }
  }
};

// Vectors of 16-bit entries.  AL: whole pieces of them start on 16 bytes.
template <int NT, bool AL>
struct Rows16 {
  static constexpr int kParts = 1;
  const uint16_t* row[NT];   // the lane's row of each tile
  struct Whole {
    typename std::conditional<AL, u32x4, Any8>::type v;
  };
  struct Edge {
    Edge8<AL> v;
  };
  __device__ void load(int n, int c, Whole& raw) const {
    if constexpr (AL) raw.v = load8<true>(row[n] + c);
    else raw.v.load(row[n] + c);
  }
  __device__ void finish(int n, int c, const Whole& raw, u32x4 (&f)[1]) const {
    if constexpr (AL) f[0] = raw.v;
    else f[0] = raw.v.get(row[n] + c);
  }
  __device__ void load_edge(int n, int c, int cols, Edge& raw) const { raw.v.load(row[n], c, cols); }
  __device__ void finish_edge(int n, int c, int cols, const Edge& raw, u32x4 (&f)[1]) const { f[0] = raw.v.get(row[n], c, cols); }
};

// Vectors of fp32 entries, entered in three 16-bit parts; fp16 after a multiplication by `scale`, a power of two
// that brings the lane's row into its range.
template <bool BF>
struct RowsSplit {
  static constexpr int kParts = 3;
  const float* row;
  float scale;   // fp16
  struct Whole {
    u32x4 a, b;
  };
  struct Edge {
    float v[8];
  };
  __device__ void split(const float (&v)[8], u32x4 (&f)[kParts]) const {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint32_t part[2][kParts];
#pragma unroll
      for (int e = 0; e < 2; ++e) split16<BF>(BF ? v[j + e] : v[j + e] * scale, part[e]);
#pragma unroll
      for (int k = 0; k < kParts; ++k) f[k][j / 2] = part[0][k] | (part[1][k] << 16);
    }
  }
  __device__ void load(int, int c, Whole& raw) const {
    raw.a = *reinterpret_cast<const u32x4_a4*>(row + c);
    raw.b = *reinterpret_cast<const u32x4_a4*>(row + c + 4);
  }
  __device__ void finish(int, int, const Whole& raw, u32x4 (&f)[kParts]) const {
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(raw.a[j]);
      v[4 + j] = __uint_as_float(raw.b[j]);
    }
    split(v, f);
  }
  // (the entries of Edge8's places: those of a row of eight and more that lie nearest)
  __device__ void load_edge(int, int c, int cols, Edge& raw) const {
    const int at = cols >= 8 ? max(0, min(c, cols - 8)) : c;
#pragma unroll
    for (int j = 0; j < 8; ++j) raw.v[j] = row[max(0, min(at + j, cols - 1))];
  }
  __device__ void finish_edge(int, int c, int cols, const Edge& raw, u32x4 (&f)[kParts]) const {
    const int at = cols >= 8 ? max(0, min(c, cols - 8)) : c;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = at + j >= max(c, 0) && at + j < min(c + 8, cols) ? raw.v[j] : 0.f;
    split(v, f);
  }
};

// acc[q][n] += the products of matrix q's 16 rows (w[q]: the lane's) with tile n's vectors, over the stretches
// of 64 columns wave, wave + WV, ...; the waves' sums together are the whole product.  shift[q]: as
// shift_of gives it for the matrix (0 with AL).  NX = 1: all matrices are shifted alike; MATS: each has its own
// reading of the vectors.  A stretch is on its way ahead of the one that is worked on.
template <bool BF, int MATS, int NT, int WV, bool AL, int NX, typename X>
__device__ __forceinline__ void rows_product(const uint16_t* const (&w)[MATS], const int (&shift)[MATS], int cols, int wave,
                                             const X& x, f32x4 (&acc)[MATS][NT]) {
  constexpr int S = 2, P = X::kParts;   // 32-column slices per stretch
  const int p = (threadIdx.x & (kWave - 1)) >> 4;
  struct Stage {
    u32x4 w[MATS][S];
  };
  struct Vectors {
    typename X::Whole v[NT][NX][S];
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
  const int stretches = (cols + most + 32 * S - 1) / (32 * S);
  // whole ones, first to full - 1: not the first where there is a shift, nor what reaches past the end
  const int first = most > 0 ? 1 : 0;
  const int full = max(first, (cols + least) / (32 * S));
  auto fetch = [&](int c, Stage& st) {
#pragma unroll
    for (int q = 0; q < MATS; ++q)
#pragma unroll
      for (int i = 0; i < S; ++i) st.w[q][i] = load8<true>(w[q] + (32 * (S * c + i) + 8 * p - shifted(q)));
  };
  // A stretch sets out while the one before it is worked on, the vectors' entries before the weights, and in the
  // steady loop no load hangs on a condition: loads come back in order, and a wait for the vectors would otherwise be
  // one for weights that were sent for later.  (Three stretches ahead instead of one: 13.8 against 12.8 us for one
  // token at 2560 x 9728, no less anywhere.)
  auto load_x = [&](int c, Vectors& xs) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < NX; ++q)
#pragma unroll
        for (int i = 0; i < S; ++i) x.load(n, 32 * (S * c + i) + 8 * p - shifted(q), xs.v[n][q][i]);
  };
  auto work = [&](int c, const Stage& st, const Vectors& xs) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < S; ++i) {
        u32x4 f[NX][P];
#pragma unroll
        for (int q = 0; q < NX; ++q) x.finish(n, 32 * (S * c + i) + 8 * p - shifted(q), xs.v[n][q][i], f[q]);
#pragma unroll
        for (int e = 0; e < P; ++e)
#pragma unroll
          for (int q = 0; q < MATS; ++q) acc[q][n] = mfma16<BF>(f[q % NX][e], st.w[q][i], acc[q][n]);
      }
  };
  // The stretches that are not whole, three at most: a wave each, the last ones, which have the fewest others.
  // Their loads and the first whole stretch's travel together.
  const int odd = WV - 1 - wave, odds = first + stretches - full;
  auto edges = [&](int odd) { return 32 * S * (odd < first ? 0 : full + odd - first) + 8 * p; };
  Edge8<AL> we[MATS][S];
  typename X::Edge xe[NX][NT][S];
  auto load_edges = [&](int at) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int q = 0; q < MATS; ++q) we[q][i].load(w[q], at + 32 * i - shifted(q), cols);
#pragma unroll
      for (int q = 0; q < NX; ++q)
#pragma unroll
        for (int n = 0; n < NT; ++n) x.load_edge(n, at + 32 * i - shifted(q), cols, xe[q][n][i]);
    }
    loads_made();
  };
  auto work_edges = [&](int at) {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int q = 0; q < MATS; ++q) {
        const int c = at + 32 * i - shifted(q);
        const u32x4 wf = we[q][i].get(w[q], c, cols);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          u32x4 f[P];
          x.finish_edge(n, c, cols, xe[q % NX][n][i], f);
#pragma unroll
          for (int k = 0; k < P; ++k) acc[q][n] = mfma16<BF>(f[k], wf, acc[q][n]);
        }
      }
  };
  Stage st[2];
  Vectors xs[2];
  int c = first + wave;
  const bool any = full > first;   // (a wave without whole stretches reads the last one)
  auto begin = [&] {
    load_x(min(c, full - 1), xs[0]);
    fetch(min(c, full - 1), st[0]);
  };
  // (one branch: were the edges' loads and their use in two, the loop would wait for loads in every round)
  if (odd < odds) {
    load_edges(edges(odd));
    if (any) begin();
    work_edges(edges(odd));
    for (int more = odd + WV; more < odds; more += WV) {   // (fewer waves than such stretches)
      load_edges(edges(more));
      work_edges(edges(more));
    }
  } else if (any) {
    begin();
  }
  if (!any) return;
  for (; c + 2 * WV < full; c += 2 * WV) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      load_x(c + (u + 1) * WV, xs[1 - u]);
      fetch(c + (u + 1) * WV, st[1 - u]);
      __builtin_amdgcn_sched_barrier(0);
      work(c + u * WV, st[u], xs[u]);
    }
  }
  if (c >= full) return;
  if (c + WV < full) {   // two left, or one
    load_x(c + WV, xs[1]);
    fetch(c + WV, st[1]);
    work(c, st[0], xs[0]);
    work(c + WV, st[1], xs[1]);
  } else {
    work(c, st[0], xs[0]);
  }
}

}  // namespace

}  // namespace externd
