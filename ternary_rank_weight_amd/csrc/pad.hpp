// Small passes around the tiled products: zeros, and rows copied to where 16-byte loads can read them.
#pragma once
#include <algorithm>

#include "device_common.hpp"
#include "frag.hpp"
#include "gated_plan.hpp"

namespace externd {

namespace {

// Zeros: a weight gradient of no tokens, and k_gated_tops' results before it.
template <typename T>
__global__ void k_fill_zero(T* __restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    p[i] = 0;
}

// Up to three matrices of 16-bit entries copied into rows of ldp entries (a
// multiple of 64), zero past their columns: what the 16-byte loads need where
// the caller's rows are not aligned.  (Reading such rows through registers in every
// step instead took 83 us for the forward of 777 tokens at 1001 x 1237; the copies
// take 5 us, and the forward on them 24.)
struct PadArgs {
  const uint16_t* src[3];
  uint16_t* dst[3];
  int64_t rows[3], ld[3], cols[3], ldp[3];
  uint32_t* zeros;   // words to clear besides, or null
  int64_t zeros_n;
};
__global__ __launch_bounds__(256) void k_pad_rows(PadArgs a) {
  const int w = blockIdx.y;
  if (a.zeros && w == 0)
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.zeros_n; i += (int64_t)gridDim.x * 256) a.zeros[i] = 0u;
  const int64_t ldp = a.ldp[w], per = ldp / 8, total = a.rows[w] * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per, c = (i - row * per) * 8, left = a.cols[w] - c;
    const uint16_t* p = a.src[w] + row * a.ld[w] + c;
    const u32x4 v = left >= 8 ? load8<false>(p) : load8_part(p, left);
    *reinterpret_cast<u32x4*>(a.dst[w] + row * ldp + c) = v;
  }
}

unsigned blocks(int64_t items) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(ceil_div64(items, 256), 1 << 15)); }

bool rows_aligned(const void* p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && ld < (1 << 22);
}
size_t region(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

}  // namespace externd
