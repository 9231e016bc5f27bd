// The linear layer's forward pass for a few tokens (up to 32): y = act(x W^T + bias) + residual with
// every weight read once from memory, which is what bounds it (rows_core.hpp): one token at 2560 x 9728, bf16, 13.6 us
// (3.7 TB/s); 7 tokens at 3001 x 1237, fp16 and unaligned, 5.6.
#include <algorithm>

#include "activation.hpp"
#include "device_common.hpp"
#include "frag.hpp"
#include "linear.hpp"
#include "rows_core.hpp"

namespace externd {

namespace {

struct LinearRows {
  const uint16_t *x, *w, *bias, *residual;
  int64_t tokens, cols, rows, ldx, ldw, ldr;
  int apart_bits, act;
  uint16_t* y;
  float* z;
};

template <bool BF, int NT, int WV, bool AL>
__global__ __launch_bounds__(WV * kWave) void k_linear_rows(LinearRows a) {
  __shared__ float red[WV][256];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15, p = lane >> 4;
  const int64_t row0 = tile_row0(blockIdx.x, a.apart_bits);
  if (row0 >= a.rows) return;
  const int64_t mine = row0 + ((int64_t)r << a.apart_bits);
  const uint16_t* const w[1] = {a.w + (mine < a.rows ? mine : row0) * a.ldw};   // (past the end: the first again)
  const int shift[1] = {AL ? 0 : shift_of(a.w + row0 * a.ldw)};
  Rows16<NT, AL> x;
#pragma unroll
  for (int n = 0; n < NT; ++n) x.row[n] = a.x + min<int64_t>(n * 16 + r, a.tokens - 1) * a.ldx;   // (a missing token: the last)
  f32x4 acc[1][NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[0][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  rows_product<BF, 1, NT, WV, AL, 1>(w, shift, (int)a.cols, wave, x, acc);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n) __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][(4 * p + e) * 16 + r] = acc[0][n][e];
    __syncthreads();
    for (int o = threadIdx.x; o < 256; o += WV * kWave) {
      const int64_t t = n * 16 + (o >> 4), row = row0 + ((int64_t)(o & 15) << a.apart_bits);
      if (t >= a.tokens || row >= a.rows) continue;
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < WV; ++q) v += red[q][o];
      if (a.bias) v += f32_from_16<BF>(a.bias[row]);
      const int64_t at = t * a.rows + row;
      if (a.z) a.z[at] = v;
      if (a.act != EXTERND_ACT_NONE) v = act_value(a.act, v);
      if (a.residual) v += f32_from_16<BF>(a.residual[t * a.ldr + row]);
      a.y[at] = (uint16_t)f32_to_16<BF>(v);
    }
  }
}

template <bool BF, int NT, bool AL>
hipError_t launch(const LinearRows& q, hipStream_t s) {
  const int64_t tiles = rows_tiles(q.rows, q.apart_bits);
  if (tiles < 512) {
    hipLaunchKernelGGL((k_linear_rows<BF, NT, 16, AL>), dim3((unsigned)tiles), dim3(16 * kWave), 0, s, q);
  } else {
    hipLaunchKernelGGL((k_linear_rows<BF, NT, 8, AL>), dim3((unsigned)tiles), dim3(8 * kWave), 0, s, q);
  }
  return hipGetLastError();
}

template <bool BF, bool AL>
hipError_t pick(const LinearRows& q, hipStream_t s) {
  return q.tokens <= 16 ? launch<BF, 1, AL>(q, s) : launch<BF, 2, AL>(q, s);
}

}  // namespace

hipError_t run_linear_rows(const LinearArgs& a, hipStream_t s) {
  LinearRows q = {};
  q.x = static_cast<const uint16_t*>(a.x);
  q.w = static_cast<const uint16_t*>(a.w);
  q.bias = static_cast<const uint16_t*>(a.bias);
  q.residual = static_cast<const uint16_t*>(a.residual);
  q.tokens = a.tokens;
  q.cols = a.cols;
  q.rows = a.rows;
  q.ldx = a.ldx;
  q.ldw = a.ldw;
  q.ldr = a.ldr;
  q.apart_bits = rows_apart_bits(a.ldw);
  q.act = a.act;
  q.y = static_cast<uint16_t*>(a.y);
  q.z = a.z;
  const bool al = linear_is_aligned(a);
  if (a.dtype == EXTERND_BF16) return al ? pick<true, true>(q, s) : pick<true, false>(q, s);
  return al ? pick<false, true>(q, s) : pick<false, false>(q, s);
}

}  // namespace externd
