// The experts of the mixture-of-experts layer, for a few tokens:
//   h = act(Wg_e x) (Wu_e x) for every slot (a token and one of its experts e),
//   y[t] = the sum over t's slots of weight * Wd_e h.
// Bound by the weights of the experts that are chosen, which are read once for each group of up to 16 of an expert's
// slots (rows_core.hpp).  h and each slot's result are fp32: the layer's output is rounded once.  h enters the second
// product in two 16-bit parts; in fp16, whose range it may leave, multiplied by a power of two for each slot.
#include <algorithm>

#include "activation.hpp"
#include "device_common.hpp"
#include "frag.hpp"
#include "gated.hpp"
#include "moe.hpp"
#include "rows_core.hpp"

namespace externd {

namespace {

struct UpArgs {
  const uint16_t *x, *w[2];
  int64_t cols, rows, ldx, ldw, stride;   // stride: from one expert to the next
  int top, apart_bits, act;
  const int32_t* groups_n;
  const MoeGroup* groups;
  const int32_t* sorted;
  uint32_t* tops;
  float* h;
  int64_t ldh;
};

template <bool BF, int WV, bool AL, int NX>
__global__ __launch_bounds__(WV * kWave) void k_moe_up(UpArgs a) {
  __shared__ float red[WV][2][256];
  if ((int)blockIdx.y >= *a.groups_n) return;
  const MoeGroup g = a.groups[blockIdx.y];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int r = lane & 15, p = lane >> 4;
  const int64_t row0 = tile_row0(blockIdx.x, a.apart_bits);
  if (row0 >= a.rows) return;
  const int64_t mine = row0 + ((int64_t)r << a.apart_bits), row = mine < a.rows ? mine : row0;   // (past the end: the first again)
  const int64_t at_expert = g.expert * a.stride;
  const uint16_t* const w[2] = {a.w[0] + at_expert + row * a.ldw, a.w[1] + at_expert + row * a.ldw};
  const int shift[2] = {AL ? 0 : shift_of(a.w[0] + at_expert + row0 * a.ldw), AL ? 0 : shift_of(a.w[1] + at_expert + row0 * a.ldw)};
  Rows16<1, AL> x;
  x.row[0] = a.x + (int64_t)(a.sorted[g.first + min(r, g.count - 1)] / a.top) * a.ldx;   // (a missing slot: the last)
  f32x4 acc[2][1];
  acc[0][0] = acc[1][0] = f32x4{0.f, 0.f, 0.f, 0.f};
  rows_product<BF, 2, 1, WV, AL, NX, 3>(w, shift, a.cols, wave, x, acc);
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][q][(4 * p + e) * 16 + r] = acc[q][0][e];
  __syncthreads();
  for (int o = threadIdx.x; o < 256; o += WV * kWave) {
    const int64_t unit = row0 + ((int64_t)(o & 15) << a.apart_bits);
    const bool in = (o >> 4) < g.count && unit < a.rows;
    const int slot = a.sorted[g.first + min(o >> 4, g.count - 1)];
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int k = 0; k < WV; ++k) v[q] += red[k][q][o];
    const float h = act_value(a.act, v[0]) * v[1];
    if (in) a.h[slot * a.ldh + unit] = h;
    if constexpr (!BF) {
      float size = in && __builtin_isfinite(h) ? fabsf(h) : 0.f;
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) size = fmaxf(size, __shfl_xor(size, k, 16));
      if (in && (o & 15) == 0) atomicMax(a.tops + slot, __float_as_uint(size));
    }
  }
}

struct DownArgs {
  const float* h;
  const uint16_t* w;
  int64_t cols, rows, ldh, ldw, stride;   // rows: of each expert's matrix, the layer's outputs
  int apart_bits;
  const int32_t* groups_n;
  const MoeGroup* groups;
  const int32_t* sorted;
  const uint32_t* tops;
  float* part;
};

template <bool BF, int WV, bool AL>
__global__ __launch_bounds__(WV * kWave) void k_moe_down(DownArgs a) {
  __shared__ float red[WV][256];
  if ((int)blockIdx.y >= *a.groups_n) return;
  const MoeGroup g = a.groups[blockIdx.y];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int r = lane & 15, p = lane >> 4;
  const int64_t row0 = tile_row0(blockIdx.x, a.apart_bits);
  if (row0 >= a.rows) return;
  const int64_t mine = row0 + ((int64_t)r << a.apart_bits);
  const uint16_t* const base = a.w + g.expert * a.stride;
  const uint16_t* const w[1] = {base + (mine < a.rows ? mine : row0) * a.ldw};
  const int shift[1] = {AL ? 0 : shift_of(base + row0 * a.ldw)};
  const int slot = a.sorted[g.first + min(r, g.count - 1)];
  Rows32<BF, 1> x;
  x.row[0] = a.h + slot * a.ldh;
  x.scale[0] = BF ? 1.f : scale_of(a.tops[slot]);
  f32x4 acc[1][1];
  acc[0][0] = f32x4{0.f, 0.f, 0.f, 0.f};
  rows_product<BF, 1, 1, WV, AL, 1, 4>(w, shift, a.cols, wave, x, acc);
#pragma unroll
  for (int e = 0; e < 4; ++e) red[wave][(4 * p + e) * 16 + r] = acc[0][0][e];
  __syncthreads();
  for (int o = threadIdx.x; o < 256; o += WV * kWave) {
    const int64_t row = row0 + ((int64_t)(o & 15) << a.apart_bits);
    if ((o >> 4) >= g.count || row >= a.rows) continue;
    const int64_t to = a.sorted[g.first + (o >> 4)];
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < WV; ++k) v += red[k][o];
    a.part[to * a.rows + row] = BF ? v : v * unscale_of(a.tops[to]);
  }
}

// y[t] = the sum over t's choices of weight * part, in the order of the choices; a choice outside the experts
// adds nothing.
template <bool BF>
__global__ __launch_bounds__(256) void k_moe_join(const float* __restrict__ part, const int32_t* __restrict__ ids,
                                                   const float* __restrict__ weights, int64_t tokens, int64_t cols, int top,
                                                   int experts, uint16_t* __restrict__ y) {
  const int64_t count = tokens * cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / cols, c = i - t * cols;
    float v = 0.f;
    for (int j = 0; j < top; ++j) {
      const int64_t slot = t * top + j;
      const int e = ids[slot];
      if (e >= 0 && e < experts) v = fmaf(weights[slot], part[slot * cols + c], v);
    }
    y[i] = (uint16_t)f32_to_16<BF>(v);
  }
}

bool pieces_aligned(const void* p, int64_t stride, int64_t ld, int64_t cols) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0 && ld % 8 == 0 && cols % 8 == 0;
}

template <bool BF>
hipError_t experts(const MoeArgs& a, const MoeSpace& s, hipStream_t stream) {
  const externd_moe_weights& w = a.w;
  const unsigned groups = (unsigned)moe_most_groups(a.slots(), w.experts);
  UpArgs u = {};
  u.x = static_cast<const uint16_t*>(a.x);
  u.w[0] = static_cast<const uint16_t*>(w.wg);
  u.w[1] = static_cast<const uint16_t*>(w.wu);
  u.cols = a.cols;
  u.rows = w.rows;
  u.ldx = a.ldx;
  u.ldw = w.up_ld;
  u.stride = w.up_stride;
  u.top = a.top;
  u.apart_bits = rows_apart_bits(w.up_ld);
  u.act = a.act;
  u.groups_n = s.groups_n;
  u.groups = s.groups;
  u.sorted = s.sorted;
  u.tops = s.tops;
  u.h = s.h;
  u.ldh = s.ldh;
  constexpr int WV = 8;
  const dim3 block(WV * kWave), up((unsigned)rows_tiles(w.rows, u.apart_bits), groups);
  const bool al = pieces_aligned(w.wg, w.up_stride, w.up_ld, a.cols) && pieces_aligned(w.wu, w.up_stride, w.up_ld, a.cols) &&
                  pieces_aligned(a.x, 0, a.ldx, a.cols);
  const bool alike = ((reinterpret_cast<uintptr_t>(w.wg) ^ reinterpret_cast<uintptr_t>(w.wu)) & 15) == 0;
  if (al) hipLaunchKernelGGL((k_moe_up<BF, WV, true, 1>), up, block, 0, stream, u);
  else if (alike) hipLaunchKernelGGL((k_moe_up<BF, WV, false, 1>), up, block, 0, stream, u);
  else hipLaunchKernelGGL((k_moe_up<BF, WV, false, 2>), up, block, 0, stream, u);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  DownArgs d = {};
  d.h = s.h;
  d.w = static_cast<const uint16_t*>(w.wd);
  d.cols = w.rows;
  d.rows = a.cols;
  d.ldh = s.ldh;
  d.ldw = w.down_ld;
  d.stride = w.down_stride;
  d.apart_bits = rows_apart_bits(w.down_ld);
  d.groups_n = s.groups_n;
  d.groups = s.groups;
  d.sorted = s.sorted;
  d.tops = s.tops;
  d.part = s.part;
  const dim3 down((unsigned)rows_tiles(a.cols, d.apart_bits), groups);
  if (pieces_aligned(w.wd, w.down_stride, w.down_ld, w.rows)) hipLaunchKernelGGL((k_moe_down<BF, WV, true>), down, block, 0, stream, d);
  else hipLaunchKernelGGL((k_moe_down<BF, WV, false>), down, block, 0, stream, d);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t grid = std::min<int64_t>((a.tokens * a.cols + 255) / 256, 1 << 14);
  hipLaunchKernelGGL(k_moe_join<BF>, dim3((unsigned)grid), dim3(256), 0, stream, s.part, a.ids, a.weights, a.tokens, a.cols, a.top,
                     (int)w.experts, static_cast<uint16_t*>(a.y));
  return hipGetLastError();
}

}  // namespace

hipError_t run_moe_experts(const MoeArgs& a, const MoeSpace& s, hipStream_t stream) {
  return a.dtype == EXTERND_BF16 ? experts<true>(a, s, stream) : experts<false>(a, s, stream);
}

}  // namespace externd
