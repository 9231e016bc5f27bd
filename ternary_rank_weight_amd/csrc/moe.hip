// The experts of the mixture-of-experts layer, for a few tokens:
//   h = act(Wg_e x) (Wu_e x) for every slot (a token and one of its experts e),
//   y[t] = the sum over t's slots of weight * Wd_e h.
// Bound by the weights of the experts that are chosen, which are read once for each group of up to 16 of an expert's
// slots (rows_core.hpp).  h and each slot's result are fp32; h enters the second product in three 16-bit parts that are
// made where it is read and whose sum it is (fp16: multiplied by a power of two for each slot, to 2^-39 of the slot's
// largest), so y is rounded once.  (In two parts, which 17 bits of bf16 and 22 of fp16 fill, outputs that cancel were off;
// one token 21.9 us then, 23 now, 7 tokens 35 and 36, 32 tokens the same.)
// bf16, us of both products: one token through 4 of 64 experts of 1024 x 2560 11.8 + 9.0 (63 MB), 32 tokens through
// 8 of 128 of 768 x 2560 157 + 94 (4.9 and 4.2 TB/s); fp16, unaligned, 7 tokens, 3 of 13 of 701 x 1237 21 + 10.4.
#include <algorithm>

#include "activation.hpp"
#include "device_common.hpp"
#include "frag.hpp"
#include "gated.hpp"
#include "moe.hpp"
#include "moe_choose.hpp"
#include "rows_core.hpp"

namespace externd {

namespace {

struct UpArgs {
  const uint16_t *x, *w[2];
  int64_t cols, rows, ldx, ldw, stride;   // stride: from one expert to the next
  int top, apart_bits, act;
  MoeGroup* groups;
  uint32_t* tops;
  float* h;
  int64_t ldh;
  // few tokens, whose choices this kernel makes
  const double* logits;
  int tokens, experts, normalize;
  int32_t* ids;
  float* weights;
};

// A workgroup of WV waves takes WV / SW tiles of 16 hidden units, SW waves each, of one group of slots.
// FEW: every workgroup works out the choices of the few tokens there are, a wave each, and which slots its group
// has: the groups are the different experts in the order in which they first come.  The first workgroup of each
// group writes it down, and the very first the choices.  (Instead of a kernel before this one: 7 tokens, 3 of 13 experts
// of 701 x 1237, whole layer: 40.1 -> 38.7 us.)
template <bool BF, int WV, int SW, bool AL, int NX, bool FEW>
__global__ __launch_bounds__(WV * kWave, 4) void k_moe_up(UpArgs a) {
  static_assert(SW > 1, "a tile's waves join their sums");
  __shared__ float red[WV][2][256];
  __shared__ int few_ids[kMoeFewSlots], few_slots[kMoeGroup];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15, p = lane >> 4, group = blockIdx.y;
  int expert, count, slot;   // slot: the lane's (a missing one: the last)
  if constexpr (FEW) {
    if (wave < a.tokens) {
      int chosen;
      float weight;
      const bool write = blockIdx.x == 0 && group == 0;
      choose<4>(a.logits + wave * a.experts, a.experts, a.top, a.normalize, write, chosen, weight);
      if (lane < a.top) {
        few_ids[wave * a.top + lane] = chosen;
        if (write) {
          a.ids[wave * a.top + lane] = chosen;
          a.weights[wave * a.top + lane] = weight;
        }
      }
    }
    __syncthreads();
    const int slots = a.tokens * a.top, mine = lane < slots ? few_ids[lane] : -1;
    uint64_t left = __ballot(lane < slots), same = 0;
    expert = -1;
    for (int g = 0; g <= group && left; ++g) {
      expert = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
      same = __ballot(mine == expert);
      left &= ~same;
      if (g < group) same = 0;
    }
    if (!same) expert = -1;   // (fewer experts than groups)
    count = __builtin_popcountll(same);
    uint64_t mask = same;
    for (int k = min(r, count - 1); k > 0; --k) mask &= mask - 1;
    slot = mask ? __builtin_ctzll(mask) : 0;
    if (wave == 0 && lane < kMoeGroup) {
      few_slots[lane] = slot;
      if (blockIdx.x == 0) {
        a.groups[group].slot[lane] = slot;
        if (lane == 0) {
          a.groups[group].expert = expert;
          a.groups[group].count = count;
        }
      }
    }
    if (expert < 0) return;
  } else {
    const MoeGroup& g = a.groups[group];
    expert = g.expert;
    count = g.count;
    slot = g.slot[r];
    if (expert < 0) return;
  }
  const int64_t tile = (int64_t)blockIdx.x * (WV / SW) + wave / SW, row0 = tile_row0(tile, a.apart_bits);
  f32x4 acc[2][1];
  acc[0][0] = acc[1][0] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (row0 < a.rows) {
    const int64_t mine = row0 + ((int64_t)r << a.apart_bits), row = mine < a.rows ? mine : row0;   // (past the end: the first again)
    const uint16_t* const base[2] = {a.w[0] + expert * a.stride, a.w[1] + expert * a.stride};
    const uint16_t* const w[2] = {base[0] + row * a.ldw, base[1] + row * a.ldw};
    const int shift[2] = {AL ? 0 : shift_of(base[0] + row0 * a.ldw), AL ? 0 : shift_of(base[1] + row0 * a.ldw)};
    Rows16<1, AL> x;
    x.row[0] = a.x + (int64_t)(slot / a.top) * a.ldx;
    rows_product<BF, 2, 1, SW, AL, NX>(w, shift, (int)a.cols, wave % SW, x, acc);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][q][(4 * p + e) * 16 + r] = acc[q][0][e];
  __syncthreads();
  if (row0 >= a.rows) return;
  // v: both projections of slot s of the group (ss: its number), unit k of the tile
  auto put = [&](int s, int ss, int k, const float (&v)[2]) {
    const int64_t unit = row0 + ((int64_t)k << a.apart_bits);
    const bool in = s < count && unit < a.rows;
    const float h = act_value(a.act, v[0]) * v[1];
    if (in) a.h[ss * a.ldh + unit] = h;
    if constexpr (!BF) {
      float size = in && __builtin_isfinite(h) ? fabsf(h) : 0.f;
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) size = fmaxf(size, __shfl_xor(size, w, 16));
      if (s < count && k == 0) atomicMax(a.tops + ss, __float_as_uint(size));
    }
  };
  for (int o = wave % SW * kWave + lane; o < 256; o += SW * kWave) {
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int k = 0; k < SW; ++k) v[q] += red[wave / SW * SW + k][q][o];
    put(o >> 4, FEW ? few_slots[o >> 4] : a.groups[group].slot[o >> 4], o & 15, v);
  }
}

struct DownArgs {
  const float* h;
  const uint16_t* w;
  int64_t cols, rows, ldh, ldw, stride;   // rows: of each expert's matrix, the layer's outputs
  int apart_bits;
  const MoeGroup* groups;
  const uint32_t* tops;
  float* part;
};

// The lane's slot of h as the second product's vectors.
template <bool BF>
__device__ __forceinline__ RowsSplit<BF> hidden_of(const DownArgs& a, int slot) {
  return {a.h + slot * a.ldh, BF ? 1.f : scale_of(a.tops[slot])};
}

// As k_moe_up, for tiles of 16 outputs.  RT > 1 (and SW = 1): a wave takes that many tiles at once, whose rows start
// alike, so that h is read once for all of them.
template <bool BF, int WV, int SW, int RT, bool AL>
__global__ __launch_bounds__(WV * kWave, 4) void k_moe_down(DownArgs a) {
  static_assert(RT == 1 || SW == 1, "a wave's own tiles");
  __shared__ float red[SW > 1 ? WV : 1][256];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15, p = lane >> 4;
  const MoeGroup& g = a.groups[blockIdx.y];
  const int expert = g.expert, count = g.count, slot = g.slot[r];
  if (expert < 0) return;
  const int64_t at = (int64_t)blockIdx.x * (WV / SW) + wave / SW;
  // tiles 2^apart_bits apart
  const int64_t tile = ((at >> a.apart_bits) * RT << a.apart_bits) + (at & (((int64_t)1 << a.apart_bits) - 1));
  int64_t row0[RT];
#pragma unroll
  for (int q = 0; q < RT; ++q) row0[q] = tile_row0(tile + ((int64_t)q << a.apart_bits), a.apart_bits);
  f32x4 acc[RT][1];
#pragma unroll
  for (int q = 0; q < RT; ++q) acc[q][0] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (row0[0] < a.rows) {
    const uint16_t* const base = a.w + expert * a.stride;
    const uint16_t* w[RT];
    int shift[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      const int64_t mine = row0[q] + ((int64_t)r << a.apart_bits);
      w[q] = base + (mine < a.rows ? mine : row0[0]) * a.ldw;   // (past the end: the first again)
      shift[q] = AL ? 0 : shift_of(base + row0[0] * a.ldw);
    }
    rows_product<BF, RT, 1, SW, AL, 1>(w, shift, (int)a.cols, wave % SW, hidden_of<BF>(a, slot), acc);
  }
  auto put = [&](int s, int64_t row, float v) {
    if (s >= count || row >= a.rows) return;
    const int64_t to = g.slot[s];
    a.part[to * a.rows + row] = BF ? v : v * unscale_of(a.tops[to]);
  };
  if constexpr (SW > 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][(4 * p + e) * 16 + r] = acc[0][0][e];
    __syncthreads();
    for (int o = wave % SW * kWave + lane; o < 256; o += SW * kWave) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < SW; ++k) v += red[wave / SW * SW + k][o];
      put(o >> 4, row0[0] + ((int64_t)(o & 15) << a.apart_bits), v);
    }
  } else {
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) put(4 * p + e, row0[q] + ((int64_t)r << a.apart_bits), acc[q][0][e]);
  }
}

// One token's outputs: a workgroup of sixteen waves takes a tile of all its experts, SL waves each (with more than sixteen
// experts, a wave several), and writes y: no results of slots, no join.  One token through 4 of 64 experts of 1024 x
// 2560, h in two parts: 7.1 us against 6.6 + 2.4 for the second product and the join; layer 28 -> 22 us.
template <bool BF, int SL, bool AL>
__global__ __launch_bounds__(16 * kWave) void k_moe_down_one(DownArgs a, const int32_t* __restrict__ ids,
                                                              const float* __restrict__ weights, int top, int experts,
                                                              uint16_t* __restrict__ y) {
  __shared__ float red[16][16];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15;
  const int64_t row0 = tile_row0(blockIdx.x, a.apart_bits);
  if (row0 >= a.rows) return;
  const int64_t mine = row0 + ((int64_t)r << a.apart_bits), row = mine < a.rows ? mine : row0;   // (past the end: the first again)
  float sum = 0.f;
  for (int slot = wave / SL; slot < top; slot += 16 / SL) {
    const int expert = ids[slot];
    if (expert < 0 || expert >= experts) continue;
    const uint16_t* const base = a.w + expert * a.stride;
    const uint16_t* const w[1] = {base + row * a.ldw};
    const int shift[1] = {AL ? 0 : shift_of(base + row0 * a.ldw)};
    f32x4 acc[1][1];
    acc[0][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    rows_product<BF, 1, 1, SL, AL, 1>(w, shift, (int)a.cols, wave % SL, hidden_of<BF>(a, slot), acc);
    const float v = BF ? acc[0][0][0] : acc[0][0][0] * unscale_of(a.tops[slot]);   // (every row of the product is the token)
    sum = fmaf(weights[slot], v, sum);
  }
  if (lane < 16) red[wave][lane] = sum;
  __syncthreads();
  if (threadIdx.x < 16 && mine < a.rows) {
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) v += red[q][threadIdx.x];
    y[mine] = (uint16_t)f32_to_16<BF>(v);
  }
}

// y[t] = the sum over t's choices of weight * part, in the order of the choices; a choice outside the experts
// adds nothing.  (Done instead by the workgroup of the second product that comes last to a column of outputs, it cost
// more than this pass: each has to wait for its stores and for the count, 150 us against 108 and 7 for 32 tokens, 8 of 128
// experts of 768 x 2560.)
template <bool BF>
__global__ __launch_bounds__(256) void k_moe_join(const float* __restrict__ part, const int32_t* __restrict__ ids,
                                                   const float* __restrict__ weights, int64_t cols, int top, int experts,
                                                   uint16_t* __restrict__ y) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (c >= cols) return;
  float v = 0.f;
#pragma unroll 8
  for (int j = 0; j < top; ++j) {
    const int64_t slot = t * top + j;
    const int e = ids[slot];
    if (e >= 0 && e < experts) v = fmaf(weights[slot], part[slot * cols + c], v);
  }
  y[t * cols + c] = (uint16_t)f32_to_16<BF>(v);
}

bool pieces_aligned(const void* p, int64_t stride, int64_t ld, int64_t cols) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0 && ld % 8 == 0 && cols % 8 == 0;
}

template <bool BF, int SW, bool FEW>
void launch_up(const UpArgs& u, bool al, bool alike, unsigned groups, hipStream_t s) {
  constexpr int WV = SW > 8 ? SW : 8;
  const int64_t tiles = rows_tiles(u.rows, u.apart_bits);
  const dim3 grid((unsigned)((tiles + WV / SW - 1) / (WV / SW)), groups), block(WV * kWave);
  if (al) hipLaunchKernelGGL((k_moe_up<BF, WV, SW, true, 1, FEW>), grid, block, 0, s, u);
  else if (alike) hipLaunchKernelGGL((k_moe_up<BF, WV, SW, false, 1, FEW>), grid, block, 0, s, u);
  else hipLaunchKernelGGL((k_moe_up<BF, WV, SW, false, 2, FEW>), grid, block, 0, s, u);
}

template <bool BF, int SW, int RT>
void launch_down(const DownArgs& d, bool al, unsigned groups, hipStream_t s) {
  constexpr int WV = SW > 8 ? SW : 8;
  const int64_t row_groups = (d.rows + ((int64_t)16 << d.apart_bits) - 1) / ((int64_t)16 << d.apart_bits);
  const int64_t units = (row_groups + RT - 1) / RT << d.apart_bits;   // of RT tiles
  const dim3 grid((unsigned)((units + WV / SW - 1) / (WV / SW)), groups), block(WV * kWave);
  if (al) hipLaunchKernelGGL((k_moe_down<BF, WV, SW, RT, true>), grid, block, 0, s, d);
  else hipLaunchKernelGGL((k_moe_down<BF, WV, SW, RT, false>), grid, block, 0, s, d);
}

template <bool BF, int SL>
void launch_one(const DownArgs& d, bool al, const MoeArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)rows_tiles(d.rows, d.apart_bits)), block(16 * kWave);
  uint16_t* const y = static_cast<uint16_t*>(a.y);
  const int experts = (int)a.w.experts;
  if (al) hipLaunchKernelGGL((k_moe_down_one<BF, SL, true>), grid, block, 0, s, d, a.ids, a.weights, a.top, experts, y);
  else hipLaunchKernelGGL((k_moe_down_one<BF, SL, false>), grid, block, 0, s, d, a.ids, a.weights, a.top, experts, y);
}

template <bool BF>
hipError_t experts(const MoeArgs& a, const MoeSpace& s, bool few, hipStream_t stream) {
  const externd_moe_weights& w = a.w;
  const int64_t groups = moe_most_groups(a.slots(), w.experts);
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
  u.groups = s.groups;
  u.tops = s.tops;
  u.h = s.h;
  u.ldh = s.ldh;
  u.logits = s.logits;
  u.tokens = (int)a.tokens;
  u.experts = (int)w.experts;
  u.normalize = a.normalize;
  u.ids = a.ids_out;
  u.weights = a.weights_out;
  const bool al = pieces_aligned(w.wg, w.up_stride, w.up_ld, a.cols) && pieces_aligned(w.wu, w.up_stride, w.up_ld, a.cols) &&
                  pieces_aligned(a.x, 0, a.ldx, a.cols);
  const bool alike = ((reinterpret_cast<uintptr_t>(w.wg) ^ reinterpret_cast<uintptr_t>(w.wu)) & 15) == 0;
  const MoeForms f = moe_forms(a.tokens, a.top, w.experts, w.rows, a.cols, w.up_ld, w.down_ld, a.cus);
  if (few) {
    if (f.up == 4) launch_up<BF, 4, true>(u, al, alike, (unsigned)groups, stream);
    else if (f.up == 8) launch_up<BF, 8, true>(u, al, alike, (unsigned)groups, stream);
    else launch_up<BF, 16, true>(u, al, alike, (unsigned)groups, stream);
  } else {
    if (f.up == 4) launch_up<BF, 4, false>(u, al, alike, (unsigned)groups, stream);
    else if (f.up == 8) launch_up<BF, 8, false>(u, al, alike, (unsigned)groups, stream);
    else launch_up<BF, 16, false>(u, al, alike, (unsigned)groups, stream);
  }
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
  d.groups = s.groups;
  d.tops = s.tops;
  d.part = s.part;
  const bool dal = pieces_aligned(w.wd, w.down_stride, w.down_ld, w.rows);
  if (a.tokens == 1) {
    if (f.one == 16) launch_one<BF, 16>(d, dal, a, stream);
    else if (f.one == 8) launch_one<BF, 8>(d, dal, a, stream);
    else if (f.one == 4) launch_one<BF, 4>(d, dal, a, stream);
    else if (f.one == 2) launch_one<BF, 2>(d, dal, a, stream);
    else launch_one<BF, 1>(d, dal, a, stream);
    return hipGetLastError();
  }
  if (f.down_tiles == 2) launch_down<BF, 1, 2>(d, dal, (unsigned)groups, stream);
  else if (f.down == 1) launch_down<BF, 1, 1>(d, dal, (unsigned)groups, stream);
  else if (f.down == 2) launch_down<BF, 2, 1>(d, dal, (unsigned)groups, stream);
  else if (f.down == 4) launch_down<BF, 4, 1>(d, dal, (unsigned)groups, stream);
  else if (f.down == 8) launch_down<BF, 8, 1>(d, dal, (unsigned)groups, stream);
  else launch_down<BF, 16, 1>(d, dal, (unsigned)groups, stream);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(k_moe_join<BF>, dim3((unsigned)((a.cols + 255) / 256), (unsigned)a.tokens), dim3(256), 0, stream, s.part, a.ids,
                     a.weights, a.cols, a.top, (int)w.experts, static_cast<uint16_t*>(a.y));
  return hipGetLastError();
}

}  // namespace

hipError_t run_moe_experts(const MoeArgs& a, const MoeSpace& s, bool few, hipStream_t stream) {
  return a.dtype == EXTERND_BF16 ? experts<true>(a, s, few, stream) : experts<false>(a, s, few, stream);
}

}  // namespace externd
