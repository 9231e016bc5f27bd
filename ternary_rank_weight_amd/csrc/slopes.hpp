// What enters the gradients' products of the gated block and of the linear layer: dg and du (or dg alone) in
// two 16-bit parts, and fp16's scales.
#pragma once
#include <type_traits>

#include "activation.hpp"
#include "device_common.hpp"
#include "frag.hpp"
#include "gated.hpp"

namespace externd {

namespace {

struct SlopeArgs {
  const float *g, *u;    // tokens x hidden; u: of the gated block
  const uint16_t* dh;    // rows lddh apart
  int64_t tokens, hidden, lddh;
};

// dg and du of token t, hidden units c .. c + 7 (0 past the hidden width).  ONCE: g and u are
// not read again soon.  Not GATED: h = act(g), and dg = dh act'(g) alone.
template <bool BF, int ACT, bool ONCE, bool GATED = true>
__device__ __forceinline__ void slopes_at(const SlopeArgs& a, int64_t t, int64_t c, float (&vg)[8], float (&vu)[8]) {
  typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
  const int64_t at = t * a.hidden + c, left = a.hidden - c;
  const uint16_t* q = a.dh + t * a.lddh + c;
  float gv[8], uv[8];
  u32x4 d;
  if (left >= 8) {
    d = (reinterpret_cast<uintptr_t>(q) & 15) == 0 ? load8<true>(q) : load8<false>(q);
    auto take = [](const float* p) {
      if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const f32x4_a4*>(p));
      else return *reinterpret_cast<const f32x4_a4*>(p);
    };
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const f32x4 x = take(a.g + at + e), y = GATED ? take(a.u + at + e) : f32x4{1.f, 1.f, 1.f, 1.f};
#pragma unroll
      for (int f = 0; f < 4; ++f) { gv[e + f] = x[f]; uv[e + f] = y[f]; }
    }
  } else {
    // (dg and du are 0 past the end: dh is)
    const int last = (int)max<int64_t>(left, 1) - 1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      gv[e] = left > 0 ? a.g[at + min(e, last)] : 0.f;
      uv[e] = !GATED ? 1.f : left > 0 ? a.u[at + min(e, last)] : 0.f;
    }
    d = load8_part(q, left);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e >= left) gv[e] = uv[e] = 0.f;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float v, slope;
    act_both_fast<ACT>(gv[e], v, slope);
    const float dv = f32_from_16<BF>((d[e / 2] >> (16 * (e & 1))) & 0xffffu);
    vg[e] = GATED ? dv * uv[e] * slope : dv * slope;
    vu[e] = dv * v;
  }
}

// fp16 has neither the range of dg and du (a finite gradient can come from a dg past 65504)
// nor that of small ones.  So each is multiplied by a power of two before it is rounded,
// which the products take back on their fp32 sums: the row of an output has a power of its own,
// from the largest finite dg or du that enters it (by token for dx, by hidden unit for
// each weight gradient), and no token or unit loses bits to another.  (bf16 has
// fp32's range and needs none of this.)  These are the largest magnitudes, as the bits of
// fp32: by token (of both dg and du), by hidden unit of dg and ldd entries on of du; zero before.
// One block: `strip` tokens x 256 hidden units, fewer where there would be few blocks (777 x 1001
// with 64: 52 blocks).  Bound by HBM: reads 4 + 4 + 2 bytes per unit and token; 41 us for
// 2048 x 9728, 7 us for 777 x 1001.
template <bool GATED = true>
__global__ __launch_bounds__(256) void k_gated_tops(SlopeArgs a, int64_t ldd, int act, int strip,
                                                     uint32_t* __restrict__ by_token, uint32_t* __restrict__ by_unit) {
  constexpr int UNITS = 256;
  __shared__ float col[2][8][UNITS];
  const int piece = threadIdx.x & 31, line = threadIdx.x >> 5;   // 8 units; every eighth token
  const int64_t strips = (a.hidden + UNITS - 1) / UNITS;
  const int64_t t0 = (int64_t)blockIdx.x / strips * strip, c0 = (int64_t)blockIdx.x % strips * UNITS, c = c0 + 8 * piece;
  float top_g[8], top_u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) top_g[e] = top_u[e] = 0.f;
  auto size = [](float v) { return __builtin_isfinite(v) ? fabsf(v) : 0.f; };
  with_act(act, [&](auto kind) {
    for (int64_t t = t0 + line; t < min(t0 + strip, a.tokens); t += 8) {
      float vg[8], vu[8], most = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) vg[e] = vu[e] = 0.f;
      if (c < a.hidden) slopes_at<false, decltype(kind)::value, false, GATED>(a, t, c, vg, vu);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        top_g[e] = fmaxf(top_g[e], size(vg[e]));
        top_u[e] = fmaxf(top_u[e], size(vu[e]));
        most = fmaxf(most, GATED ? fmaxf(size(vg[e]), size(vu[e])) : size(vg[e]));
      }
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) most = fmaxf(most, __shfl_xor(most, w, 32));
      if (piece == 0) atomicMax(by_token + t, __float_as_uint(most));
    }
  });
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    col[0][line][8 * piece + e] = top_g[e];
    col[1][line][8 * piece + e] = top_u[e];
  }
  __syncthreads();
  const int64_t unit = c0 + threadIdx.x;
  if (unit >= a.hidden) return;
#pragma unroll
  for (int q = 0; q < (GATED ? 2 : 1); ++q) {
    float most = 0.f;
#pragma unroll
    for (int l = 0; l < 8; ++l) most = fmaxf(most, col[q][l][threadIdx.x]);
    atomicMax(by_unit + q * ldd + unit, __float_as_uint(most));
  }
}

// dg and du in rows of ldd entries (a multiple of 8; zero past the hidden width), each
// in two parts of the operands' type: the rounded value, and `rest` entries further on
// what the rounding took away.  Bound by HBM: reads 4 + 4 + 2 bytes, writes
// 4 + 4 per hidden unit and token; 62 us for 2048 x 9728 (5.8 TB/s: part of what
// it writes stays in the last-level cache).  fp16: scaled by the power of two that
// k_gated_tops' bits give for the token, or for the hidden unit of dg and of du (the other null).  Not GATED: dg alone,
// in fp16 scaled by token into dg's place and by hidden unit into du's, each where its bits are given.
// This is one thread's part, `id` of `threads`.
template <bool BF, bool GATED>
__device__ __forceinline__ void put_slopes(const SlopeArgs& a, int64_t ldd, int act, int64_t rest, const uint32_t* __restrict__ by_token,
                                           const uint32_t* __restrict__ by_unit, uint16_t* __restrict__ dg, uint16_t* __restrict__ du,
                                           int64_t id, int64_t threads) {
  const int64_t per = ldd / 8, total = a.tokens * per;
  with_act(act, [&](auto kind) {
    for (int64_t i = id; i < total; i += threads) {
      const int64_t t = i / per, c = (i - t * per) * 8;
      float vg[8], vu[8];
      slopes_at<BF, decltype(kind)::value, BF, GATED>(a, t, c, vg, vu);
      if constexpr (!BF) {
        const float all = by_token ? scale_of(by_token[t]) : 0.f;
        u32x4 tg[2] = {}, tu[2] = {};
        if (GATED ? !by_token : by_unit != nullptr) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tg[h] = *reinterpret_cast<const u32x4*>(by_unit + c + 4 * h);
            if constexpr (GATED) tu[h] = *reinterpret_cast<const u32x4*>(by_unit + ldd + c + 4 * h);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if constexpr (!GATED) {
            vu[e] = vg[e] * scale_of(tg[e / 4][e & 3]);
            vg[e] *= all;
            continue;
          }
          vg[e] *= by_token ? all : scale_of(tg[e / 4][e & 3]);
          if constexpr (GATED) vu[e] *= by_token ? all : scale_of(tu[e / 4][e & 3]);
        }
      }
      u32x4 og, ou, rg, ru;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        uint32_t wg[2], wu[2], lg[2], lu[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          wg[f] = f32_to_16<BF>(vg[e + f]);
          wu[f] = f32_to_16<BF>(vu[e + f]);
          const float tg = vg[e + f] - f32_from_16<BF>(wg[f]), tu = vu[e + f] - f32_from_16<BF>(wu[f]);
          lg[f] = __builtin_isfinite(tg) ? f32_to_16<BF>(tg) : 0u;   // (infinite and NaN are in the first part)
          lu[f] = __builtin_isfinite(tu) ? f32_to_16<BF>(tu) : 0u;
        }
        og[e / 2] = wg[0] | (wg[1] << 16);
        ou[e / 2] = wu[0] | (wu[1] << 16);
        rg[e / 2] = lg[0] | (lg[1] << 16);
        ru[e / 2] = lu[0] | (lu[1] << 16);
      }
      const bool first = GATED || BF || by_token, second = GATED || (!BF && by_unit);
      if (first) *reinterpret_cast<u32x4*>(dg + t * ldd + c) = og;
      if (second) *reinterpret_cast<u32x4*>(du + t * ldd + c) = ou;
      if (first) *reinterpret_cast<u32x4*>(dg + rest + t * ldd + c) = rg;
      if (second) *reinterpret_cast<u32x4*>(du + rest + t * ldd + c) = ru;
    }
  });
}

template <bool BF>
__global__ __launch_bounds__(256) void k_gated_slopes(SlopeArgs a, int64_t ldd, int act, int64_t rest,
                                                       const uint32_t* __restrict__ by_token,
                                                       const uint32_t* __restrict__ by_unit,
                                                       uint16_t* __restrict__ dg, uint16_t* __restrict__ du) {
  put_slopes<BF, true>(a, ldd, act, rest, by_token, by_unit, dg, du, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

}  // namespace

}  // namespace externd
