// The choice of a token's experts, for the kernels that make it.
#pragma once
#include "device_common.hpp"

namespace externd {

namespace {

// A double's order as that of unsigned numbers; NaN below all.
__device__ __forceinline__ uint64_t order_of(double v) {
  const int64_t b = __double_as_longlong(v);
  if (v != v) return 0ull;
  return b < 0 ? ~(uint64_t)b : (uint64_t)b | 0x8000000000000000ull;
}

// One token's choices by a wave: lane l holds the logits of experts l C .. l C + C - 1.  Lane j < top has choice j in
// `chosen`, and in `weight` exp(logit - the largest) over the sum of those of the chosen (normalize), or of all (weighted; else 0).
template <int C>
__device__ void choose(const double* __restrict__ logits, int experts, int top, bool normalize, bool weighted, int& chosen, float& weight) {
  const int lane = threadIdx.x & (kWave - 1);
  double v[C];
  uint64_t key[C];   // 0 and taken: past the end, or chosen before
  bool taken[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = lane * C + c;
    taken[c] = e >= experts;
    v[c] = taken[c] ? 0.0 : logits[e];
    key[c] = order_of(v[c] + 0.0);   // (-0 is 0)
  }
  double largest = 0.0, mine = 0.0;   // mine: the logit of this lane's choice
  chosen = 0;
  for (int j = 0; j < top; ++j) {
    // the lane's largest, the first of equal ones; lanes without one are out
    int at = -1;
    uint64_t best = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (!taken[c] && (at < 0 || key[c] > best)) { at = c; best = key[c]; }
    const uint32_t hi = at < 0 ? 0u : (uint32_t)(best >> 32), lo = (uint32_t)best;
    const uint32_t top_hi = __builtin_amdgcn_readlane(wave_umax_to63(hi), 63);
    const bool in = at >= 0 && hi == top_hi;
    const uint32_t top_lo = __builtin_amdgcn_readlane(wave_umax_to63(in ? lo : 0u), 63);
    const int who = __builtin_ctzll(__ballot(in && lo == top_lo));
    double value = 0.0;
    int expert = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c == at) {
        value = v[c];
        expert = lane * C + c;
        if (lane == who) taken[c] = true;
      }
    const int64_t bits = __double_as_longlong(value);
    const double got = __longlong_as_double(((int64_t)__builtin_amdgcn_readlane((int)(bits >> 32), who) << 32) |
                                            (uint32_t)__builtin_amdgcn_readlane((int)bits, who));
    expert = __builtin_amdgcn_readlane(expert, who);
    if (j == 0) largest = got;
    if (lane == j) { mine = got; chosen = expert; }
  }
  weight = 0.f;
  if (!weighted) return;
  const double e = lane < top ? exp(mine - largest) : 0.0;
  double part = e;
  if (!normalize) {
    part = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (lane * C + c < experts) part += exp(v[c] - largest);
  }
  weight = (float)(e / lane63(wave_sum_to63(part)));
}

}  // namespace

}  // namespace externd
