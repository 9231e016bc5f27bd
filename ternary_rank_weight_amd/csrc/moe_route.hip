// Routing of the mixture-of-experts layer: logits x Wr^T, the largest `top` of each token's, their weights,
// and the slots sorted by expert.
//
// The choice is a comparison, so logits are summed in 64 bits (products of 16-bit entries
// are exact there): it then depends neither on the order of the sums nor on how many tokens go
// together, but for logits that agree to 16 digits.
#include <algorithm>

#include "device_common.hpp"
#include "frag.hpp"
#include "moe.hpp"
#include "q4.hpp"

namespace externd {

namespace {

constexpr int kTokens = 4, kRouteWaves = 4;   // tokens and experts of a workgroup of k_moe_logits

// A wave takes one expert's row and four tokens, 512 entries of each at a time.
template <int DT, int WT>
__global__ __launch_bounds__(kRouteWaves * kWave) void k_moe_logits(MoeArgs a, double* __restrict__ logits) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t expert = (int64_t)blockIdx.x * kRouteWaves + wave, t0 = (int64_t)blockIdx.y * kTokens;
  if (expert >= a.w.experts) return;
  double acc[kTokens] = {};
  for (int64_t c = lane * 8; c < a.cols; c += kWave * 8) {
    const int64_t left = a.cols - c;
    float w[8], x[kTokens][8];
    load_weights<WT>(a.wr, expert * a.ldr + c, left, w);
#pragma unroll
    for (int t = 0; t < kTokens; ++t) load_weights<DT>(a.x, min(t0 + t, a.tokens - 1) * a.ldx + c, left, x[t]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int t = 0; t < kTokens; ++t) acc[t] = fma((double)w[j], (double)x[t][j], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
    const double v = wave_sum_to63(acc[t]);
    if (lane == kWave - 1 && t0 + t < a.tokens) logits[(t0 + t) * a.w.experts + expert] = v;
  }
}

// A double's order as that of unsigned numbers; NaN below all.
__device__ __forceinline__ uint64_t order_of(double v) {
  const int64_t b = __double_as_longlong(v);
  if (v != v) return 0ull;
  return b < 0 ? ~(uint64_t)b : (uint64_t)b | 0x8000000000000000ull;
}

// One token's choice by a wave: lane l holds the logits of experts l C .. l C + C - 1.
// Weights: exp(logit - the largest) over the sum of those of the chosen, or of all.
template <int C>
__device__ void choose(const double* __restrict__ logits, int experts, int top, bool normalize, int32_t* __restrict__ ids,
                       float* __restrict__ weights) {
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
  double largest = 0.0, sum = 0.0, mine = 0.0;   // mine: the value of this lane's choice
  int chosen = 0;
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
    const double e = exp(got - largest);
    if (normalize) sum += e;
    if (lane == j) { mine = e; chosen = expert; }
  }
  if (!normalize) {
    double part = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (lane * C + c < experts) part += exp(v[c] - largest);
    sum = lane63(wave_sum_to63(part));
  }
  if (lane < top) {
    ids[lane] = chosen;
    weights[lane] = (float)(mine / sum);
  }
}

struct PlanArgs {
  int32_t* groups_n;
  MoeGroup* groups;
  int32_t* sorted;
  uint32_t* tops;   // cleared
};

// Choice of every token (logits given), and the groups (p.groups given): one workgroup.
template <int C>
__global__ __launch_bounds__(1024) void k_moe_choose(MoeArgs a, const double* __restrict__ logits, PlanArgs p) {
  __shared__ int count[kMoeExperts], at[kMoeExperts], sums[2][16];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int experts = (int)a.w.experts, slots = (int)(a.tokens * a.top);
  count[tid] = 0;
  const int32_t* ids = a.ids;
  if (logits) {
    for (int64_t t = wave; t < a.tokens; t += 16)
      choose<C>(logits + t * experts, experts, a.top, a.normalize, a.ids_out + t * a.top, a.weights_out + t * a.top);
    ids = a.ids_out;
  }
  if (!p.groups) return;
  __syncthreads();   // (also orders the choice before it is read below)
  for (int i = tid; i < slots; i += 1024) {
    const int e = ids[i];
    if (e >= 0 && e < experts) atomicAdd(&count[e], 1);
    p.tops[i] = 0u;
  }
  __syncthreads();
  // where each expert's slots and groups begin
  const int n = count[tid], g = (n + kMoeGroup - 1) / kMoeGroup;
  int sn = n, sg = g;   // sums up to this expert
#pragma unroll
  for (int w = 1; w < kWave; w <<= 1) {
    const int un = __shfl_up(sn, w, kWave), ug = __shfl_up(sg, w, kWave);
    if (lane >= w) { sn += un; sg += ug; }
  }
  if (lane == kWave - 1) { sums[0][wave] = sn; sums[1][wave] = sg; }
  __syncthreads();
  for (int q = 0; q < wave; ++q) { sn += sums[0][q]; sg += sums[1][q]; }
  if (tid == 1023) *p.groups_n = sg;
  at[tid] = sn - n;
  for (int q = 0; q < g; ++q) p.groups[sg - g + q] = MoeGroup{tid, sn - n + q * kMoeGroup, min(kMoeGroup, n - q * kMoeGroup), 0};
  __syncthreads();
  // (the order of an expert's slots does not matter: each has its own results)
  for (int i = tid; i < slots; i += 1024) {
    const int e = ids[i];
    if (e >= 0 && e < experts) p.sorted[atomicAdd(&at[e], 1)] = i;
  }
}

hipError_t launch_choose(const MoeArgs& a, const double* logits, const PlanArgs& p, hipStream_t s) {
  const int64_t e = logits ? a.w.experts : 1;
  const dim3 grid(1), block(1024);
  if (e <= 64) hipLaunchKernelGGL(k_moe_choose<1>, grid, block, 0, s, a, logits, p);
  else if (e <= 128) hipLaunchKernelGGL(k_moe_choose<2>, grid, block, 0, s, a, logits, p);
  else if (e <= 256) hipLaunchKernelGGL(k_moe_choose<4>, grid, block, 0, s, a, logits, p);
  else hipLaunchKernelGGL(k_moe_choose<16>, grid, block, 0, s, a, logits, p);
  return hipGetLastError();
}

template <int DT>
void launch_logits(const MoeArgs& a, double* logits, hipStream_t s) {
  const dim3 grid((unsigned)((a.w.experts + kRouteWaves - 1) / kRouteWaves), (unsigned)((a.tokens + kTokens - 1) / kTokens)),
      block(kRouteWaves * kWave);
  if (a.wr_dtype == EXTERND_F32) hipLaunchKernelGGL((k_moe_logits<DT, EXTERND_F32>), grid, block, 0, s, a, logits);
  else hipLaunchKernelGGL((k_moe_logits<DT, DT>), grid, block, 0, s, a, logits);
}

}  // namespace

int64_t moe_most_groups(int64_t slots, int64_t experts) {
  return std::min(slots, std::min(slots, experts) + slots / kMoeGroup);
}

MoeSpace moe_space(void* base, int64_t tokens, int64_t experts, int64_t top, int64_t rows, int64_t cols, bool router, bool experts_too) {
  MoeSpace s = {};
  char* const begin = static_cast<char*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = begin + at;
    at += (bytes + 255) / 256 * 256;
    return static_cast<void*>(p);
  };
  const int64_t slots = tokens * top;
  if (router) s.logits = static_cast<double*>(take(8 * (size_t)(tokens * experts)));
  if (experts_too) {
    s.ldh = (rows + 3) / 4 * 4;
    s.groups_n = static_cast<int32_t*>(take(4));
    s.groups = static_cast<MoeGroup*>(take(sizeof(MoeGroup) * (size_t)moe_most_groups(slots, experts)));
    s.sorted = static_cast<int32_t*>(take(4 * (size_t)slots));
    s.tops = static_cast<uint32_t*>(take(4 * (size_t)slots));
    s.h = static_cast<float*>(take(4 * (size_t)(slots * s.ldh)));
    s.part = static_cast<float*>(take(4 * (size_t)(slots * cols)));
  }
  s.bytes = at;
  return s;
}

hipError_t run_moe_route(const MoeArgs& a, const MoeSpace& s, bool plan, hipStream_t stream) {
  if (a.dtype == EXTERND_BF16) launch_logits<EXTERND_BF16>(a, s.logits, stream);
  else launch_logits<EXTERND_F16>(a, s.logits, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_choose(a, s.logits, plan ? PlanArgs{s.groups_n, s.groups, s.sorted, s.tops} : PlanArgs{}, stream);
}

hipError_t run_moe_plan(const MoeArgs& a, const MoeSpace& s, hipStream_t stream) {
  return launch_choose(a, nullptr, PlanArgs{s.groups_n, s.groups, s.sorted, s.tops}, stream);
}

}  // namespace externd
