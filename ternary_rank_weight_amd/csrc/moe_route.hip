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
#include "moe_choose.hpp"
#include "q4.hpp"

namespace externd {

namespace {

constexpr int kTokens = 4, kSplit = 4;   // tokens of a workgroup of k_moe_logits; waves that share a row

// A workgroup takes one expert's row and four tokens; its waves take 512 entries of each in turn, and
// their sums are joined in wave order.  The first clears tops.  Latency: 4 us for one token of 64 experts at 2560, 8 for
// 32 of 128.
template <int DT, int WT>
__global__ __launch_bounds__(kSplit * kWave) void k_moe_logits(MoeArgs a, double* __restrict__ logits, uint32_t* __restrict__ tops) {
  __shared__ double red[kSplit][kTokens];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t expert = blockIdx.x, t0 = (int64_t)blockIdx.y * kTokens;
  if (tops && blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < a.tokens * a.top; i += kSplit * kWave) tops[i] = 0u;
  const int tokens = (int)min<int64_t>(kTokens, a.tokens - t0);
  double acc[kTokens] = {};
  for (int64_t c = (wave * kWave + lane) * 8; c < a.cols; c += kSplit * kWave * 8) {
    const int64_t left = a.cols - c;
    float w[8], x[kTokens][8];
    load_weights<WT>(a.wr, expert * a.ldr + c, left, w);
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
      if (t < tokens) load_weights<DT>(a.x, (t0 + t) * a.ldx + c, left, x[t]);
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
      if (t < tokens) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t] = fma((double)w[j], (double)x[t][j], acc[t]);
      }
  }
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
    const double v = wave_sum_to63(acc[t]);
    if (lane == kWave - 1) red[wave][t] = v;
  }
  __syncthreads();
  if (threadIdx.x < tokens) {
    double v = red[0][threadIdx.x];
#pragma unroll
    for (int q = 1; q < kSplit; ++q) v += red[q][threadIdx.x];
    logits[(t0 + threadIdx.x) * a.w.experts + expert] = v;
  }
}

constexpr int kMostGroups = kMoeExperts + EXTERND_MOE_SLOTS / kMoeGroup;

// Choice of every token (logits given), and the groups (given): one workgroup, since the groups need every token's choice
// (routing alone, which makes none, runs it too).  Bound by latency, a chain of reductions over a wave for each choice: 12 us for 32 tokens, 8 of 128.
template <int C>
__global__ __launch_bounds__(1024) void k_moe_choose(MoeArgs a, const double* __restrict__ logits, MoeGroup* __restrict__ groups,
                                                      int most, uint32_t* __restrict__ tops) {
  __shared__ int ids[EXTERND_MOE_SLOTS], sorted[EXTERND_MOE_SLOTS];
  __shared__ int count[kMoeExperts], at[kMoeExperts], sums[2][16];
  __shared__ int expert_of[kMostGroups], first_of[kMostGroups], count_of[kMostGroups];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int experts = (int)a.w.experts, slots = (int)(a.tokens * a.top);
  count[tid] = 0;
  if (logits) {
    for (int64_t t = wave; t < a.tokens; t += 16) {
      int chosen;
      float weight;
      choose<C>(logits + t * experts, experts, a.top, a.normalize, true, chosen, weight);
      if (lane < a.top) {
        ids[t * a.top + lane] = chosen;
        a.ids_out[t * a.top + lane] = chosen;
        a.weights_out[t * a.top + lane] = weight;
      }
    }
  } else {
    for (int i = tid; i < slots; i += 1024) {
      ids[i] = a.ids[i];
      tops[i] = 0u;
    }
  }
  if (!groups) return;
  __syncthreads();
  for (int i = tid; i < slots; i += 1024) {
    const int e = ids[i];
    if (e >= 0 && e < experts) atomicAdd(&count[e], 1);
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
  int total = 0;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    if (q < wave) { sn += sums[0][q]; sg += sums[1][q]; }
    total += sums[1][q];
  }
  at[tid] = sn - n;
  for (int q = 0; q < g; ++q) {
    expert_of[sg - g + q] = tid;
    first_of[sg - g + q] = sn - n + q * kMoeGroup;
    count_of[sg - g + q] = min(kMoeGroup, n - q * kMoeGroup);
  }
  __syncthreads();
  // (the order of an expert's slots does not matter: each has its own results)
  for (int i = tid; i < slots; i += 1024) {
    const int e = ids[i];
    if (e >= 0 && e < experts) sorted[atomicAdd(&at[e], 1)] = i;
  }
  __syncthreads();
  for (int i = tid; i < most * kMoeGroup; i += 1024) {
    const int q = i / kMoeGroup, k = i % kMoeGroup;
    if (q < total) groups[q].slot[k] = sorted[first_of[q] + min(k, count_of[q] - 1)];
    if (k == 0) {
      groups[q].expert = q < total ? expert_of[q] : -1;
      groups[q].count = q < total ? count_of[q] : 0;
    }
  }
}

template <int DT>
void launch_logits(const MoeArgs& a, const MoeSpace& s, hipStream_t stream) {
  const dim3 grid((unsigned)a.w.experts, (unsigned)((a.tokens + kTokens - 1) / kTokens)), block(kSplit * kWave);
  if (a.wr_dtype == EXTERND_F32) hipLaunchKernelGGL((k_moe_logits<DT, EXTERND_F32>), grid, block, 0, stream, a, s.logits, s.tops);
  else hipLaunchKernelGGL((k_moe_logits<DT, DT>), grid, block, 0, stream, a, s.logits, s.tops);
}

}  // namespace

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
    s.ldh = (rows + 7) / 8 * 8;
    s.groups = static_cast<MoeGroup*>(take(sizeof(MoeGroup) * (size_t)moe_most_groups(slots, experts)));
    s.tops = static_cast<uint32_t*>(take(4 * (size_t)slots));
    s.h = static_cast<float*>(take(4 * (size_t)(slots * s.ldh)));
    s.part = static_cast<float*>(take(4 * (size_t)(slots * cols)));
  }
  s.bytes = at;
  return s;
}

hipError_t run_moe_logits(const MoeArgs& a, const MoeSpace& s, hipStream_t stream) {
  if (a.dtype == EXTERND_BF16) launch_logits<EXTERND_BF16>(a, s, stream);
  else launch_logits<EXTERND_F16>(a, s, stream);
  return hipGetLastError();
}

hipError_t run_moe_choose(const MoeArgs& a, const MoeSpace& s, bool router, bool plan, hipStream_t stream) {
  const double* logits = router ? s.logits : nullptr;
  MoeGroup* groups = plan ? s.groups : nullptr;
  const int most = (int)moe_most_groups(a.slots(), a.w.experts);
  const int64_t e = router ? a.w.experts : 1;
  const dim3 grid(1), block(1024);
  if (e <= 64) hipLaunchKernelGGL(k_moe_choose<1>, grid, block, 0, stream, a, logits, groups, most, s.tops);
  else if (e <= 128) hipLaunchKernelGGL(k_moe_choose<2>, grid, block, 0, stream, a, logits, groups, most, s.tops);
  else if (e <= 256) hipLaunchKernelGGL(k_moe_choose<4>, grid, block, 0, stream, a, logits, groups, most, s.tops);
  else hipLaunchKernelGGL(k_moe_choose<16>, grid, block, 0, stream, a, logits, groups, most, s.tops);
  return hipGetLastError();
}

}  // namespace externd
