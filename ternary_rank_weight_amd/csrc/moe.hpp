// The mixture-of-experts layer for a few tokens: arguments and workspace shared by the C ABI, the
// routing (moe_route.hip) and the experts' products (moe.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/externd.h"
#include "moe_plan.hpp"

namespace externd {

constexpr int kMoeExperts = 1024;   // most experts: a thread each when the slots are sorted
constexpr int kMoeTop = 64;         // most experts of a token

// A slot is one of a token's choices: slot = token top + choice.  A group is up to 16 slots of one expert; slots
// past `count` repeat the last, and a group of expert -1 is not there.
struct MoeGroup {
  int expert, count, pad[2];
  int slot[kMoeGroup];
};

struct MoeArgs {
  const void *x, *wr;
  int64_t tokens, cols, ldx, ldr;   // ldr: rows of the router
  int wr_dtype, dtype, act, top, normalize;
  externd_moe_weights w;
  const int32_t* ids;               // the choice, and its weights: read by the experts
  const float* weights;
  int32_t* ids_out;                 // written by the router
  float* weights_out;
  void* y;
  int cus;
  int64_t slots() const { return tokens * top; }
};

// Where things lie in the workspace.
struct MoeSpace {
  double* logits;      // tokens x experts
  MoeGroup* groups;    // moe_most_groups of them
  uint32_t* tops;      // fp16: the largest magnitude of each slot's h, as bits of fp32; cleared by a call's first kernel
  float* h;            // slots x ldh
  float* part;         // slots x cols: what each slot's expert gives
  int64_t ldh;
  size_t bytes;
};
// experts_too: for the experts' products; without, for the router alone
MoeSpace moe_space(void* base, int64_t tokens, int64_t experts, int64_t top, int64_t rows, int64_t cols, bool router, bool experts_too);

hipError_t run_moe_logits(const MoeArgs& a, const MoeSpace& s, hipStream_t stream);
// Choice and weights from the logits, or a choice that was made elsewhere (router false); and, where plan is given, the groups.
hipError_t run_moe_choose(const MoeArgs& a, const MoeSpace& s, bool router, bool plan, hipStream_t stream);
// few: the choice is not made yet
hipError_t run_moe_experts(const MoeArgs& a, const MoeSpace& s, bool few, hipStream_t stream);

}  // namespace externd
