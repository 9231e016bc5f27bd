// The products of the gated block and of the linear layer: arguments shared by the passes (gated.hip,
// linear.hip) and the units that instantiate the kernels (one per operand type).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gated_plan.hpp"

namespace externd {

// One operand of a product: `outer` output rows (or columns) by `inner`
// contraction entries.  Two sources: the forward's gate and up rows, dx's weights,
// dW's two outputs.
struct GatedOperand {
  const uint16_t* p[2];
  int64_t ld;
  int64_t outer;
};

struct GatedGemm {
  GatedOperand a, b;         // a: output rows, b: output columns
  // The contraction is `segs` segments of `inner` entries each.  Segment s of a lies
  // s * rest entries past its source; b's source is the second from segment segs / 2 on in
  // dx, whose a has dg's parts and then du's, and the same for both parts of dW.  (The linear layer's
  // dx has one weight matrix: both of b's sources.)
  int segs;
  int64_t rest;
  int64_t inner;        // contraction length of one segment
  int64_t full;         // whole steps of one segment
  int64_t split_steps;  // whole steps per split; the last split also takes the partial steps
  int64_t mt, nt;       // tiles
  int64_t splits;
  uint16_t* out[2];     // forward: h (linear: y); dx: dx; dw: dWg, dWu (linear: dW)
  int64_t mo, ldo;      // rows and columns of the outputs
  float* save[2];       // forward: g, u (linear: z) or null
  float* part;          // SPLIT: where the splits' sums go, fp32 (split, output, mo, ldo)
  int act;
  const uint16_t *bias, *residual;   // linear forward, or null
  int64_t ldr;          // entries from one row of the residual to the next
  // fp16 gradients: a's row m was scaled by scale_of(tops[m]), for dWu tops[tops_of_up + m]; null: not scaled
  const uint32_t* tops;
  int64_t tops_of_up;
};

// The power of two that brings a magnitude (its fp32 bits) to 2^14 .. 2^15, the largest
// that fp16 holds with room for a rounding, and the power that takes it back.  (Not past 2^100:
// what is that small leaves no gradient in fp16.)
__device__ __forceinline__ int scale_shift(uint32_t top) { return min(141 - (int)(top >> 23), 100); }
__device__ __forceinline__ float scale_of(uint32_t top) { return __uint_as_float((uint32_t)(127 + scale_shift(top)) << 23); }
__device__ __forceinline__ float unscale_of(uint32_t top) { return __uint_as_float((uint32_t)(127 - scale_shift(top)) << 23); }

// One product and, when split, its join.  part: room for the splits' sums.
hipError_t gated_product_bf16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                              hipStream_t s);
hipError_t gated_product_f16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                             hipStream_t s);
hipError_t linear_product_bf16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                               hipStream_t s);
hipError_t linear_product_f16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                              hipStream_t s);
// dx and dW together, in the numbers of workgroups and tiles that linear_join says.
hipError_t linear_gradients_bf16(const GatedGemm& dx, const GatedGemm& dw, int64_t first, int64_t rest, GatedKind kind, hipStream_t s);
hipError_t linear_gradients_f16(const GatedGemm& dx, const GatedGemm& dw, int64_t first, int64_t rest, GatedKind kind, hipStream_t s);

}  // namespace externd
