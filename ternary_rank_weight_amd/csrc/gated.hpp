// The products of the gated block: arguments shared by the passes (gated.hip)
// and the units that instantiate the kernels (one per operand type).
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
  // dx, whose a has dg's parts and then du's, and the same for both parts of dW.
  int segs;
  int64_t rest;
  int64_t inner;        // contraction length of one segment
  int64_t full;         // whole steps of one segment
  int64_t split_steps;  // whole steps per split; the last split also takes the partial steps
  int64_t mt, nt;       // tiles
  int64_t splits;
  uint16_t* out[2];     // forward: h; dx: dx; dw: dWg, dWu
  int64_t mo, ldo;      // rows and columns of the outputs
  float* save[2];       // forward: g, u (or null)
  float* part;          // SPLIT: where the splits' sums go, fp32 (split, output, mo, ldo)
  int act;
  // fp16 gradients: a's row m was scaled by scale_of(tops[m]), for dWu tops[tops_of_up + m]
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

}  // namespace externd
