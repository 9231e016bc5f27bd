// The products of the gated block: arguments shared by the planning (gated.hip)
// and the units that instantiate the kernels (one per operand type).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace externd {

enum GatedProduct { kFwd = 0, kDx = 1, kDw = 2 };
constexpr int kBK = 64;   // contraction entries per step: two 16x16x32 products, 128 bytes of a row

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

// How a product is run: 256 x 256 tiles, 128 x 128 tiles two to a CU, or one to a CU
// with loads three steps ahead; and the splits of its contraction.
enum GatedKind { kBig, kPair, kDeep };
struct GatedPlan {
  GatedKind kind;
  int64_t splits;
  int64_t stacked = 1;   // 2 (kDeep only): output rows are the sums of the first and the second half of a's
};

inline int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// One product and, when split, its join.  part: room for the splits' sums.
hipError_t gated_product_bf16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                              hipStream_t s);
hipError_t gated_product_f16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                             hipStream_t s);

}  // namespace externd
