// The linear layer's products on fp16 operands.
#include "gated_gemm.hpp"

namespace externd {

hipError_t linear_product_f16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                              hipStream_t s) {
  return any_linear<false>(mode, g, plan, part, cus, s);
}
hipError_t linear_gradients_f16(const GatedGemm& dx, const GatedGemm& dw, int64_t first, int64_t rest, GatedKind kind, hipStream_t s) {
  return both_gradients<false>(dx, dw, first, rest, kind, s);
}

}  // namespace externd
