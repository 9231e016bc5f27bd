// The linear layer's products on bf16 operands.
#include "gated_gemm.hpp"

namespace externd {

hipError_t linear_product_bf16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                              hipStream_t s) {
  return any_linear<true>(mode, g, plan, part, cus, s);
}
hipError_t linear_gradients_bf16(const GatedGemm& dx, const GatedGemm& dw, int64_t first, int64_t rest, GatedKind kind, hipStream_t s) {
  return both_gradients<true>(dx, dw, first, rest, kind, s);
}

}  // namespace externd
