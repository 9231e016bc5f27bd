// The linear layer's products on bf16 operands.
#include "gated_gemm.hpp"

namespace externd {

hipError_t linear_product_bf16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                              hipStream_t s) {
  return any_linear<true>(mode, g, plan, part, cus, s);
}
hipError_t linear_gradients_bf16(const GatedGemm& dx, const GatedGemm& dw, hipStream_t s) { return both_gradients<true>(dx, dw, s); }

}  // namespace externd
