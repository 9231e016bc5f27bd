// The linear layer's products on bf16 operands.
#include "gated_gemm.hpp"

namespace externd {

hipError_t linear_product_bf16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                              hipStream_t s) {
  return any_linear<true>(mode, g, plan, part, cus, s);
}

}  // namespace externd
