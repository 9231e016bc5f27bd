// The gated block's products on bf16 operands.
#include "gated_gemm.hpp"

namespace externd {

hipError_t gated_product_bf16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                             hipStream_t s) {
  return any_product<true>(mode, g, plan, part, cus, s);
}

}  // namespace externd
