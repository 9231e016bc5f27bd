// The gated block's products on fp16 operands.
#include "gated_gemm.hpp"

namespace externd {

hipError_t gated_product_f16(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                             hipStream_t s) {
  return any_product<false>(mode, g, plan, part, cus, s);
}

}  // namespace externd
