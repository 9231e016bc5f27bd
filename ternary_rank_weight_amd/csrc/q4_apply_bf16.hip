// The 4-bit products on bf16 operands (bf16 and fp32 x).
#include "q4_apply.hpp"

namespace externd {

hipError_t q4_product_bf16(const Q4Args& a, int gpc, int mats, int out_type, hipStream_t s) {
  return pick_group<true>(a, gpc, mats, out_type, s);
}

}  // namespace externd
