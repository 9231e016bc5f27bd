// The 4-bit products on fp16 operands.
#include "q4_apply.hpp"

namespace externd {

hipError_t q4_product_f16(const Q4Args& a, int gpc, int mats, int out_type, hipStream_t s) {
  return pick_group<false>(a, gpc, mats, out_type, s);
}

}  // namespace externd
