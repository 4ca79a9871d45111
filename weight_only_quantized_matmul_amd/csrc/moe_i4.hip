// The expert layer's products with int4 weights.
#include "moe_products.h"

namespace wq {

hipError_t launch_moe_i4(MoeArgs &a, hipStream_t st) { return launch_both<WQ_I4>(a, st); }

} // namespace wq
