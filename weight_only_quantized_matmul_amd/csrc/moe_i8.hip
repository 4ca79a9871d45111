// The expert layer's products with int8 weights.
#include "moe_products.h"

namespace wq {

hipError_t launch_moe_i8(MoeArgs &a, hipStream_t st) { return launch_both<WQ_I8>(a, st); }

} // namespace wq
