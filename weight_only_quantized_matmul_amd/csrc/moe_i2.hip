// The expert layer's products with int2 weights.
#include "moe_products.h"

namespace wq {

hipError_t launch_moe_i2(MoeArgs &a, hipStream_t st) { return launch_both<WQ_I2>(a, st); }

} // namespace wq
