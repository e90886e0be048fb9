// The int8 product of mc2_linear_i8, rounded to either 16-bit type (gemm_linear.hpp).
#include "gemm_linear.hpp"

namespace mc2 {
namespace lin {
template hipError_t launch_product_i8<DT_BF16>(const Product&, int, const Plan&, hipStream_t);
template hipError_t launch_product_i8<DT_F16>(const Product&, int, const Plan&, hipStream_t);
}  // namespace lin
}  // namespace mc2
