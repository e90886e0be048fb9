// The linear's tiled product for bf16 (gemm_linear.hpp).
#include "gemm_linear.hpp"

namespace mc2 {
namespace lin {
template hipError_t launch_product<DT_BF16>(const Product&, int, int, const Plan&, hipStream_t);
}  // namespace lin
}  // namespace mc2
