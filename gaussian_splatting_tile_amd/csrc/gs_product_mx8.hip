// The linear layer's products of 8-bit operands with a power-of-two scale per
// 32 values (scaled matrix instructions, 128 k each).
#include "gs_linear.h"

namespace gsi {

hipError_t launch_product_mx8(const gemm::Args &a, const LinearEpilogue::Args &e, const ProductPlan &plan, hipStream_t s)
{
    using E = LinearEpilogue;
    if (plan.tile == 0) return gemm::launch<gemm::kMX8, 1, 2, 64, 256, 256, 2, 4, false, false, false, false, E>(a, e, plan.splits, 1, s);
    if (plan.tile == 1) return gemm::launch<gemm::kMX8, 1, 2, 64, 128, 128, 2, 4, false, false, false, false, E>(a, e, plan.splits, 1, s);
    return gemm::launch<gemm::kMX8, 1, 3, 64, 64, 64, 2, 2, false, false, false, false, E>(a, e, plan.splits, 1, s);
}

}  // namespace gsi
