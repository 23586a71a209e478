// The linear layer's products of fp32 operands: three bf16 limbs and six
// products (see gs_gemm.h), from limb planes or split while a tile goes from
// memory to LDS.
#include "gs_linear.h"

namespace gsi {

template <bool PT, bool QT>
static hipError_t launch_tiles(const gemm::Args &a, const LinearEpilogue::Args &e, const ProductPlan &plan, hipStream_t s)
{
    using E = LinearEpilogue;
    if (plan.staged && plan.tile == 1) return gemm::launch<gemm::kBF16, 3, 2, 32, 128, 128, 2, 4, PT, QT, true, false, E>(a, e, plan.splits, 1, s);
    if (plan.staged) return gemm::launch<gemm::kBF16, 3, 2, 32, 64, 64, 2, 2, PT, QT, true, false, E>(a, e, plan.splits, 1, s);
    if (plan.tile == 1) return gemm::launch<gemm::kBF16, 3, 3, 32, 128, 128, 2, 4, PT, QT, false, false, E>(a, e, plan.splits, 1, s);
    return gemm::launch<gemm::kBF16, 3, 3, 32, 64, 64, 2, 2, PT, QT, false, false, E>(a, e, plan.splits, 1, s);
}

hipError_t launch_product_f32(const gemm::Args &a, const LinearEpilogue::Args &e, const ProductPlan &plan, hipStream_t s)
{
    if (plan.pt && plan.qt) return launch_tiles<true, true>(a, e, plan, s);
    if (plan.pt) return launch_tiles<true, false>(a, e, plan, s);
    return launch_tiles<false, false>(a, e, plan, s);
}

}  // namespace gsi
