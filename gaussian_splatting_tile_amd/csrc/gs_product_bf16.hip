// The linear layer's products of bf16 operands.
#include "gs_product_16.h"

namespace gsi {

hipError_t launch_product_bf16(const gemm::Args &a, const LinearEpilogue::Args &e, const ProductPlan &plan, hipStream_t s)
{
    return launch_product_16<gemm::kBF16>(a, e, plan, s);
}

}  // namespace gsi
