// The linear layer's products of 16-bit operands, for one of the two types
// (included by gs_product_bf16.hip and gs_product_f16.hip).
#pragma once

#include "gs_linear.h"

namespace gsi {

template <int KIND, bool PT, bool QT>
hipError_t launch_product_16(const gemm::Args &a, const LinearEpilogue::Args &e, const ProductPlan &plan, hipStream_t s)
{
    using E = LinearEpilogue;
    if constexpr (!PT) {
        if (plan.staged && plan.tile == 1) return gemm::launch<KIND, 1, 2, 32, 128, 128, 2, 4, PT, QT, true, false, E>(a, e, plan.splits, 1, s);
        if (plan.staged) return gemm::launch<KIND, 1, 2, 32, 64, 64, 2, 2, PT, QT, true, false, E>(a, e, plan.splits, 1, s);
    }
    if (plan.tile == 0) return gemm::launch<KIND, 1, 2, 64, 256, 256, 2, 4, PT, QT, false, true, E>(a, e, plan.splits, 1, s);
    if (plan.tile == 1) {
        // a block alone on its CU wants a third stage on the way, two blocks
        // cover for each other: 4096 x 1024 x 16384 by 256 blocks takes 138 us
        // with three stages and 181 with two, by 512 blocks 135 with two
        const int64_t blocks = (int64_t)((a.P + 127) / 128) * ((a.Q + 127) / 128) * plan.splits;
        if (blocks <= 256) return gemm::launch<KIND, 1, 3, 64, 128, 128, 2, 4, PT, QT, false, false, E>(a, e, plan.splits, 1, s);
        return gemm::launch<KIND, 1, 2, 64, 128, 128, 2, 4, PT, QT, false, false, E>(a, e, plan.splits, 1, s);
    }
    return gemm::launch<KIND, 1, 3, 64, 64, 64, 2, 2, PT, QT, false, false, E>(a, e, plan.splits, 1, s);
}

template <int KIND>
hipError_t launch_product_16(const gemm::Args &a, const LinearEpilogue::Args &e, const ProductPlan &plan, hipStream_t s)
{
    if (plan.pt && plan.qt) return launch_product_16<KIND, true, true>(a, e, plan, s);
    if (plan.pt) return launch_product_16<KIND, true, false>(a, e, plan, s);
    return launch_product_16<KIND, false, false>(a, e, plan, s);
}

}  // namespace gsi
