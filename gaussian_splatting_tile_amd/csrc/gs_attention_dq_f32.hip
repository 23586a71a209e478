// Cross attention, backward for the queries: fp32 as three bf16 limbs.
#include "gs_attention_bwd.h"

namespace gsi {
namespace attn {

hipError_t launch_dq_f32(const Args &a, int waves, hipStream_t s) { return launch_dq_kind<gemm::kBF16, 3>(a, waves, s); }

}  // namespace attn
}  // namespace gsi
