// Cross attention, backward for the queries: float16.
#include "gs_attention_bwd.h"

namespace gsi {
namespace attn {

hipError_t launch_dq_f16(const Args &a, int waves, hipStream_t s) { return launch_dq_kind<gemm::kF16, 1>(a, waves, s); }

}  // namespace attn
}  // namespace gsi
