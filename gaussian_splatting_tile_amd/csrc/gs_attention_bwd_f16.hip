// Cross attention, backward: float16.
#include "gs_attention_bwd.h"

namespace gsi {
namespace attn {

hipError_t launch_bwd_f16(const Args &a, int waves, hipStream_t s) { return launch_bwd_kind<gemm::kF16, 1>(a, waves, s); }

}  // namespace attn
}  // namespace gsi
