// Cross attention, forward: float16.
#include "gs_attention_fwd.h"

namespace gsi {
namespace attn {

hipError_t launch_fwd_f16(const Args &a, hipStream_t s) { return launch_fwd_kind<gemm::kF16, 1>(a, s); }

}  // namespace attn
}  // namespace gsi
