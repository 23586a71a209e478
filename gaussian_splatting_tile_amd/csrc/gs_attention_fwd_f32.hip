// Cross attention, forward: fp32 as three bf16 limbs.
#include "gs_attention_fwd.h"

namespace gsi {
namespace attn {

hipError_t launch_fwd_f32(const Args &a, hipStream_t s) { return launch_fwd_kind<gemm::kBF16, 3>(a, s); }

}  // namespace attn
}  // namespace gsi
