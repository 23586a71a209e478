// Cross attention, backward: fp32 as three bf16 limbs.
#include "gs_attention_bwd.h"

namespace gsi {
namespace attn {

hipError_t launch_bwd_f32(const Args &a, int waves, hipStream_t s) { return launch_bwd_kind<gemm::kBF16, 3>(a, waves, s); }

}  // namespace attn
}  // namespace gsi
