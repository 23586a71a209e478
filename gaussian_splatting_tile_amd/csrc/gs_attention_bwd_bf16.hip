// Cross attention, backward: bfloat16.
#include "gs_attention_bwd.h"

namespace gsi {
namespace attn {

hipError_t launch_bwd_bf16(const Args &a, int waves, hipStream_t s) { return launch_bwd_kind<gemm::kBF16, 1>(a, waves, s); }

}  // namespace attn
}  // namespace gsi
