// Cross attention, forward: bfloat16.
#include "gs_attention_fwd.h"

namespace gsi {
namespace attn {

hipError_t launch_fwd_bf16(const Args &a, hipStream_t s) { return launch_fwd_kind<gemm::kBF16, 1>(a, s); }

}  // namespace attn
}  // namespace gsi
