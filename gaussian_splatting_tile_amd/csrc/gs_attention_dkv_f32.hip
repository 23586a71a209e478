// Cross attention, backward for keys and values: fp32 as three bf16 limbs.
#include "gs_attention_bwd.h"

namespace gsi {
namespace attn {

hipError_t launch_dkv_f32(const Args &a, int waves, hipStream_t s) { return launch_dkv_kind<gemm::kBF16, 3>(a, waves, s); }

}  // namespace attn
}  // namespace gsi
