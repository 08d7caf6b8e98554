// norm_rope.cu -- the q, k norm with the rotation by one position (norm_rope.cuh).

#include "norm_rope.cuh"

namespace gdn {

cudaError_t launch_qk_norm_rope(const RopeCall& c, InType ty, bool bwd, cudaStream_t st) {
    return ty == InType::BF16 ? launch_t<__nv_bfloat16, 0>(c, bwd, st) : launch_t<float, 0>(c, bwd, st);
}

}  // namespace gdn
