// norm_rope_apart.cu -- the q, k norm with the rotation by several positions, angle by angle
// (norm_rope.cuh).

#include "norm_rope.cuh"

namespace gdn {

cudaError_t launch_qk_norm_rope_apart(const RopeCall& c, InType ty, bool bwd, cudaStream_t st) {
    return ty == InType::BF16 ? launch_t<__nv_bfloat16, 2>(c, bwd, st) : launch_t<float, 2>(c, bwd, st);
}

}  // namespace gdn
