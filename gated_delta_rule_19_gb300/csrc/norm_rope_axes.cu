// norm_rope_axes.cu -- the q, k norm with the rotation by a position on each of several
// axes (norm_rope.cuh).

#include "norm_rope.cuh"

namespace gdn {

cudaError_t launch_qk_norm_rope_axes(const RopeCall& c, InType ty, bool bwd, cudaStream_t st) {
    return ty == InType::BF16 ? launch_t<__nv_bfloat16, true>(c, bwd, st) : launch_t<float, true>(c, bwd, st);
}

}  // namespace gdn
