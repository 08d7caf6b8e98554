// norm_rope_axes.cu -- the q, k norm with the rotation by a position on each of several
// axes (norm_rope.cuh).

#include "norm_rope.cuh"

namespace gdn {
namespace {

// Whether the pairs of every unit of angles that a lane copies at once have one axis: four
// neighbouring pairs, or the two of interleaved float32.
bool whole_units(const RopeCall& c, InType ty) {
    const int unit = c.interleaved && ty == InType::F32 ? 2 : 4;
    auto axis = [&](int i) { return c.map.w[i >> 5] >> (2 * (i & 31)) & 3; };
    for (int i = 0; i < c.R / 2; ++i)
        if (axis(i) != axis(i - i % unit)) return false;
    return true;
}

template <typename T>
cudaError_t launch(const RopeCall& c, InType ty, bool bwd, cudaStream_t st) {
    return whole_units(c, ty) ? launch_t<T, 1>(c, bwd, st) : launch_t<T, 2>(c, bwd, st);
}

}  // namespace

cudaError_t launch_qk_norm_rope_axes(const RopeCall& c, InType ty, bool bwd, cudaStream_t st) {
    return ty == InType::BF16 ? launch<__nv_bfloat16>(c, ty, bwd, st) : launch<float>(c, ty, bwd, st);
}

}  // namespace gdn
