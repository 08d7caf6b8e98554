// norm_rope_axes.cu -- the q, k norm with the rotation by a position on each of several
// axes (norm_rope.cuh), where the pairs' axes allow whole copies or the angles are gathered.

#include "norm_rope.cuh"

namespace gdn {
namespace {

// Each token's cosines and sines [tokens][R / 2] from the rows of its pairs' axes, four pairs a
// thread; NaN where a position is outside the tables.  Bound by writing them, R / 2 * 8 bytes
// a token, which the kernel behind reads from L2 for every item of heads (B8 T4096, 6 + 6 heads of
// 128, bf16, the axes' pairs in turn: forward 49.2 -> 42.4 us, backward 79.5 -> 61.9).
__global__ void __launch_bounds__(kThreads)
rope_gather_kernel(int64_t tokens, int quads, int rows, Tables t, float* __restrict__ cos, float* __restrict__ sin) {
    await_previous();
    const int64_t n = tokens * quads, step = (int64_t)gridDim.x * kThreads;
    Walk at((int64_t)blockIdx.x * kThreads + threadIdx.x, step, quads);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += step, at.move()) {
        const int64_t tok = at.hi;
        float c[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int pair = 4 * at.lo + j, row = t.pos[axis_of(t.map, pair) * tokens + tok];
            const bool in = row >= 0 && row < rows;
            const int64_t e = (int64_t)row * (4 * quads) + pair;
            c[j] = in ? __ldg(t.cos + e) : __int_as_float(0x7fc00000);
            s[j] = in ? __ldg(t.sin + e) : __int_as_float(0x7fc00000);
        }
        reinterpret_cast<float4*>(cos)[i] = make_float4(c[0], c[1], c[2], c[3]);
        reinterpret_cast<float4*>(sin)[i] = make_float4(s[0], s[1], s[2], s[3]);
    }
}

// The call on gathered angles.
cudaError_t gather(RopeCall& c, cudaStream_t st) {
    const Tables t{c.cos, c.sin, c.pos, c.axes, c.map};
    float *cos = c.gathered, *sin = c.gathered + c.tokens * (c.R / 2);
    const int64_t want = (c.tokens * (c.R / 8) + kThreads - 1) / kThreads, cap = 8 * (int64_t)sm_count();
    cudaError_t e = launch_dependent(rope_gather_kernel, dim3((unsigned)(want < cap ? want : cap)), kThreads, 0, st, c.tokens,
                                     c.R / 8, c.rows, t, cos, sin);
    c.cos = cos, c.sin = sin, c.pos = nullptr, c.rows = (int)c.tokens;
    return e;
}

}  // namespace

// Whether the pairs of every unit of angles that a lane copies at once have one axis: four
// neighbouring pairs, or the two of interleaved float32.
bool rope_whole_units(const RopeCall& c, InType ty) {
    const int unit = c.interleaved && ty == InType::F32 ? 2 : 4;
    auto axis = [&](int i) { return c.map.w[i >> 5] >> (2 * (i & 31)) & 3; };
    for (int i = 0; i < c.R / 2; ++i)
        if (axis(i) != axis(i - i % unit)) return false;
    return true;
}

cudaError_t launch_qk_norm_rope_axes(const RopeCall& call, InType ty, bool bwd, cudaStream_t st) {
    RopeCall c = call;
    if (c.gathered) {
        cudaError_t e = gather(c, st);
        if (e != cudaSuccess) return e;
        return ty == InType::BF16 ? launch_t<__nv_bfloat16, 3>(c, bwd, st) : launch_t<float, 3>(c, bwd, st);
    }
    if (!rope_whole_units(c, ty)) return launch_qk_norm_rope_apart(c, ty, bwd, st);
    return ty == InType::BF16 ? launch_t<__nv_bfloat16, 1>(c, bwd, st) : launch_t<float, 1>(c, bwd, st);
}

}  // namespace gdn
