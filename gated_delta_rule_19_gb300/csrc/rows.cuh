// rows.cuh -- what the row-wise kernels of the layer share: 16-byte pieces of a row
// as floats, sums over the lanes that hold a row, and the column sums of a weight's
// gradient.
//
// A row of D elements is held by a group of G neighbouring lanes (G a power of two,
// D <= G * 2 * VEC), each with two 16-byte pieces of VEC elements: 32 bytes a lane
// per load pair keep the loads full width at every D, and the two pieces can be the
// two partners of a rotation.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {
namespace rows {

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// One 16-byte piece as floats, and back (bf16 rounds to nearest even).
__device__ __forceinline__ void get(const uint4& x, float (&f)[4]) {
    f[0] = __uint_as_float(x.x), f[1] = __uint_as_float(x.y);
    f[2] = __uint_as_float(x.z), f[3] = __uint_as_float(x.w);
}
__device__ __forceinline__ void get(const uint4& x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 put(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
template <typename T>
__device__ __forceinline__ uint4 ldg16(const T* p) {
    return __ldg(reinterpret_cast<const uint4*>(p));
}
// Streaming forms, for rows that are read or written once.
template <typename T>
__device__ __forceinline__ uint4 lds16(const T* p) {
    return __ldcs(reinterpret_cast<const uint4*>(p));
}
template <typename T>
__device__ __forceinline__ void sts16(T* p, const uint4& x) {
    __stcs(reinterpret_cast<uint4*>(p), x);
}
// N floats (a multiple of four, 16-byte aligned).
template <int N>
__device__ __forceinline__ void ldf(const float* p, float (&f)[N]) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(p + j));
        f[j] = x.x, f[j + 1] = x.y, f[j + 2] = x.z, f[j + 3] = x.w;
    }
}

// Sum over aligned groups of G lanes.
template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// Lanes a row of D elements takes: the smallest power of two of 2 * VEC pieces each.
inline int lanes_for(int D, int vec) {
    int g = 1;
    while (g * 2 * vec < D) g *= 2;
    return g;
}

// Sum of one value per group over the block's groups, for every column of a row:
// acc holds this lane's 2 * VEC columns (columns c0.. and c1..).  The warp's groups
// are added by shuffles, the warps through shared memory in a fixed order, so the
// same call gives the same bits.  Result: out[0 .. D-1], written by the block.
template <int G, int VEC, int WARPS>
__device__ __forceinline__ void block_columns(float (&acc)[2 * VEC], int c0, int c1, bool live, int D, float* sm,
                                              float* out) {
#pragma unroll
    for (int j = 0; j < 2 * VEC; ++j)
#pragma unroll
        for (int off = G; off < 32; off <<= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], off);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane < G && live) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            sm[warp * D + c0 + j] = acc[j];
            sm[warp * D + c1 + j] = acc[VEC + j];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += WARPS * 32) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += sm[w * D + c];
        out[c] = s;
    }
    __syncthreads();
}

}  // namespace rows
}  // namespace gdn
