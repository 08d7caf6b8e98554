// rows.cuh -- what the row-wise kernels of the layer share: 16-byte pieces of a row
// as floats, sums over the lanes that hold a row, and the column sums of a weight's
// gradient.
//
// A row of D elements is held by a group of G neighbouring lanes (G a power of two,
// D <= G * 2 * VEC), each with two 16-byte pieces of VEC elements, one from each half of
// the row: neighbouring lanes have neighbouring pieces, so that a load fills whole
// 32-byte sectors (a lane's pieces side by side asked for every sector twice, 41 instead
// of 30 us for 150 MB), and the two pieces can be the two partners of a rotation.
//
// The kernels are bound by reading and writing the rows, so a block is persistent and
// keeps the rows of its next items in flight while it works on one: each thread copies
// its pieces asynchronously into a ring of slots of its own in shared memory, so its own
// wait orders everything and no barrier is needed.  Loads held in registers instead,
// all of an item's at once, reached half of the memory's rate.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "f32x2.cuh"

namespace gdn {
namespace rows {

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// One 16-byte piece as pairs of floats, and back (bf16 rounds to nearest even).
__device__ __forceinline__ void get(const uint4& x, uint64_t (&f)[2]) {
    f[0] = pair(__uint_as_float(x.x), __uint_as_float(x.y));
    f[1] = pair(__uint_as_float(x.z), __uint_as_float(x.w));
}
__device__ __forceinline__ void get(const uint4& x, uint64_t (&f)[4]) {
    f[0] = bf16_pair(x.x), f[1] = bf16_pair(x.y), f[2] = bf16_pair(x.z), f[3] = bf16_pair(x.w);
}
__device__ __forceinline__ uint4 put(const uint64_t (&f)[2]) {
    float a, b, c, d;
    unpair(f[0], a, b);
    unpair(f[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}
__device__ __forceinline__ uint32_t pack2(uint64_t p) {
    float lo, hi;
    unpair(p, lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 put(const uint64_t (&f)[4]) {
    return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}

// 1 / (1 + e^-z) by the PTX approximations ex2.approx.ftz (relative error about 2^-22)
// and rcp.approx.ftz (1 ulp), for float32 gates too: with the rounding of z log2(e), half an
// ulp of up to 128, the relative error is below 1e-6 for z >= -10 and grows to 5e-6 at
// z = -87, where the value is 1e-38; below that it is 0.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t z) {
    const float l = -1.4426950408889634f;
    float x, y;
    unpair(mul2(z, twice(l)), x, y);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(y));
    unpair(add2(pair(x, y), twice(1.f)), x, y);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(y));
    return pair(x, y);
}

constexpr int kThreads = 256;

// NP pieces of 16 bytes for each of S items and each thread of the block.
template <int NP, int S>
struct Ring {
    static constexpr int BYTES = NP * S * kThreads * 16;
    uint32_t base;
    __device__ __forceinline__ explicit Ring(void* sm)
        : base((uint32_t)__cvta_generic_to_shared(sm) + threadIdx.x * 16) {}
    __device__ __forceinline__ uint32_t at(int slot, int piece) const {
        return base + (uint32_t)((slot * NP + piece) * kThreads * 16);
    }
    // zeros where `on` is false (nothing is read then)
    __device__ __forceinline__ void copy(int slot, int piece, const void* src, bool on) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(slot, piece)), "l"(src), "r"(on ? 16 : 0)
                     : "memory");
    }
    // through L1, for what the block's other groups read too
    __device__ __forceinline__ void copy_shared(int slot, int piece, const void* src) const {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(at(slot, piece)), "l"(src) : "memory");
    }
    // 8 bytes at a time, to the piece's half `half`
    __device__ __forceinline__ void copy8(int slot, int piece, int half, const void* src) const {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at(slot, piece) + 8 * half), "l"(src) : "memory");
    }
    __device__ __forceinline__ void put(int slot, int piece, float x) const {
        asm volatile("st.shared.v4.f32 [%0], {%1, %1, %1, %1};" ::"r"(at(slot, piece)), "f"(x) : "memory");
    }
    __device__ __forceinline__ uint4 get(int slot, int piece) const {
        uint4 x;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(at(slot, piece))
                     : "memory");
        return x;
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // the oldest of S groups in flight has landed
    static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory"); }
    static __device__ __forceinline__ int after(int slot) { return slot + 1 == S ? 0 : slot + 1; }
    static __device__ __forceinline__ void wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
};

// An index split into (hi, lo) = (i / n, i % n), moved on by a fixed step without
// dividing again.
struct Walk {
    int64_t hi, step_hi;
    int lo, step_lo, n;
    __device__ __forceinline__ Walk(int64_t i, int64_t step, int n_)
        : hi(i / n_), step_hi(step / n_), lo((int)(i - hi * n_)), step_lo((int)(step - step_hi * n_)), n(n_) {}
    __device__ __forceinline__ void move() {
        hi += step_hi;
        lo += step_lo;
        if (lo >= n) lo -= n, ++hi;
    }
};

template <typename T>
__device__ __forceinline__ uint4 ldg16(const T* p) {
    return __ldg(reinterpret_cast<const uint4*>(p));
}
// Streaming store, for rows that are written once.
template <typename T>
__device__ __forceinline__ void sts16(T* p, const uint4& x) {
    __stcs(reinterpret_cast<uint4*>(p), x);
}
// Sum over aligned groups of G lanes.
template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// Blocks of a persistent kernel: all that fit on the GPU at once, or as many as there are
// items of kThreads / G groups each.
inline int64_t blocks_for(int64_t items, int lanes, int per_sm, int sms) {
    const int64_t per = kThreads / lanes, want = (items + per - 1) / per, cap = (int64_t)per_sm * sms;
    return want < cap ? want : cap;
}

// Lanes a row of D elements takes: the smallest power of two of 2 * VEC pieces each.
inline int lanes_for(int D, int vec) {
    int g = 1;
    while (g * 2 * vec < D) g *= 2;
    return g;
}

// Sum of one value per group over the block's groups, for every column of a row: acc
// holds this lane's 2 * VEC columns (from c0, then from c1 on) as pairs.  The warp's
// groups are added by shuffles, the warps through shared memory in a fixed order, so
// the same call gives the same bits.  Result: out[0 .. D-1], written by the block.
template <int G, int VEC>
__device__ __forceinline__ void block_columns(const uint64_t (&acc)[VEC], int c0, int c1, bool live, int D, float* sm,
                                              float* out) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        float f[2];
        unpair(acc[j], f[0], f[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int off = G; off < 32; off <<= 1) f[e] += __shfl_xor_sync(0xffffffffu, f[e], off);
            if (lane < G && live) sm[warp * D + (j < VEC / 2 ? c0 : c1 - VEC) + 2 * j + e] = f[e];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) s += sm[w * D + c];
        out[c] = s;
    }
    __syncthreads();
}

}  // namespace rows
}  // namespace gdn
