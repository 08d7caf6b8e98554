// state_cache.cu -- recurrent states of waiting sequences, kept in 8 bits: written into the
// slots of a cache and read back.
//
// Row s of K float32 elements (one v of a head's state): step = max|s| / 127,
// code = the whole number nearest to s / step, and s' = code * step when it is read back.
// Whole numbers and not 8-bit floats: the elements of a row are of one size, where three
// bits of mantissa are off by up to 1/16 of each element, and 255 even steps by up to 1/254
// of the row's largest (0.6% rms for a row of 128 normal numbers).  The running state stays
// in float32: only what waits is rounded, once for each time that it is parked.
//
// Bound by reading and writing states: K/4 neighbouring lanes hold a row, each thread four
// vectors of four elements, 1 KB of a warp's neighbouring bytes apart, all in flight at once.

#include "gdn_internal.h"
#include "rows.cuh"

namespace gdn {
namespace {

using namespace rows;

constexpr int kVectors = 4;  // a thread's

// Nearest whole number to x / step, ties to even, exactly: the product by the inverse may
// be off by one where the quotient is next to the middle between two numbers, but the
// remainder x - q step is exact (a multiple of half of step's last bit, below step in size).
__device__ __forceinline__ int code_of(float x, float step, float inverse) {
    const float q = rintf(x * inverse), left = fmaf(-q, step, x), half = 0.5f * step;
    const float over = fabsf(left) - half;
    float c = q;
    if (over > 0.f || (over == 0.f && ((int)q & 1))) c += left > 0.f ? 1.f : -1.f;
    return (int)c;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// blockIdx.y: the sequence; `vectors`: of four elements, of one sequence's state.
template <int LANES>
__global__ void __launch_bounds__(kThreads)
state_store_kernel(int B, int64_t vectors, int64_t slots, const float* __restrict__ states,
                   const int32_t* __restrict__ slot_of, signed char* __restrict__ cache, float* __restrict__ scales) {
    await_previous();
    const int b = blockIdx.y;
    const int64_t slot = slot_of[b];
    if (slot < 0 || slot >= slots) return;
    // of sequences with one slot the last one is kept
    bool later = false;
    for (int j = b + 1 + threadIdx.x; j < B; j += kThreads) later |= slot_of[j] == slot;
    if (__syncthreads_or(later)) return;
    const float4* from = (const float4*)states + b * vectors;
    const int64_t v0 = (int64_t)blockIdx.x * (kThreads * kVectors) + threadIdx.x;
    float4 x[kVectors];
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
        const int64_t v = v0 + j * kThreads;
        x[j] = v < vectors ? __ldcs(from + v) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
        const int64_t v = v0 + j * kThreads;
        float m = max_nan(max_nan(fabsf(x[j].x), fabsf(x[j].y)), max_nan(fabsf(x[j].z), fabsf(x[j].w)));
#pragma unroll
        for (int off = LANES / 2; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        // no subnormal step, whose inverse would be infinite; a row that is not finite keeps
        // a step that is not, and is read back as NaN
        float step = m / 127.f;
        if (step < 1.17549435e-38f) step = 1.17549435e-38f;
        const float inverse = 1.f / step;
        if (v >= vectors) continue;
        uint32_t c = 0;
        if (step <= 3.402823466e38f) {
            c = (uint32_t)(code_of(x[j].x, step, inverse) & 255) | (uint32_t)(code_of(x[j].y, step, inverse) & 255) << 8 |
                (uint32_t)(code_of(x[j].z, step, inverse) & 255) << 16 | (uint32_t)code_of(x[j].w, step, inverse) << 24;
        } else {
            step = __int_as_float(0x7fc00000);
        }
        reinterpret_cast<uint32_t*>(cache)[slot * vectors + v] = c;
        if (threadIdx.x % LANES == 0) scales[(slot * vectors + v) / LANES] = step;
    }
}

template <int LANES>
__global__ void __launch_bounds__(kThreads)
state_load_kernel(int64_t vectors, int64_t slots, const signed char* __restrict__ cache,
                  const float* __restrict__ scales, const int32_t* __restrict__ slot_of, float* __restrict__ states) {
    await_previous();
    const int64_t b = blockIdx.y, slot = slot_of[b];
    const bool known = slot >= 0 && slot < slots;
    const int64_t v0 = (int64_t)blockIdx.x * (kThreads * kVectors) + threadIdx.x;
    uint32_t c[kVectors];
    float step[kVectors];
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
        const int64_t v = v0 + j * kThreads;
        const bool on = known && v < vectors;
        c[j] = on ? __ldg((const uint32_t*)cache + slot * vectors + v) : 0u;
        step[j] = on ? __ldg(scales + (slot * vectors + v) / LANES) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
        const int64_t v = v0 + j * kThreads;
        if (v >= vectors) break;
        const float4 x = make_float4((float)(signed char)(c[j] & 255) * step[j], (float)(signed char)(c[j] >> 8 & 255) * step[j],
                                     (float)(signed char)(c[j] >> 16 & 255) * step[j], (float)(signed char)(c[j] >> 24) * step[j]);
        __stcs((float4*)states + b * vectors + v, x);
    }
}

template <int LANES>
cudaError_t launch_k(const StateCall& c, bool load, cudaStream_t st) {
    const int64_t vectors = c.rows * LANES, per = kThreads * kVectors;
    const dim3 grid((unsigned)((vectors + per - 1) / per), (unsigned)c.B);
    if (load)
        return launch_dependent(state_load_kernel<LANES>, grid, kThreads, 0, st, vectors, c.slots,
                                (const signed char*)c.cache, (const float*)c.scales, c.slot_of, c.out);
    return launch_dependent(state_store_kernel<LANES>, grid, kThreads, 0, st, c.B, vectors, c.slots, c.states, c.slot_of,
                            (signed char*)c.cache, c.scales);
}

}  // namespace

cudaError_t launch_state_cache(const StateCall& c, bool load, cudaStream_t st) {
    switch (c.K) {
        case 16: return launch_k<4>(c, load, st);
        case 32: return launch_k<8>(c, load, st);
        case 64: return launch_k<16>(c, load, st);
        default: return launch_k<32>(c, load, st);
    }
}

}  // namespace gdn
