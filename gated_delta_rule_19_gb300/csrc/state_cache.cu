// state_cache.cu -- recurrent states of waiting sequences, kept in 8 bits: written into the
// slots of a cache and read back.
//
// Row s of K float32 elements (one v of a head's state): step = max|s| (1/127) in float32,
// code = the whole number nearest to s / step, and s' = code * step when it is read back.
// Whole numbers and not 8-bit floats: the elements of a row are of one size, where three
// bits of mantissa are off by up to 1/16 of each element, and 255 even steps by up to 1/254
// of the row's largest (0.6% rms for a row of 128 normal numbers).  The running state stays
// in float32: only what waits is rounded, once for each time that it is parked.
//
// Bound by reading and writing states.  Storing: neighbouring lanes hold a row, sixteen
// elements each (eight of a row of 16), in vectors of four a stride of the lanes apart, so
// that loads and stores fill whole sectors and a row's largest element takes three exchanges
// for sixteen elements.  Loading: four vectors of a thread in flight at once.

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

// The four codes of a vector, one a byte; `near` takes the largest distance of a quotient
// from its code.  1.5 * 2^23 added to a quotient leaves its nearest whole number in the
// sum's low bits.
__device__ __forceinline__ uint32_t codes_of(const float4& x, float inverse, float& near) {
    const uint64_t p[2] = {pair(x.x, x.y), pair(x.z, x.w)}, by = twice(inverse), magic = twice(12582912.f);
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint64_t t = fma2(p[i], by, magic);
        const uint64_t d = fma2(p[i], by, fma2(t, twice(-1.f), magic));
        float lo, hi;
        unpair(d, lo, hi);
        near = fmaxf(near, fmaxf(fabsf(lo), fabsf(hi)));
        unpair(t, lo, hi);
        b[2 * i] = __float_as_uint(lo), b[2 * i + 1] = __float_as_uint(hi);
    }
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// blockIdx.y: the sequence; `rows`: of one sequence's state.
template <int K>
__global__ void __launch_bounds__(kThreads)
state_store_kernel(int B, int64_t rows, int64_t slots, const float* __restrict__ states,
                   const int32_t* __restrict__ slot_of, signed char* __restrict__ cache, float* __restrict__ scales) {
    constexpr int LANES = K >= 32 ? K / 16 : 2, EACH = K / 4 / LANES, ROWS = kVectors / EACH;
    await_previous();
    const int b = blockIdx.y;
    const int64_t slot = slot_of[b];
    if (slot < 0 || slot >= slots) return;
    // of sequences with one slot the last one is kept
    bool later = false;
    for (int j = b + 1 + threadIdx.x; j < B; j += kThreads) later |= slot_of[j] == slot;
    if (__syncthreads_or(later)) return;
    const int u = threadIdx.x % LANES;
    const int64_t row0 = (int64_t)blockIdx.x * (kThreads / LANES * ROWS) + threadIdx.x / LANES;
    const float4* from = (const float4*)states + b * rows * (K / 4) + u;
    float4 x[ROWS][EACH];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t row = row0 + r * (kThreads / LANES);
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            x[r][i] = row < rows ? __ldcs(from + row * (K / 4) + i * LANES) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t row = row0 + r * (kThreads / LANES);
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            m = max_nan(m, max_nan(max_nan(fabsf(x[r][i].x), fabsf(x[r][i].y)), max_nan(fabsf(x[r][i].z), fabsf(x[r][i].w))));
#pragma unroll
        for (int off = LANES / 2; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        // no subnormal step, whose inverse would be infinite
        float step = m * (1.f / 127.f);
        if (step < 1.17549435e-38f) step = 1.17549435e-38f;
        const float inverse = inverse_of(step);
        float near = 0.f;
        uint32_t c[EACH];
#pragma unroll
        for (int i = 0; i < EACH; ++i) c[i] = codes_of(x[r][i], inverse, near);
        // the quotients are off by up to 127 * 2^-23 = 1.5e-5: next to a middle the remainder
        // decides (one element of 12500)
        if (near > 0.49996f) {
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                c[i] = (uint32_t)(code_of(x[r][i].x, step, inverse) & 255) | (uint32_t)(code_of(x[r][i].y, step, inverse) & 255) << 8 |
                       (uint32_t)(code_of(x[r][i].z, step, inverse) & 255) << 16 | (uint32_t)code_of(x[r][i].w, step, inverse) << 24;
        }
        // a row that is not finite is read back as NaN
        const bool fine = step <= 3.402823466e38f;
        if (row >= rows) continue;
        uint32_t* to = reinterpret_cast<uint32_t*>(cache) + (slot * rows + row) * (K / 4) + u;
#pragma unroll
        for (int i = 0; i < EACH; ++i) to[i * LANES] = fine ? c[i] : 0;
        if (u == 0) scales[slot * rows + row] = fine ? step : __int_as_float(0x7fc00000);
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

template <int K>
cudaError_t launch_k(const StateCall& c, bool load, cudaStream_t st) {
    const int64_t vectors = c.rows * (K / 4), per = kThreads * kVectors;
    const dim3 grid((unsigned)((vectors + per - 1) / per), (unsigned)c.B);
    if (load)
        return launch_dependent(state_load_kernel<K / 4>, grid, kThreads, 0, st, vectors, c.slots,
                                (const signed char*)c.cache, (const float*)c.scales, c.slot_of, c.out);
    return launch_dependent(state_store_kernel<K>, grid, kThreads, 0, st, c.B, c.rows, c.slots, c.states, c.slot_of,
                            (signed char*)c.cache, c.scales);
}

}  // namespace

cudaError_t launch_state_cache(const StateCall& c, bool load, cudaStream_t st) {
    switch (c.K) {
        case 16: return launch_k<16>(c, load, st);
        case 32: return launch_k<32>(c, load, st);
        case 64: return launch_k<64>(c, load, st);
        default: return launch_k<128>(c, load, st);
    }
}

}  // namespace gdn
