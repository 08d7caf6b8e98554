// f32x2.cuh -- two float32 operations in one instruction (sm_100 and later): a pair of
// values in a 64-bit register.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ void unpair(uint64_t p, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t twice(float x) { return pair(x, x); }
__device__ __forceinline__ float sum2(uint64_t p) {
    float x, y;
    unpair(p, x, y);
    return x + y;
}
// Two bf16 (the lower half first) as a pair.
__device__ __forceinline__ uint64_t bf16_pair(uint32_t v) {
    return pair(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

}  // namespace gdn
