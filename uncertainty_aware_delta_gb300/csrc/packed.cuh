// Two fp32 operations an instruction.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kdn {

typedef unsigned long long pair_t;

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<pair_t&>(d)) : "l"(reinterpret_cast<pair_t&>(a)), "l"(reinterpret_cast<pair_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<pair_t&>(d)) : "l"(reinterpret_cast<pair_t&>(a)), "l"(reinterpret_cast<pair_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(reinterpret_cast<pair_t&>(d))
        : "l"(reinterpret_cast<pair_t&>(a)), "l"(reinterpret_cast<pair_t&>(b)), "l"(reinterpret_cast<pair_t&>(c)));
    return d;
}
// two bf16 values
__device__ __forceinline__ float2 unpack2(uint32_t x) { return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)); }

}  // namespace kdn
