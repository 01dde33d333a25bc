// Arithmetic on pairs of binary32 values. (Not in cpt_device.cuh, whose text keys the gradient return's traffic record.)
#pragma once

#include <stdint.h>

namespace cpt {

// Two binary32 values in one register pair, and their arithmetic (round to
// nearest): one issue slot for two elements.
struct F2 {
    uint64_t v;
};

__device__ __forceinline__ F2 pair_of(uint32_t a, uint32_t b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ F2 pair_of(float a, float b) { return pair_of(__float_as_uint(a), __float_as_uint(b)); }

__device__ __forceinline__ float2 both(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}

__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

}  // namespace cpt
