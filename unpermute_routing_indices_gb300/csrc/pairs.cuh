// Arithmetic on pairs of fp32 values (sm_100 and later).
#pragma once

#include "common.cuh"

namespace mp {

// Two fp32 values in a register pair, and arithmetic on both at once.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float a, float b)
{
    f2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float2 both(f2 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ float sum2(f2 v)
{
    const float2 r = both(v);
    return r.x + r.y;
}

}  // namespace mp
