// packed.cuh -- fp32 arithmetic on pairs (one instruction for two values): the
// kernels that are bound by instruction issue use it; each half rounds as its
// scalar counterpart does.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace gdn2 {

using f2 = uint64_t;

__device__ __forceinline__ f2 pack2(float x, float y)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ f2 both(float x) { return pack2(x, x); }
__device__ __forceinline__ float2 unpack2(f2 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 x, f2 y, f2 z)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 x, f2 y)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ f2 add2(f2 x, f2 y)
{
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ float sum2(f2 v)
{
    const float2 u = unpack2(v);
    return u.x + u.y;
}

// Two consecutive elements as a pair, and back.
__device__ __forceinline__ f2 pair_of(const float *e) { return pack2(e[0], e[1]); }
__device__ __forceinline__ f2 pair_of(const __nv_bfloat16 *e)
{
    const uint32_t w = *reinterpret_cast<const uint32_t *>(e);
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t bf16_pair(f2 v)
{
    const float2 u = unpack2(v);
    const __nv_bfloat162 h = __floats2bfloat162_rn(u.x, u.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

}  // namespace gdn2
