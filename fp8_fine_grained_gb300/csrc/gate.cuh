// The gate of a gated feed-forward: silu(g) * u with silu(g) = g * sigmoid(g),
// shared by the forward epilogues and the backward kernel.
#pragma once

#include <cuda_runtime.h>

namespace fp8fg {

// sigmoid(v) = 1 / (1 + 2^(-v log2 e)) of a pair. ex2.approx is good to 2^-22
// relative and the exponent's rounding adds |v| 2^-24, rcp.approx to 1 ulp: far
// inside the E4M3 (or bf16) rounding of whatever is made from it. An infinite
// power gives 0. Two special-function instructions per element and the rest on
// pairs: the gate is a third of the kernels' arithmetic.
__device__ __forceinline__ float2 sigmoid2(float2 v)
{
    const float2 x = __fmul2_rn(v, make_float2(-1.44269504f, -1.44269504f));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(x.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(x.y));
    e = __fadd2_rn(e, make_float2(1.0f, 1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
    return e;
}

// silu(g) * u
__device__ __forceinline__ float2 silu_mul2(float2 g, float2 u) { return __fmul2_rn(__fmul2_rn(g, sigmoid2(g)), u); }

}  // namespace fp8fg
