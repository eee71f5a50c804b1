// The gate of a gated feed-forward: silu(g) * u with silu(g) = g * sigmoid(g),
// shared by the forward epilogues and the backward kernel.
#pragma once

#include <cuda_runtime.h>

namespace fp8fg {

// sigmoid(v), and its complement sigmoid(-v) without the cancellation of
// 1 - sigmoid(v).
struct Sigmoid2 {
    float2 s, c;
};

// With e = exp(-v): s = 1 / (1 + e), c = e / (1 + e), as good as FP32 products
// and sums are (8 2^-24 relative, however large |v| is).
//
// A rounded exponent of 2^(-v log2 e) alone would make e wrong by |v| 2^-24.
// So the argument is split in Cody and Waite's manner: the exponent h is -v log2 e
// rounded to a multiple of 2^-12, which FP32 holds with room to spare, and what
// the rounding left out, lo = -v - h ln 2 in two fused steps, comes back as the
// factor 1 + lo (lo below 2^-13; the next term of exp(lo) below 2^-27). e and 1
// are carried with a factor 2^-64, so that neither e nor the quotient leaves the
// range of normal numbers from v = -110, where sigmoid(v) rounds to 0, up to v =
// 43, where c no longer counts beside s; c is 0 beyond. The result's factor 2^-64
// is exact, or one rounding to a subnormal number. The hardware's power of two is
// good to 2 ulp, its reciprocal to 1.
//
// The bare approximations (a rounded exponent, flushed to zero below 2^-126) are
// six instructions a pair, this is thirteen: the gate backward of 4096 x 18432
// takes 147 us with it and 138 without, the forward pass of 4096 x 7168 x 18432
// 815 and 806. With the exponential function and a division they take 165 and
// 828.
__device__ __forceinline__ Sigmoid2 sigmoid2(float2 v)
{
    constexpr float GRID = 3072.0f;          // its ulp is 2^-12
    constexpr float ONE = 0x1p-64f;
    constexpr float LN2_HI = 0.693147180559945309417f;
    constexpr float LN2_LO = (float)(0.693147180559945309417 - (double)LN2_HI);
    const auto splat = [](float a) { return make_float2(a, a); };
    const float2 w = make_float2(fminf(-v.x, 110.0f), fminf(-v.y, 110.0f));
    const float2 grid = __ffma2_rn(w, splat(1.44269504088896340736f), splat(GRID));
    const float2 h = __fadd2_rn(grid, splat(-GRID)), hs = __fadd2_rn(grid, splat(-GRID - 64.0f));
    const float2 lo = __ffma2_rn(h, splat(-LN2_LO), __ffma2_rn(h, splat(-LN2_HI), w));
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(hs.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(hs.y));
    e = __ffma2_rn(e, lo, e);
    const float2 d = __fadd2_rn(e, splat(ONE));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    return {__fmul2_rn(r, splat(ONE)), __fmul2_rn(e, r)};
}

// silu(g) * u
__device__ __forceinline__ float2 silu_mul2(float2 g, float2 u)
{
    return __fmul2_rn(__fmul2_rn(g, sigmoid2(g).s), u);
}

}  // namespace fp8fg
