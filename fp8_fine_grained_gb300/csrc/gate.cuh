// The gate of a gated feed-forward: silu(g) * u with silu(g) = g * sigmoid(g),
// shared by the forward epilogues and the backward kernel.
#pragma once

#include <cuda_runtime.h>

namespace fp8fg {

// sigmoid(v) = 1 / (1 + exp(-v)). The hardware exponential's relative error is
// about 2 ulp plus |v| 2^-24 and the quotient's 2 ulp: far inside the E4M3 (or
// bf16) rounding of whatever is made from it. exp(-v) = inf gives 0.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

__device__ __forceinline__ float silu_mul(float g, float u) { return g * sigmoid(g) * u; }

}  // namespace fp8fg
