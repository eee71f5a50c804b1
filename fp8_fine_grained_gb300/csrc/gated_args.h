// Arguments of fp8_gated_gemm after its checks, passed between the two
// translation units that hold its kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8fg {

struct GatedArgs {
    const uint8_t *xq;  // [M][ldx]
    const float *sx;    // [K/128][ld_sx]
    const uint8_t *wq;  // [2I][ldw]: gate rows, then up rows
    const float *sw;    // [2I/128][K/128]
    int64_t ldx, ld_sx, ldw, M, K, I;
    uint8_t *h;  // [M][ldh]
    float *sh;   // [I/128][ld_sh]
    int64_t ldh, ld_sh;
    uint16_t *gu;  // bf16 [M][ld_gu] or nullptr
    int64_t ld_gu;
    int pow2;
};

// 128 rows x 128 columns of h per tile (gemm.cu).
int gated_gemm_tiles(const GatedArgs &g, cudaStream_t s);

}  // namespace fp8fg
