// Gated feed-forward of E4M3 operands: both projections, the activation and
// the product in one kernel, with an E4M3 output in 1x128 groups.
//
//   G = X Wg^T, U = X Wu^T      (promoted block-scaled products, W = [Wg; Wu])
//   h = silu(G) * U             FP32, quantised by the group rule
//
// The tiles are those of the block-scaled GEMM (gemm.cu, mode GATED).
#include "gated_args.h"
#include "host_common.h"

using namespace fp8fg;

extern "C" int fp8_gated_gemm(const uint8_t *xq, const float *sx, int64_t ldx, int64_t ld_sx, const uint8_t *wq,
                              const float *sw, int64_t ldw, int64_t M, int64_t I, int64_t K, uint8_t *h, int64_t ldh,
                              float *scales, int64_t ld_s, void *gu, int64_t ldgu, int pow2, void *stream)
{
    if (M < 0 || I < 0 || K < 128 || I % 128 != 0 || K % 128 != 0 || (pow2 != 0 && pow2 != 1))
        return FP8FG_EINVAL;
    if (M >= (1ll << 31) || I >= (1ll << 30) || K >= (1ll << 31))
        return FP8FG_EINVAL;
    if (ldx < K || ldw < K || ld_sx < M || ldh < I || ld_s < M || (gu && ldgu < 2 * I))
        return FP8FG_EINVAL;
    if (M == 0 || I == 0)
        return FP8FG_OK;
    if (!xq || !sx || !wq || !sw || !h || !scales)
        return FP8FG_EINVAL;
    if (!aligned16(xq) || !aligned16(sx) || !aligned16(wq) || !aligned16(h) || !aligned16(scales) || ldx % 16 != 0 ||
        ldw % 16 != 0 || ldh % 16 != 0 || ld_sx % 4 != 0 || ld_s % 4 != 0 ||
        (reinterpret_cast<uintptr_t>(sw) & 3u) != 0)
        return FP8FG_EALIGN;
    if (gu && (!aligned16(gu) || ldgu % 8 != 0))
        return FP8FG_EALIGN;
    if (!device_supported())
        return FP8FG_EUNSUPPORTED;
    GatedArgs g{};
    g.xq = xq, g.sx = sx, g.wq = wq, g.sw = sw;
    g.ldx = ldx, g.ld_sx = ld_sx, g.ldw = ldw, g.M = M, g.K = K, g.I = I;
    g.h = h, g.sh = scales, g.ldh = ldh, g.ld_sh = ld_s;
    g.gu = static_cast<uint16_t *>(gu), g.ld_gu = ldgu;
    g.pow2 = pow2;
    return gated_gemm_tiles(g, static_cast<cudaStream_t>(stream));
}
