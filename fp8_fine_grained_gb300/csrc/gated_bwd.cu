// Backward pass of the gate of a gated feed-forward, quantised for the GEMMs
// that follow.
//
// Forward: h = silu(G) * U with silu(v) = v * sigmoid(v). With dh the
// gradient of h, sg = sigmoid(G) and a = G * sg:
//   dG = dh * U * (sg + a * (1 - sg)),   dU = dh * a,   h = a * U.
// Three products consume them, and each wants its operand in E4M3 with groups
// of 128 along its own contraction dimension:
//   dX   = [dG dU] W      groups along the columns of a row   (q, scales)
//   dW   = [dG dU]^T X    groups along the rows of a column   (qT, scalesT)
//   dWdn = dY^T h         groups along the rows of a column   (hqT, hscalesT)
// One kernel reads G, U and dh once (6 bytes per element of h) and writes the
// five quantised matrices (5 bytes): the FP32 values live in registers
// between, so every code is one rounding of the FP32 result.
//
// GB300 design: one persistent CTA of 16 warps per SM over 128x128 tiles (the
// smallest tile that holds whole groups in both directions). 4096 x 18432 takes
// 147 us: 11.16 bytes per element, 5.7 TB/s or 0.84 of the measured copy; the
// sigmoid's arithmetic is the last 10 us of it. Warp w computes
// rows 8w..8w+7, lane l columns 4l..4l+3: 96 FP32 values per thread. The row
// groups are reduced inside the warp, the column groups across the warps
// through shared memory; the transposed codes pass through shared memory so
// that their stores are whole 128-byte runs. The input tiles come by TMA; they
// are dead once the threads hold them in registers, so the next tile's loads
// run under the arithmetic and the stores of the current one.
#include <cuda_bf16.h>

#include "gate.cuh"
#include "group_rule.cuh"
#include "host_common.h"
#include "ptx.cuh"
#include "tensor_map.h"

namespace fp8fg {
namespace {

constexpr int GROUP = 128;
constexpr int WARPS = 16;
constexpr int THREADS = WARPS * 32;
constexpr int ROWS = GROUP / WARPS;  // rows of a tile per warp
constexpr uint32_t TILE_BYTES = GROUP * GROUP * 2;

struct Smem {
    uint16_t in[3][GROUP][GROUP];    // G, U, dh as the TMA boxes land
    uint8_t codes[3][GROUP][GROUP];  // dG, dU, h: row = column of the tile, 8-byte pieces swizzled
    float cmax[3][WARPS][GROUP];     // column maxima of each warp's rows
    float cinv[3][GROUP];
    uint64_t bar;
    int abort;
};

// (volatile: the inputs are in registers before the barrier that lets the next
// tile overwrite them)
__device__ __forceinline__ uint2 lds8(const uint16_t *p)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(smem_u32(p)));
    return v;
}

struct Params {
    int64_t tiles_c, n_tiles, I;
    uint8_t *q;
    int64_t ldq;
    float *scales;
    int64_t ld_s;
    uint8_t *qT;
    int64_t ldqT;
    float *scalesT;
    int64_t ld_sT;
    uint8_t *hqT;
    int64_t ldhT;
    float *hscalesT;
    int64_t ld_hsT;
    int *status;
    uint64_t wait_limit_ns;
    int skip_first_load;
};

template <bool P2>
__global__ void __launch_bounds__(THREADS, 1)
    gated_bwd_kernel(const __grid_constant__ CUtensorMap tm_gu, const __grid_constant__ CUtensorMap tm_dh,
                     const Params p)
{
    extern __shared__ __align__(128) uint8_t raw[];
    Smem &S = *reinterpret_cast<Smem *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t bar = smem_u32(&S.bar);
    griddep_launch_dependents();
    if (tid == 0) {
        mbar_init(bar, 1);
        S.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_gu);
        tma_prefetch_desc(&tm_dh);
    }
    __syncthreads();
    griddep_wait();
    const WaitCtl wc{&S.abort, p.status, p.wait_limit_ns};
    auto fetch = [&](int64_t t) {
        const int32_t c0 = (int32_t)((t % p.tiles_c) * GROUP), r0 = (int32_t)((t / p.tiles_c) * GROUP);
        mbar_arrive_expect_tx(bar, 3 * TILE_BYTES);
        tma_load_2d(smem_u32(&S.in[0][0][0]), &tm_gu, c0, r0, bar);
        tma_load_2d(smem_u32(&S.in[1][0][0]), &tm_gu, (int32_t)p.I + c0, r0, bar);
        tma_load_2d(smem_u32(&S.in[2][0][0]), &tm_dh, c0, r0, bar);
    };
    // (test hook: CTA 0 withholds its first copies, so that its bounded wait
    // runs out and the launch reports FP8FG_ETIMEOUT)
    if (tid == 0 && (int64_t)blockIdx.x < p.n_tiles && !(p.skip_first_load && blockIdx.x == 0))
        fetch(blockIdx.x);
    uint32_t phase = 0;
    for (int64_t t = blockIdx.x; t < p.n_tiles; t += gridDim.x, phase ^= 1) {
        const int64_t c0 = (t % p.tiles_c) * GROUP, r0 = (t / p.tiles_c) * GROUP;
        const bool got = mbar_wait(bar, phase, wc, FP8FG_ETIMEOUT);
        if (!__syncthreads_and(got)) {
            if (tid == 0) {  // copies in flight land before the CTA leaves
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(bar, phase) && global_timer_ns() - t0 < p.wait_limit_ns) {
                }
            }
            return;
        }
        uint2 gw[ROWS], uw[ROWS], dw[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int row = warp * ROWS + i;
            gw[i] = lds8(&S.in[0][row][4 * lane]);
            uw[i] = lds8(&S.in[1][row][4 * lane]);
            dw[i] = lds8(&S.in[2][row][4 * lane]);
        }
        __syncthreads();
        // every thread holds its inputs: the next tile may land
        if (tid == 0 && t + gridDim.x < p.n_tiles)
            fetch(t + gridDim.x);
        // v[0] = dG, v[1] = dU, v[2] = h, in pairs of columns
        float2 v[3][ROWS][2];
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t gb = j ? gw[i].y : gw[i].x, ub = j ? uw[i].y : uw[i].x, db = j ? dw[i].y : dw[i].x;
                const float2 g = make_float2(bf16_lo(gb), bf16_hi(gb));
                const float2 u = make_float2(bf16_lo(ub), bf16_hi(ub));
                const float2 d = make_float2(bf16_lo(db), bf16_hi(db));
                const Sigmoid2 sg = sigmoid2(g);
                const float2 a = __fmul2_rn(g, sg.s);
                v[0][i][j] = __fmul2_rn(__fmul2_rn(d, u), __ffma2_rn(a, sg.c, sg.s));
                v[1][i][j] = __fmul2_rn(d, a);
                v[2][i][j] = __fmul2_rn(a, u);
            }
        // column maxima of this warp's rows
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    m[2 * j] = fmaxf(m[2 * j], fabsf(v[k][i][j].x));
                    m[2 * j + 1] = fmaxf(m[2 * j + 1], fabsf(v[k][i][j].y));
                }
            *reinterpret_cast<float4 *>(&S.cmax[k][warp][4 * lane]) = make_float4(m[0], m[1], m[2], m[3]);
        }
        __syncthreads();
        // column groups: one thread each
        if (tid < 3 * GROUP) {
            const int k = tid / GROUP, c = tid % GROUP;
            float m = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                m = fmaxf(m, S.cmax[k][w][c]);
            const ScalePair sp = group_scale_rule<P2>(m);
            S.cinv[k][c] = sp.inv;
            const int64_t rg = r0 / GROUP;
            if (k < 2)
                p.scalesT[rg * p.ld_sT + k * p.I + c0 + c] = sp.s;
            else
                p.hscalesT[rg * p.ld_hsT + c0 + c] = sp.s;
        }
        // row groups of dG and dU: the warp's 16 maxima, then one division
        // sequence with lane 8k + i on group (k, i)
        float mine = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const float m = fmaxf(fmaxf(fabsf(v[k][i][0].x), fabsf(v[k][i][0].y)),
                                      fmaxf(fabsf(v[k][i][1].x), fabsf(v[k][i][1].y)));
                const uint32_t r = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
                mine = (lane & 15) == ROWS * k + i ? __uint_as_float(r) : mine;
            }
        const ScalePair rp = group_scale_rule<P2>(mine);
        if (lane < 2 * ROWS) {
            const int k = lane / ROWS, i = lane % ROWS;
            p.scales[((k * p.I + c0) / GROUP) * p.ld_s + r0 + warp * ROWS + i] = rp.s;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const float inv = __shfl_sync(0xffffffffu, rp.inv, ROWS * k + i);
                const float2 lo = __fmul2_rn(v[k][i][0], make_float2(inv, inv));
                const float2 hi = __fmul2_rn(v[k][i][1], make_float2(inv, inv));
                const uint32_t w = cvt_e4m3x2(lo.x, lo.y) | (cvt_e4m3x2(hi.x, hi.y) << 16);
                *reinterpret_cast<uint32_t *>(p.q + (r0 + warp * ROWS + i) * p.ldq + k * p.I + c0 + 4 * lane) = w;
            }
        __syncthreads();
        // transposed codes: 8 rows of a column are one 8-byte piece, piece
        // `warp` of its column at slot warp ^ (lane & 15): a half-warp's
        // stores (columns 4l + j, l = 0..15) then cover all banks
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const float4 iv = *reinterpret_cast<const float4 *>(&S.cinv[k][4 * lane]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 inv = j ? make_float2(iv.z, iv.w) : make_float2(iv.x, iv.y);
                uint32_t w0[2], w1[2];  // columns 2j and 2j + 1
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2 s2[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s2[i] = __fmul2_rn(v[k][4 * h + i][j], inv);
                    w0[h] = cvt_e4m3x2(s2[0].x, s2[1].x) | (cvt_e4m3x2(s2[2].x, s2[3].x) << 16);
                    w1[h] = cvt_e4m3x2(s2[0].y, s2[1].y) | (cvt_e4m3x2(s2[2].y, s2[3].y) << 16);
                }
                const int piece = 8 * (warp ^ (lane & 15));
                *reinterpret_cast<uint2 *>(&S.codes[k][4 * lane + 2 * j][piece]) = make_uint2(w0[0], w0[1]);
                *reinterpret_cast<uint2 *>(&S.codes[k][4 * lane + 2 * j + 1][piece]) = make_uint2(w1[0], w1[1]);
            }
        }
        __syncthreads();
        // 16 codes per thread and store: eight threads write one column's run
#pragma unroll
        for (int n = 0; n < 6; ++n) {
            const int k = n >> 1, c = (n & 1) * 64 + (tid >> 3), pc = tid & 7;  // pieces 2pc, 2pc + 1
            const int f = (c >> 2) & 15;
            const uint4 w = *reinterpret_cast<const uint4 *>(&S.codes[k][c][16 * (pc ^ (f >> 1))]);
            const uint4 o = (f & 1) ? make_uint4(w.z, w.w, w.x, w.y) : w;
            uint8_t *dst = k < 2 ? p.qT + (k * p.I + c0 + c) * p.ldqT : p.hqT + (c0 + c) * p.ldhT;
            *reinterpret_cast<uint4 *>(dst + r0 + 16 * pc) = o;
        }
    }
}

template <bool P2>
int launch(const CUtensorMap &gu, const CUtensorMap &dh, const Params &p, cudaStream_t s)
{
    auto k = gated_bwd_kernel<P2>;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(k, sizeof(Smem), done))
        return FP8FG_ECUDA;
    const int64_t sms = sm_count();
    const unsigned grid = (unsigned)(p.n_tiles < sms ? p.n_tiles : (sms > 0 ? sms : 1));
    return launch_pss(k, dim3(grid), THREADS, sizeof(Smem), s, gu, dh, p);
}

}  // namespace
}  // namespace fp8fg

using namespace fp8fg;

extern "C" int fp8_gated_bwd(const void *gu, int64_t ldgu, const void *dh, int64_t lddh, int64_t M, int64_t I,
                             uint8_t *q, int64_t ldq, float *scales, int64_t ld_s, uint8_t *qT, int64_t ldqT,
                             float *scalesT, int64_t ld_sT, uint8_t *hqT, int64_t ldhT, float *hscalesT,
                             int64_t ld_hsT, int pow2, void *stream)
{
    if (M < 0 || I < 0 || M % GROUP != 0 || I % GROUP != 0 || (pow2 != 0 && pow2 != 1))
        return FP8FG_EINVAL;
    if (M >= (1ll << 31) || I >= (1ll << 30) || ldgu < 2 * I || lddh < I || ldq < 2 * I || ld_s < M || ldqT < M ||
        ld_sT < 2 * I || ldhT < M || ld_hsT < I)
        return FP8FG_EINVAL;
    if (M == 0 || I == 0)
        return FP8FG_OK;
    if (!gu || !dh || !q || !scales || !qT || !scalesT || !hqT || !hscalesT)
        return FP8FG_EINVAL;
    if (!aligned16(gu) || !aligned16(dh) || !aligned16(q) || !aligned16(scales) || !aligned16(qT) ||
        !aligned16(scalesT) || !aligned16(hqT) || !aligned16(hscalesT) || ldgu % 8 != 0 || lddh % 8 != 0 ||
        ldq % 16 != 0 || ldqT % 16 != 0 || ldhT % 16 != 0 || ld_s % 4 != 0 || ld_sT % 4 != 0 || ld_hsT % 4 != 0)
        return FP8FG_EALIGN;
    if (!device_supported())
        return FP8FG_EUNSUPPORTED;
    Params p{};
    p.tiles_c = I / GROUP;
    p.n_tiles = p.tiles_c * (M / GROUP);
    p.I = I;
    p.q = q, p.ldq = ldq, p.scales = scales, p.ld_s = ld_s;
    p.qT = qT, p.ldqT = ldqT, p.scalesT = scalesT, p.ld_sT = ld_sT;
    p.hqT = hqT, p.ldhT = ldhT, p.hscalesT = hscalesT, p.ld_hsT = ld_hsT;
    p.status = status_word_ptr();
    p.wait_limit_ns = wait_limit_ns();
    p.skip_first_load = take_skip_first_load() ? 1 : 0;
    CUtensorMap tg, td;
    if (!p.status ||
        !make_map_bf16_tile(&tg, gu, (uint64_t)(2 * I), (uint64_t)M, (uint64_t)ldgu, GROUP, GROUP) ||
        !make_map_bf16_tile(&td, dh, (uint64_t)I, (uint64_t)M, (uint64_t)lddh, GROUP, GROUP))
        return FP8FG_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return pow2 ? launch<true>(tg, td, p, s) : launch<false>(tg, td, p, s);
}
