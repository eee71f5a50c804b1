// Root-mean-square norm with the residual's addition and an E4M3 output in
// 1x128 groups, its transposed output for the weight gradient, and its
// backward pass.
//
//   h[t]    = bf16(x[t] + r[t])                    (r optional)
//   rstd[t] = (mean_j h[t][j]^2 + eps)^(-1/2)
//   y[t][j] = h[t][j] * rstd[t] * gamma[j]
//
// y exists in FP32 registers only; its groups of 128 columns are quantised by
// the group rule (group_rule.cuh), so the codes carry one rounding. The norm
// is taken of the rounded h because h is what the next block and the backward
// pass read.
//
// Backward, with a = dy * gamma and c = mean_j(a[j] * h[j]) * rstd:
//   dx[j]    = rstd * (a[j] - h[j] * rstd * c) (+ dres[j])
//   dgamma[j] = sum_t dy[t][j] * h[t][j] * rstd[t]
//
// All three are streams of whole rows: the row's chunks of 8 columns (16
// bytes) stay in registers from the load to the last store, so each tensor
// crosses the memory once.
#include <cuda_bf16.h>

#include "group_rule.cuh"
#include "host_common.h"
#include "ptx.cuh"

namespace fp8fg {
namespace {

constexpr int GROUP = 128;
constexpr int64_t NORM_MAX_D = 18432;  // 768 threads x 3 chunks of 8 columns

// largest CTA of a kernel whose threads own CPT chunks of a row (row_shape)
constexpr int max_threads(int cpt) { return 256 * cpt; }

// (not the read-only path: the outputs may be the inputs' own buffers)
__device__ __forceinline__ uint4 ld_stream(const uint16_t *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    f[0] = bf16_lo(v.x);
    f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y);
    f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z);
    f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w);
    f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// the norm's weight at columns 8c .. 8c+7
__device__ __forceinline__ void load_gamma(const void *gamma, bool f32, int c, float (&g)[8])
{
    if (f32) {
        const float4 a = __ldg(static_cast<const float4 *>(gamma) + 2 * c);
        const float4 b = __ldg(static_cast<const float4 *>(gamma) + 2 * c + 1);
        g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w, g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
    } else {
        unpack8(__ldg(static_cast<const uint4 *>(gamma) + c), g);
    }
}

// Sum over the block in a fixed order. `part` holds one slot per warp and is
// rewritten by the next call, so calls alternate between two of them: a
// thread that writes slot set b again has passed the barrier of the call on
// the other set, which every reader of b reaches after its reads.
__device__ __forceinline__ float block_sum(float v, float *part, int nwarps)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if (nwarps == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (int)(threadIdx.x & 31) < nwarps ? part[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct NormFwd {
    const uint16_t *x, *r;
    const void *gamma;
    uint16_t *h;
    uint8_t *q;
    float *scales, *rstd;
    int64_t T, ldx, ldr, ldh, ldq, ld_s;
    int D;
    float eps;
    bool gamma_f32;
};

// One row per CTA at a time: thread t owns chunks t, t + blockDim, ...; a
// half-warp's 16 chunks are one 128-column group (D % 128 == 0 and blockDim
// % 32 == 0 keep every group inside one half-warp).
template <int CPT, bool RES, bool P2>
__global__ void __launch_bounds__(max_threads(CPT)) rmsnorm_fwd_kernel(const NormFwd p)
{
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float part[2][32];
    const int nchunk = p.D / 8, nwarps = blockDim.x >> 5;
    int b = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, b ^= 1) {
        uint4 v[CPT], rv[CPT];
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            v[i] = rv[i] = make_uint4(0, 0, 0, 0);
            if (c < nchunk) {
                v[i] = ld_stream(p.x + t * p.ldx + 8 * c);
                if constexpr (RES)
                    rv[i] = ld_stream(p.r + t * p.ldr + 8 * c);
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            float f[8];
            unpack8(v[i], f);
            if constexpr (RES) {
                float r[8];
                unpack8(rv[i], r);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] += r[e];
                v[i] = pack8(f);
                unpack8(v[i], f);  // the rounded sum
                const int c = threadIdx.x + i * blockDim.x;
                if (c < nchunk)
                    *reinterpret_cast<uint4 *>(p.h + t * p.ldh + 8 * c) = v[i];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                ss = fmaf(f[e], f[e], ss);
        }
        ss = block_sum(ss, part[b], nwarps);
        const float rstd = rsqrtf(ss / (float)p.D + p.eps);
        if (threadIdx.x == 0)
            p.rstd[t] = rstd;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            const bool live = c < nchunk;
            float f[8], g[8];
            unpack8(v[i], f);
            load_gamma(p.gamma, p.gamma_f32, live ? c : 0, g);
            float amax = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = f[e] * rstd * g[e];
                amax = fmaxf(amax, fabsf(f[e]));
            }
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const ScalePair sp = group_scale_rule<P2>(amax);
            if (live) {
                uint2 o;
                o.x = cvt_e4m3x2(f[0] * sp.inv, f[1] * sp.inv) | (cvt_e4m3x2(f[2] * sp.inv, f[3] * sp.inv) << 16);
                o.y = cvt_e4m3x2(f[4] * sp.inv, f[5] * sp.inv) | (cvt_e4m3x2(f[6] * sp.inv, f[7] * sp.inv) << 16);
                *reinterpret_cast<uint2 *>(p.q + t * p.ldq + 8 * c) = o;
                if ((c & 15) == 0)
                    p.scales[(int64_t)(c >> 4) * p.ld_s + t] = sp.s;
            }
        }
    }
}

// y^T in groups of 128 rows: CTA tile 128 rows x 64 columns. Thread (c, part)
// holds rows 32*part .. +31 of column c of the tile; the four parts' maxima
// meet in shared memory and each thread writes its 32 codes as two 16-byte
// pieces of row c of the output.
constexpr int NT_COLS = 64;

template <bool P2>
__global__ void __launch_bounds__(256) rmsnorm_t_kernel(const uint16_t *__restrict__ h, int64_t ldh,
                                                        const float *__restrict__ rstd, const void *gamma,
                                                        bool gamma_f32, int64_t cols, uint8_t *__restrict__ qT,
                                                        int64_t ldq, float *__restrict__ scales, int64_t ld_s)
{
    griddep_launch_dependents();
    griddep_wait();
    __shared__ __align__(16) uint16_t tile[GROUP][NT_COLS + 2];
    __shared__ float s_rstd[GROUP], s_max[4][NT_COLS];
    const int tid = threadIdx.x;
    const int64_t c0 = (int64_t)blockIdx.x * NT_COLS, r0 = (int64_t)blockIdx.y * GROUP;
    if (tid < GROUP)
        s_rstd[tid] = rstd[r0 + tid];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int rr = (i * 256 + tid) >> 3, cc = (tid & 7) * 8;
        const uint4 v = ld_stream(h + (r0 + rr) * ldh + c0 + cc);
        uint32_t *d = reinterpret_cast<uint32_t *>(&tile[rr][cc]);
        d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
    }
    __syncthreads();
    const int c = tid & (NT_COLS - 1), part = tid >> 6;
    const float g = gamma_f32 ? static_cast<const float *>(gamma)[c0 + c]
                              : __bfloat162float(static_cast<const __nv_bfloat16 *>(gamma)[c0 + c]);
    float y[32], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int rr = part * 32 + i;
        y[i] = __uint_as_float((uint32_t)tile[rr][c] << 16) * s_rstd[rr] * g;
        amax = fmaxf(amax, fabsf(y[i]));
    }
    s_max[part][c] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(s_max[0][c], s_max[1][c]), fmaxf(s_max[2][c], s_max[3][c]));
    const ScalePair sp = group_scale_rule<P2>(amax);
    if (part == 0)
        scales[(int64_t)blockIdx.y * ld_s + c0 + c] = sp.s;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = cvt_e4m3x2(y[4 * i] * sp.inv, y[4 * i + 1] * sp.inv) |
               (cvt_e4m3x2(y[4 * i + 2] * sp.inv, y[4 * i + 3] * sp.inv) << 16);
    uint4 *o = reinterpret_cast<uint4 *>(qT + (c0 + c) * ldq + r0 + part * 32);
    o[0] = make_uint4(w[0], w[1], w[2], w[3]);
    o[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

struct NormBwd {
    const uint16_t *dy, *h, *dres;
    const float *rstd;
    const void *gamma;
    uint16_t *dx;
    float *part;  // [gridDim.x][D]
    int64_t T, lddy, ldh, lddres, lddx;
    int D;
    bool gamma_f32;
};

// Rows blockIdx, blockIdx + grid, ...; the thread's columns are the same in
// every row, so its dgamma terms add up in registers and leave once, as the
// CTA's row of `part`. norm_dgamma_kernel adds those rows up in order, so the
// result does not depend on the schedule.
template <int CPT, bool RES>
__global__ void __launch_bounds__(max_threads(CPT)) rmsnorm_bwd_kernel(const NormBwd p)
{
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float sums[2][32];
    const int nchunk = p.D / 8, nwarps = blockDim.x >> 5;
    float dg[CPT][8];
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            dg[i][e] = 0.0f;
    int b = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, b ^= 1) {
        uint4 dv[CPT], hv[CPT], rv[CPT];
        const float rstd = __ldg(p.rstd + t);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            dv[i] = hv[i] = rv[i] = make_uint4(0, 0, 0, 0);
            if (c < nchunk) {
                dv[i] = ld_stream(p.dy + t * p.lddy + 8 * c);
                hv[i] = ld_stream(p.h + t * p.ldh + 8 * c);
                if constexpr (RES)
                    rv[i] = ld_stream(p.dres + t * p.lddres + 8 * c);
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            float d[8], h[8], g[8];
            unpack8(dv[i], d);
            unpack8(hv[i], h);
            load_gamma(p.gamma, p.gamma_f32, c < nchunk ? c : 0, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dh = d[e] * h[e];
                dg[i][e] = fmaf(dh, rstd, dg[i][e]);
                dot = fmaf(dh, g[e], dot);
            }
        }
        dot = block_sum(dot, sums[b], nwarps);
        const float k = dot / (float)p.D * rstd * rstd;  // dx = rstd * (a - h k)
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nchunk)
                continue;
            float d[8], h[8], g[8], r[8];
            unpack8(dv[i], d);
            unpack8(hv[i], h);
            unpack8(rv[i], r);
            load_gamma(p.gamma, p.gamma_f32, c, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = rstd * fmaf(-h[e], k, d[e] * g[e]);
                d[e] = RES ? v + r[e] : v;
            }
            *reinterpret_cast<uint4 *>(p.dx + t * p.lddx + 8 * c) = pack8(d);
        }
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nchunk) {
            float4 *o = reinterpret_cast<float4 *>(p.part + (int64_t)blockIdx.x * p.D + 8 * c);
            o[0] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
            o[1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
        }
    }
}

// dgamma[c] = sum over the rows of part: 32 columns per CTA, 16 slices of the
// rows summed side by side and then in slice order.
constexpr int DG_SLICES = 16;

__global__ void __launch_bounds__(32 * DG_SLICES) norm_dgamma_kernel(const float *__restrict__ part, int rows, int D,
                                                                     float *__restrict__ dgamma)
{
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float s[DG_SLICES][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
    float v = 0.0f;
    for (int r = slice; r < rows; r += DG_SLICES)
        v += part[(int64_t)r * D + c];
    s[slice][threadIdx.x & 31] = v;
    __syncthreads();
    if (slice == 0) {
#pragma unroll
        for (int i = 1; i < DG_SLICES; ++i)
            v += s[i][threadIdx.x];
        dgamma[c] = v;
    }
}

// chunks per thread (the loads of a tensor that a thread has in flight) and
// threads of a row of D columns
struct RowShape {
    int cpt, threads;
};

RowShape row_shape(int64_t D)
{
    const int chunks = (int)(D / 8);
    const int cpt = chunks <= 256 ? 1 : (chunks <= 1024 ? 2 : 3);
    const int threads = ((chunks + cpt - 1) / cpt + 31) / 32 * 32;
    return {cpt, threads};
}

// CTAs of the forward kernel: what the device holds at once (48 registers a
// thread), so that every CTA runs from the start and strides over the rows
int fwd_grid(int64_t T, int threads)
{
    const int per_sm = 1344 / threads < 1 ? 1 : (1344 / threads > 32 ? 32 : 1344 / threads);
    const int64_t cap = (int64_t)sm_count() * per_sm;
    return (int)(T < cap ? T : (cap > 0 ? cap : 1));
}

// The backward kernel holds more per thread, and each CTA adds a row to the
// partial sums of dgamma.
int bwd_grid(int64_t T, int64_t D)
{
    const int threads = row_shape(D).threads;
    const int per_sm = 896 / threads < 1 ? 1 : (896 / threads > 8 ? 8 : 896 / threads);
    const int64_t cap = (int64_t)sm_count() * per_sm;
    return (int)(T < cap ? T : (cap > 0 ? cap : 1));
}

template <int CPT>
int launch_fwd(const NormFwd &p, int grid, int threads, bool p2, cudaStream_t s)
{
    if (p.r)
        return p2 ? launch_pss(rmsnorm_fwd_kernel<CPT, true, true>, dim3(grid), threads, 0, s, p)
                  : launch_pss(rmsnorm_fwd_kernel<CPT, true, false>, dim3(grid), threads, 0, s, p);
    return p2 ? launch_pss(rmsnorm_fwd_kernel<CPT, false, true>, dim3(grid), threads, 0, s, p)
              : launch_pss(rmsnorm_fwd_kernel<CPT, false, false>, dim3(grid), threads, 0, s, p);
}

template <int CPT>
int launch_bwd(const NormBwd &p, int grid, int threads, cudaStream_t s)
{
    return p.dres ? launch_pss(rmsnorm_bwd_kernel<CPT, true>, dim3(grid), threads, 0, s, p)
                  : launch_pss(rmsnorm_bwd_kernel<CPT, false>, dim3(grid), threads, 0, s, p);
}

bool norm_width_ok(int64_t D) { return D >= 0 && D % GROUP == 0 && D <= NORM_MAX_D; }

}  // namespace
}  // namespace fp8fg

using namespace fp8fg;

extern "C" int fp8_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *gamma,
                           int gamma_kind, int64_t T, int64_t D, float eps, void *h, int64_t ldh, uint8_t *q,
                           int64_t ldq, float *scales, int64_t ld_s, float *rstd, int pow2, void *stream)
{
    if (T < 0 || !norm_width_ok(D) || !(eps > 0.0f) || isinf(eps) || (pow2 != 0 && pow2 != 1) ||
        (gamma_kind != FP8FG_OUT_F32 && gamma_kind != FP8FG_OUT_BF16))
        return FP8FG_EINVAL;
    if (T >= (1ll << 31) || ldx < D || ldq < D || ld_s < T || (residual && (ldr < D || ldh < D)))
        return FP8FG_EINVAL;
    if (T == 0 || D == 0)
        return FP8FG_OK;
    if (!x || !gamma || !q || !scales || !rstd || (residual && !h))
        return FP8FG_EINVAL;
    if (!aligned16(x) || !aligned16(gamma) || !aligned16(q) || !aligned16(scales) || ldx % 8 != 0 || ldq % 16 != 0 ||
        ld_s % 4 != 0 || (reinterpret_cast<uintptr_t>(rstd) & 3u) != 0)
        return FP8FG_EALIGN;
    if (residual && (!aligned16(residual) || !aligned16(h) || ldr % 8 != 0 || ldh % 8 != 0))
        return FP8FG_EALIGN;
    if (!device_supported())
        return FP8FG_EUNSUPPORTED;
    NormFwd p{};
    p.x = static_cast<const uint16_t *>(x);
    p.r = static_cast<const uint16_t *>(residual);
    p.gamma = gamma;
    p.h = static_cast<uint16_t *>(h);
    p.q = q;
    p.scales = scales;
    p.rstd = rstd;
    p.T = T, p.ldx = ldx, p.ldr = ldr, p.ldh = ldh, p.ldq = ldq, p.ld_s = ld_s;
    p.D = (int)D;
    p.eps = eps;
    p.gamma_f32 = gamma_kind == FP8FG_OUT_F32;
    const RowShape rs = row_shape(D);
    const int grid = fwd_grid(T, rs.threads);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (rs.cpt) {
    case 1: return launch_fwd<1>(p, grid, rs.threads, pow2 != 0, s);
    case 2: return launch_fwd<2>(p, grid, rs.threads, pow2 != 0, s);
    default: return launch_fwd<3>(p, grid, rs.threads, pow2 != 0, s);
    }
}

extern "C" int fp8_rmsnorm_t(const void *h, int64_t ldh, const float *rstd, const void *gamma, int gamma_kind,
                             int64_t T, int64_t D, uint8_t *qT, int64_t ldqT, float *scalesT, int64_t ld_sT, int pow2,
                             void *stream)
{
    if (T < 0 || T % GROUP != 0 || !norm_width_ok(D) || (pow2 != 0 && pow2 != 1) ||
        (gamma_kind != FP8FG_OUT_F32 && gamma_kind != FP8FG_OUT_BF16))
        return FP8FG_EINVAL;
    if (T / GROUP > 65535 || ldh < D || ldqT < T || ld_sT < D)
        return FP8FG_EINVAL;
    if (T == 0 || D == 0)
        return FP8FG_OK;
    if (!h || !rstd || !gamma || !qT || !scalesT)
        return FP8FG_EINVAL;
    if (!aligned16(h) || !aligned16(gamma) || !aligned16(qT) || !aligned16(scalesT) || ldh % 8 != 0 ||
        ldqT % 16 != 0 || ld_sT % 4 != 0 || (reinterpret_cast<uintptr_t>(rstd) & 3u) != 0)
        return FP8FG_EALIGN;
    if (!device_supported())
        return FP8FG_EUNSUPPORTED;
    const dim3 grid((unsigned)(D / NT_COLS), (unsigned)(T / GROUP));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint16_t *hp = static_cast<const uint16_t *>(h);
    const bool f32 = gamma_kind == FP8FG_OUT_F32;
    return pow2 ? launch_pss(rmsnorm_t_kernel<true>, grid, 256, 0, s, hp, ldh, rstd, gamma, f32, D, qT, ldqT, scalesT, ld_sT)
                : launch_pss(rmsnorm_t_kernel<false>, grid, 256, 0, s, hp, ldh, rstd, gamma, f32, D, qT, ldqT, scalesT,
                             ld_sT);
}

extern "C" int64_t fp8_rmsnorm_bwd_workspace(int64_t T, int64_t D)
{
    if (T <= 0 || D <= 0 || !norm_width_ok(D))
        return 0;
    return (int64_t)bwd_grid(T, D) * D * 4;
}

extern "C" int fp8_rmsnorm_bwd(const void *dy, int64_t lddy, const void *h, int64_t ldh, const float *rstd,
                               const void *gamma, int gamma_kind, const void *dres, int64_t lddres, int64_t T,
                               int64_t D, void *dx, int64_t lddx, float *dgamma, void *workspace,
                               int64_t workspace_bytes, void *stream)
{
    if (T < 0 || !norm_width_ok(D) || (gamma_kind != FP8FG_OUT_F32 && gamma_kind != FP8FG_OUT_BF16))
        return FP8FG_EINVAL;
    if (T >= (1ll << 31) || lddy < D || ldh < D || lddx < D || (dres && lddres < D))
        return FP8FG_EINVAL;
    if (D == 0)
        return FP8FG_OK;
    if (!dgamma)
        return FP8FG_EINVAL;
    if (!aligned16(dgamma))
        return FP8FG_EALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {  // an empty sum
        if (!device_supported())
            return FP8FG_EUNSUPPORTED;
        if (cudaMemsetAsync(dgamma, 0, (size_t)D * 4, s) != cudaSuccess) {
            cudaGetLastError();
            return FP8FG_ECUDA;
        }
        return FP8FG_OK;
    }
    if (!dy || !h || !rstd || !gamma || !dx || !workspace)
        return FP8FG_EINVAL;
    if (!aligned16(dy) || !aligned16(h) || !aligned16(gamma) || !aligned16(dx) || !aligned16(workspace) ||
        lddy % 8 != 0 || ldh % 8 != 0 || lddx % 8 != 0 || (reinterpret_cast<uintptr_t>(rstd) & 3u) != 0)
        return FP8FG_EALIGN;
    if (dres && (!aligned16(dres) || lddres % 8 != 0))
        return FP8FG_EALIGN;
    if (!device_supported())
        return FP8FG_EUNSUPPORTED;
    const int grid = bwd_grid(T, D);
    if (workspace_bytes < (int64_t)grid * D * 4)
        return FP8FG_EINVAL;
    NormBwd p{};
    p.dy = static_cast<const uint16_t *>(dy);
    p.h = static_cast<const uint16_t *>(h);
    p.dres = static_cast<const uint16_t *>(dres);
    p.rstd = rstd;
    p.gamma = gamma;
    p.dx = static_cast<uint16_t *>(dx);
    p.part = static_cast<float *>(workspace);
    p.T = T, p.lddy = lddy, p.ldh = ldh, p.lddres = lddres, p.lddx = lddx;
    p.D = (int)D;
    p.gamma_f32 = gamma_kind == FP8FG_OUT_F32;
    const RowShape rs = row_shape(D);
    int rc;
    switch (rs.cpt) {
    case 1: rc = launch_bwd<1>(p, grid, rs.threads, s); break;
    case 2: rc = launch_bwd<2>(p, grid, rs.threads, s); break;
    default: rc = launch_bwd<3>(p, grid, rs.threads, s); break;
    }
    if (rc != FP8FG_OK)
        return rc;
    return launch_pss(norm_dgamma_kernel, dim3((unsigned)(D / 32)), 32 * DG_SLICES, 0, s, p.part, grid, (int)D, dgamma);
}
