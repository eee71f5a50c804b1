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
// Forward and backward are streams of whole rows. A row has to be reduced
// before its first output is known, so a CTA that loads, reduces and stores one
// row after the other leaves the memory idle most of the time. Each CTA
// therefore has its next rows brought into a ring in shared memory by bulk
// copies while it works on the current one; the row's values stay in registers
// from there to the last store, so each tensor crosses the memory once. In
// flight per SM from 1024 columns on: 80 to 190 KB forward and 96 to 216
// backward (rows of over 8192 columns without a residual 48 to 72 forward);
// narrower rows are bound by their CTAs' number, 14 KB at 128 columns.
#include <cuda_bf16.h>

#include <algorithm>

#include "group_rule.cuh"
#include "host_common.h"
#include "ptx.cuh"

namespace fp8fg {
namespace {

constexpr int GROUP = 128;
constexpr int64_t NORM_MAX_D = 18432;  // 768 threads x 3 chunks of 8 columns

// Widths of a kernel: chunks of 8 columns per thread, the largest CTA and the
// CTAs of that size per SM that the registers must allow. Rows of up to 1024
// columns take one warp; WIDE starts above 8192 columns.
enum Width { ONE = 0, TWO = 1, FOUR = 2, WIDE = 3 };
constexpr int cpt_of(int w) { return w == ONE ? 1 : (w == TWO ? 2 : (w == FOUR ? 4 : 3)); }
constexpr int max_threads(int w) { return w < FOUR ? 32 : (w == FOUR ? 256 : 768); }
constexpr int min_ctas(int w, bool bwd) { return w < FOUR ? (bwd ? 12 : 28) : (w == FOUR ? (bwd ? 2 : 3) : 1); }

// Every kernel here may start before the stream's previous kernel ends, so what
// that kernel may have written is read after griddep_wait and never by the
// read-only path (__ldg, const __restrict__), which promises data that does not
// change while the grid runs. (The outputs may be the inputs' own buffers, too.)
__device__ __forceinline__ uint4 ld_stream(const uint16_t *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// 8 bf16 values <-> 4 pairs of FP32 (the arithmetic below is on pairs: one
// instruction for two elements)
__device__ __forceinline__ void unpack8(const uint4 &v, float2 (&f)[4])
{
    f[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
    f[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
    f[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z));
    f[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
}

__device__ __forceinline__ uint32_t pack2(float2 a)
{
    const __nv_bfloat162 h = __float22bfloat162_rn(a);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint4 pack8(const float2 (&f)[4])
{
    return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}

// bf16(a + b) of two pairs: one exact sum, one rounding
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 s = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                        *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&s);
}

// the norm's weight at columns 8c .. 8c+7 (global or shared memory)
__device__ __forceinline__ void load_gamma(const void *gamma, bool f32, int c, float2 (&g)[4])
{
    if (f32) {
        const float4 a = static_cast<const float4 *>(gamma)[2 * c];
        const float4 b = static_cast<const float4 *>(gamma)[2 * c + 1];
        g[0] = make_float2(a.x, a.y), g[1] = make_float2(a.z, a.w);
        g[2] = make_float2(b.x, b.y), g[3] = make_float2(b.z, b.w);
    } else {
        unpack8(static_cast<const uint4 *>(gamma)[c], g);
    }
}

// x^(-1/2) for x > 0: the hardware's approximation and one Newton step, within
// an ulp (the correctly rounded intrinsic is 1 us slower over 8191 rows); an
// overflowed sum of squares gives 0
__device__ __forceinline__ float inv_sqrt(float x)
{
    const float r = rsqrtf(x);
    return isinf(x) ? r : fmaf(0.5f * r, fmaf(-x * r, r, 1.0f), r);
}

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// Sum over the block in a fixed order. `part` holds one slot per warp and is
// rewritten by the next call, so calls alternate between two of them: a
// thread that writes slot set b again has passed the barrier of the call on
// the other set, which every reader of b reaches after its reads.
__device__ __forceinline__ float block_sum(float v, float *part, int nwarps)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if (nwarps == 1) {
        __syncwarp();
        return v;
    }
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (int)(threadIdx.x & 31) < nwarps ? part[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A half-warp's CPT groups (chunk i of its 16 threads is group i) are reduced
// together: each exchange also halves the groups that a thread still holds, 5
// shuffles for four groups in place of 16. Group i's maximum ends in the
// LANES threads from i * LANES on, which share the division sequence of
// its scales.
template <int CPT> constexpr int LANES = CPT == 1 ? 16 : (CPT == 2 ? 8 : 4);

template <int CPT>
__device__ __forceinline__ float group_max(const float (&m)[CPT])
{
    const int lane = threadIdx.x;
    float v = m[0];
    if constexpr (CPT > 2) {
        const bool hi = lane & 8, odd = lane & 4;
        const float m3 = CPT > 3 ? m[CPT - 1] : 0.0f;
        const float a = fmaxf(hi ? m[2] : m[0], __shfl_xor_sync(0xffffffffu, hi ? m[0] : m[2], 8));
        const float b = fmaxf(hi ? m3 : m[1], __shfl_xor_sync(0xffffffffu, hi ? m[1] : m3, 8));
        v = fmaxf(odd ? b : a, __shfl_xor_sync(0xffffffffu, odd ? a : b, 4));
    } else if constexpr (CPT == 2) {
        const bool hi = lane & 8;
        v = fmaxf(hi ? m[1] : m[0], __shfl_xor_sync(0xffffffffu, hi ? m[0] : m[1], 8));
    }
#pragma unroll
    for (int o = LANES<CPT> / 2; o >= 1; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Dynamic shared memory: the ring, `slots` slots of `tensors` rows of D bf16
// values each; one "row landed" barrier per slot; gamma where it is staged.
// Rows are the CTA's own: blockIdx, blockIdx + grid, ...
//
// The rows are dealt out evenly, so every SM has to hold the same number of
// CTAs. A kernel that let the next one start on entry would see that one's
// CTAs placed unevenly, on whichever SMs drain first, so a CTA lets the
// next kernel start after its last row (on entry when it has one row only:
// there the next kernel's set-up hides behind this one), and the shared memory
// asked for leaves no room for a further CTA on the SM. In a stream of such
// calls, with an early start and without the padding in brackets: forward 8191 x
// 7168 with a residual 63.6 us (67.7), 8192 x 5120 without 23.9 (33.5). Backward
// the kernel for dgamma runs in between, and both are alike.
constexpr int MAX_SLOTS = 3;
constexpr uint32_t BAR_BYTES = (8 * MAX_SLOTS + 15) / 16 * 16;  // (gamma follows)

// Where gamma is staged in shared memory: in the backward pass, which reads it
// twice per row, and in the forward pass without a residual (8192 x 7168: 34.5
// us, from global memory 36.6). With a residual the loads from global memory
// are moved over the reduction's barrier and the space serves L1 better (63.7
// us, staged 70.2). The widest rows need the space for their second slot.
constexpr bool stages_gamma(int w, bool bwd, int tensors) { return w != WIDE && (bwd || tensors == 1); }

__device__ __forceinline__ void stage_gamma(uint8_t *dst, const void *gamma, uint32_t bytes)
{
    for (uint32_t i = threadIdx.x; i < bytes / 16; i += blockDim.x)
        reinterpret_cast<uint4 *>(dst)[i] = static_cast<const uint4 *>(gamma)[i];
}

struct Ring {
    uint32_t base, bars, slot_bytes;
    int slots;
    // of the row being worked on
    int slot = 0;
    uint32_t phase = 0;

    __device__ __forceinline__ void next()
    {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
    }
    __device__ __forceinline__ uint32_t bar() const { return bars + 8 * slot; }
};

__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// A wait that ran out (FP8FG_ETIMEOUT is recorded) does not leave the loop,
// whose barriers need every thread: the CTA's remaining rows are worked on
// with whatever the ring holds, no further copy is issued, and before the CTA
// exits thread 0 waits (bounded) for those in flight.
__device__ __forceinline__ void drain(const Ring &ring, uint32_t pending, uint32_t parity, uint64_t limit_ns)
{
    const uint64_t t0 = global_timer_ns();
    for (int s = 0; s < ring.slots; ++s)
        while (((pending >> s) & 1u) && !mbar_try_wait(ring.bars + 8 * s, (parity >> s) & 1u) &&
               global_timer_ns() - t0 < limit_ns) {
        }
}

struct NormFwd {
    const uint16_t *x, *r;
    const void *gamma;
    uint16_t *h;
    uint8_t *q;
    float *scales, *rstd;
    int64_t T, ldx, ldr, ldh, ldq, ld_s;
    int D;
    float eps, inv_d;
    bool gamma_f32, one_row;  // one_row: per CTA
    int slots;
    int *status;
    uint64_t wait_limit_ns;
    int skip_first_load;  // test hook: row 0 is never fetched, so that the wait for it runs out
};

// 7 bytes per element with a residual: 8191 x 7168 in 63.4 us, 6.5 TB/s or 0.96
// of the measured copy. Without one (3 bytes) it is bound by issue and latency,
// 110 warp instructions per 256 elements: 8192 x 7168 in 34.5 us, 0.75; with one
// CTA more per SM (at 64 registers) narrow rows gained nothing and 5120 columns
// went from 33 us to 35.
//
// The widest rows lose by what the others gain from: 4096 x 18432 with a residual
// takes 86 us (0.91), and took 80 when each chunk's group was reduced by itself
// and not the thread's groups together (group_max).
//
// The mean is the sum times 1 / D as FP32 rounds it: with the reciprocal root's
// ulp, rstd is within 3 2^-24 of the sum's root. Over 12000 rows of 7168 rstd's
// error is 4.2e-8 rms; by torch's mean and 1 / sqrt 4.6e-8.
//
// One row per CTA at a time: thread t owns chunks t, t + blockDim, ...; a
// half-warp's 16 chunks are one 128-column group (D % 128 == 0 and blockDim
// % 32 == 0 keep every group inside one half-warp).
template <int W, bool RES, bool P2>
__global__ void __launch_bounds__(max_threads(W), min_ctas(W, false)) rmsnorm_fwd_kernel(const NormFwd p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float part[2][32];
    __shared__ int abort_flag;
    constexpr int TENSORS = RES ? 2 : 1, CPT = cpt_of(W);
    const int nchunk = p.D / 8, nwarps = blockDim.x >> 5;
    const uint32_t row_bytes = 2 * (uint32_t)p.D;
    Ring ring{smem_u32(smem), smem_u32(smem) + p.slots * TENSORS * row_bytes, TENSORS * row_bytes, p.slots};
    constexpr bool STAGED = stages_gamma(W, false, TENSORS);
    uint8_t *const staged = smem + p.slots * TENSORS * row_bytes + BAR_BYTES;
    const void *const gamma = STAGED ? staged : p.gamma;
    const WaitCtl wc{&abort_flag, p.status, p.wait_limit_ns};
    uint32_t pending = 0, parity = 0;  // thread 0: slots ever filled, parity of the last fill
    auto fetch = [&](int64_t t, int slot, uint32_t par) {
        if (p.skip_first_load && t == 0)
            return;
        const uint32_t bar = ring.bars + 8 * slot, dst = ring.base + slot * ring.slot_bytes;
        mbar_arrive_expect_tx(bar, ring.slot_bytes);
        bulk_load(dst, p.x + t * p.ldx, row_bytes, bar);
        if constexpr (RES)
            bulk_load(dst + row_bytes, p.r + t * p.ldr, row_bytes, bar);
        pending |= 1u << slot;
        parity = (parity & ~(1u << slot)) | (par << slot);
    };
    if (p.one_row)
        griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.slots; ++s)
            mbar_init(ring.bars + 8 * s, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    griddep_wait();
    if (threadIdx.x == 0)
        for (int s = 0; s < p.slots && blockIdx.x + (int64_t)s * gridDim.x < p.T; ++s)
            fetch(blockIdx.x + (int64_t)s * gridDim.x, s, 0);
    if constexpr (STAGED)
        stage_gamma(staged, p.gamma, p.gamma_f32 ? 4 * p.D : 2 * p.D);
    __syncthreads();
    int b = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, b ^= 1, ring.next()) {
        mbar_wait(ring.bar(), ring.phase, wc, FP8FG_ETIMEOUT);
        const uint32_t src = ring.base + ring.slot * ring.slot_bytes;
        uint4 v[CPT];
        float2 ss2 = splat(0.0f);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            v[i] = make_uint4(0, 0, 0, 0);
            if (c < nchunk) {
                v[i] = lds16(src + 16 * c);
                if constexpr (RES) {
                    const uint4 r = lds16(src + row_bytes + 16 * c);
                    v[i] = make_uint4(add_bf16x2(v[i].x, r.x), add_bf16x2(v[i].y, r.y), add_bf16x2(v[i].z, r.z),
                                      add_bf16x2(v[i].w, r.w));
                    *reinterpret_cast<uint4 *>(p.h + t * p.ldh + 8 * c) = v[i];
                }
            }
            float2 f[4];
            unpack8(v[i], f);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                ss2 = __ffma2_rn(f[e], f[e], ss2);
        }
        const float ss = block_sum(ss2.x + ss2.y, part[b], nwarps);
        // (the sum's barrier: every thread has read the slot)
        if (threadIdx.x == 0) {
            const int64_t ahead = t + (int64_t)p.slots * gridDim.x;
            if (ahead < p.T && !*wc.abort_flag)
                fetch(ahead, ring.slot, ring.phase ^ 1);
        }
        const float rstd = inv_sqrt(fmaf(ss, p.inv_d, p.eps));
        if (threadIdx.x == 0)
            p.rstd[t] = rstd;
        const float2 rstd2 = splat(rstd);
        float2 y[CPT][4];
        float amax[CPT];
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            float2 g[4];
            unpack8(v[i], y[i]);
            load_gamma(gamma, p.gamma_f32, c < nchunk ? c : 0, g);
            amax[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[i][e] = __fmul2_rn(__fmul2_rn(y[i][e], rstd2), g[e]);
                amax[i] = fmaxf(amax[i], fmaxf(fabsf(y[i][e].x), fabsf(y[i][e].y)));
            }
        }
        const ScalePair sp = group_scale_rule<P2>(group_max<CPT>(amax));
        const int mine = (threadIdx.x & 15) / LANES<CPT>;  // this thread's group
        if ((threadIdx.x & (LANES<CPT> - 1)) == 0 && mine < CPT) {
            const int c = (threadIdx.x & ~15) + mine * blockDim.x;
            if (c < nchunk)
                p.scales[(int64_t)(c >> 4) * p.ld_s + t] = sp.s;
        }
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            const float2 inv = splat(__shfl_sync(0xffffffffu, sp.inv, (threadIdx.x & 16) + i * LANES<CPT>));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[i][e] = __fmul2_rn(y[i][e], inv);
            if (c < nchunk) {
                uint2 o;
                o.x = cvt_e4m3x2(y[i][0].x, y[i][0].y) | (cvt_e4m3x2(y[i][1].x, y[i][1].y) << 16);
                o.y = cvt_e4m3x2(y[i][2].x, y[i][2].y) | (cvt_e4m3x2(y[i][3].x, y[i][3].y) << 16);
                *reinterpret_cast<uint2 *>(p.q + t * p.ldq + 8 * c) = o;
            }
        }
    }
    if (!p.one_row)
        griddep_launch_dependents();
    if (threadIdx.x == 0 && *wc.abort_flag)
        drain(ring, pending, parity, p.wait_limit_ns);
}

// y^T in groups of 128 rows: CTA tile 128 rows x 64 columns. Warp `part` takes
// rows 16*part .. +15 and each of its threads a pair of columns (a 32-bit word
// of every row); the parts' maxima meet in shared memory and each thread writes
// its 2 x 16 codes, which pass through shared memory so that eight threads
// write whole 128-byte runs of a row of the output. 8192 x 7168: 32.9 us (3.03
// bytes per element, 0.80 of the measured copy); 39 with 16-byte stores
// straight from the registers, half a sector each.
constexpr int NT_COLS = 64;

template <bool P2>
__global__ void __launch_bounds__(256, 5) rmsnorm_t_kernel(const uint16_t *h, int64_t ldh, const float *rstd,
                                                           const void *gamma, bool gamma_f32, int64_t cols,
                                                           uint8_t *qT, int64_t ldq, float *scales, int64_t ld_s)
{
    griddep_launch_dependents();
    griddep_wait();
    __shared__ __align__(128) uint8_t buf[GROUP * NT_COLS * 2];
    __shared__ __align__(16) float s_rstd[GROUP];
    __shared__ float2 s_max[8][NT_COLS / 2];
    __shared__ __align__(8) float s_inv[NT_COLS];
    uint16_t(*const tile)[NT_COLS] = reinterpret_cast<uint16_t(*)[NT_COLS]>(buf);  // the input, then
    uint8_t(*const codes)[GROUP] = reinterpret_cast<uint8_t(*)[GROUP]>(buf);       // the columns' codes
    const int tid = threadIdx.x, cp = tid & 31, part = tid >> 5;
    const int64_t c0 = (int64_t)blockIdx.x * NT_COLS, r0 = (int64_t)blockIdx.y * GROUP;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = ld_stream(h + (r0 + 32 * i + (tid >> 3)) * ldh + c0 + (tid & 7) * 8);
    if (tid < GROUP)
        s_rstd[tid] = rstd[r0 + tid];
    float2 g;
    if (gamma_f32) {
        g = static_cast<const float2 *>(gamma)[(c0 >> 1) + cp];
    } else {
        const uint32_t w = static_cast<const uint32_t *>(gamma)[(c0 >> 1) + cp];
        g = make_float2(bf16_lo(w), bf16_hi(w));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(&tile[32 * i + (tid >> 3)][(tid & 7) * 8]) = v[i];
    __syncthreads();
    float2 y[16], m = splat(0.0f);
#pragma unroll
    for (int i4 = 0; i4 < 4; ++i4) {
        const float4 r4 = *reinterpret_cast<const float4 *>(&s_rstd[part * 16 + 4 * i4]);
        const float r[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 4 * i4 + e;
            const uint32_t w = *reinterpret_cast<const uint32_t *>(&tile[part * 16 + i][2 * cp]);
            y[i] = __fmul2_rn(__fmul2_rn(make_float2(bf16_lo(w), bf16_hi(w)), splat(r[e])), g);
            m = make_float2(fmaxf(m.x, fabsf(y[i].x)), fmaxf(m.y, fabsf(y[i].y)));
        }
    }
    s_max[part][cp] = m;
    __syncthreads();
    if (tid < NT_COLS) {
        // column tid: its group's scale pair, once per column
        const float *col = reinterpret_cast<const float *>(&s_max[0][0]) + tid;
        float amax = col[0];
#pragma unroll
        for (int p = 1; p < 8; ++p)
            amax = fmaxf(amax, col[p * NT_COLS]);
        const ScalePair sp = group_scale_rule<P2>(amax);
        s_inv[tid] = sp.inv;
        scales[(int64_t)blockIdx.y * ld_s + c0 + tid] = sp.s;
    }
    __syncthreads();
    const float2 inv = *reinterpret_cast<const float2 *>(&s_inv[2 * cp]);
    uint32_t a[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float2 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = __fmul2_rn(y[4 * k + i], inv);
        a[k] = cvt_e4m3x2(q[0].x, q[1].x) | (cvt_e4m3x2(q[2].x, q[3].x) << 16);
        b[k] = cvt_e4m3x2(q[0].y, q[1].y) | (cvt_e4m3x2(q[2].y, q[3].y) << 16);
    }
    // piece `part` of a column at slot part ^ (cp & 7): eight threads of a
    // store, and of a load, cover all banks
    const int slot = 16 * (part ^ (cp & 7));
    *reinterpret_cast<uint4 *>(&codes[2 * cp][slot]) = make_uint4(a[0], a[1], a[2], a[3]);
    *reinterpret_cast<uint4 *>(&codes[2 * cp + 1][slot]) = make_uint4(b[0], b[1], b[2], b[3]);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int c = 32 * n + (tid >> 3), pc = tid & 7;
        const uint4 w = *reinterpret_cast<const uint4 *>(&codes[c][16 * (pc ^ ((c >> 1) & 7))]);
        *reinterpret_cast<uint4 *>(qT + (c0 + c) * ldq + r0 + 16 * pc) = w;
    }
}

struct NormBwd {
    const uint16_t *dy, *h, *dres;
    const float *rstd;
    const void *gamma;
    uint16_t *dx;
    float *part;  // [gridDim.x][D]
    int64_t T, lddy, ldh, lddres, lddx;
    int D;
    float inv_d;
    bool gamma_f32, one_row;  // one_row: per CTA
    int slots;
    int *status;
    uint64_t wait_limit_ns;
    int skip_first_load;  // test hook: row 0 is never fetched, so that the wait for it runs out
};

// 8 bytes per element with dres: 8192 x 7168 in 74.9 us with the reduction of
// dgamma (about 4 us of it), 6.3 TB/s or 0.92 of the measured copy; 6 bytes
// without: 57.9 us, 0.90.
//
// The thread's columns are the same in every row, so its dgamma terms add up
// in registers and leave once, as the CTA's row of `part`.
// norm_dgamma_kernel adds those rows up in order, so the result does not
// depend on the schedule. The row's values go from the ring to registers as
// they are (bf16), so that the slot can be refilled under the second half of
// the row's work: with two slots a CTA then always has two rows in flight
// (8192 x 7168 with dres 74.9 us; 87 when the row was read from the ring
// twice and held its slot).
template <int W, bool RES>
__global__ void __launch_bounds__(max_threads(W), min_ctas(W, true)) rmsnorm_bwd_kernel(const NormBwd p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sums[2][32];
    __shared__ int abort_flag;
    constexpr int TENSORS = RES ? 3 : 2, CPT = cpt_of(W);
    const int nchunk = p.D / 8, nwarps = blockDim.x >> 5;
    const uint32_t row_bytes = 2 * (uint32_t)p.D;
    Ring ring{smem_u32(smem), smem_u32(smem) + p.slots * TENSORS * row_bytes, TENSORS * row_bytes, p.slots};
    constexpr bool STAGED = stages_gamma(W, true, TENSORS);
    uint8_t *const staged = smem + p.slots * TENSORS * row_bytes + BAR_BYTES;
    const void *const gamma = STAGED ? staged : p.gamma;
    const WaitCtl wc{&abort_flag, p.status, p.wait_limit_ns};
    uint32_t pending = 0, parity = 0;
    auto fetch = [&](int64_t t, int slot, uint32_t par) {
        if (p.skip_first_load && t == 0)
            return;
        const uint32_t bar = ring.bars + 8 * slot, dst = ring.base + slot * ring.slot_bytes;
        mbar_arrive_expect_tx(bar, ring.slot_bytes);
        bulk_load(dst, p.dy + t * p.lddy, row_bytes, bar);
        bulk_load(dst + row_bytes, p.h + t * p.ldh, row_bytes, bar);
        if constexpr (RES)
            bulk_load(dst + 2 * row_bytes, p.dres + t * p.lddres, row_bytes, bar);
        pending |= 1u << slot;
        parity = (parity & ~(1u << slot)) | (par << slot);
    };
    if (p.one_row)
        griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.slots; ++s)
            mbar_init(ring.bars + 8 * s, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    griddep_wait();
    // (read ahead of the ring's fill, but for the widest rows, whose kernel would
    // spill over it: 110 us in place of 86 for 3000 x 18432 with dres)
    float rstd = 0.0f;
    if (W != WIDE && blockIdx.x < p.T)
        rstd = p.rstd[blockIdx.x];
    if (threadIdx.x == 0)
        for (int s = 0; s < p.slots && blockIdx.x + (int64_t)s * gridDim.x < p.T; ++s)
            fetch(blockIdx.x + (int64_t)s * gridDim.x, s, 0);
    if constexpr (STAGED)
        stage_gamma(staged, p.gamma, p.gamma_f32 ? 4 * p.D : 2 * p.D);
    __syncthreads();
    float2 dg[CPT][4];
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            dg[i][e] = splat(0.0f);
    int b = 0;
    if (W == WIDE && blockIdx.x < p.T)
        rstd = p.rstd[blockIdx.x];
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, b ^= 1, ring.next()) {
        const float rstd_next = t + gridDim.x < p.T ? p.rstd[t + gridDim.x] : 0.0f;
        mbar_wait(ring.bar(), ring.phase, wc, FP8FG_ETIMEOUT);
        const uint32_t src = ring.base + ring.slot * ring.slot_bytes;
        uint4 dv[CPT], hv[CPT], rv[CPT];
        float2 dot2 = splat(0.0f);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < nchunk) {
                dv[i] = lds16(src + 16 * c);
                hv[i] = lds16(src + row_bytes + 16 * c);
                if constexpr (RES)
                    rv[i] = lds16(src + 2 * row_bytes + 16 * c);
                float2 d[4], h[4], g[4];
                unpack8(dv[i], d);
                unpack8(hv[i], h);
                load_gamma(gamma, p.gamma_f32, c, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 dh = __fmul2_rn(d[e], h[e]);
                    dg[i][e] = __ffma2_rn(dh, splat(rstd), dg[i][e]);
                    dot2 = __ffma2_rn(dh, g[e], dot2);
                }
            }
        }
        const float dot = block_sum(dot2.x + dot2.y, sums[b], nwarps);
        // (the sum's barrier: every thread has read the slot)
        if (threadIdx.x == 0) {
            const int64_t ahead = t + (int64_t)p.slots * gridDim.x;
            if (ahead < p.T && !*wc.abort_flag)
                fetch(ahead, ring.slot, ring.phase ^ 1);
        }
        const float k = dot * p.inv_d * rstd * rstd;  // dx = rstd * (a - h k)
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nchunk)
                continue;
            float2 d[4], h[4], g[4];
            unpack8(dv[i], d);
            unpack8(hv[i], h);
            load_gamma(gamma, p.gamma_f32, c, g);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                d[e] = __ffma2_rn(h[e], splat(-k), __fmul2_rn(d[e], g[e]));
            if constexpr (RES) {
                unpack8(rv[i], h);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    d[e] = __ffma2_rn(d[e], splat(rstd), h[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    d[e] = __fmul2_rn(d[e], splat(rstd));
            }
            *reinterpret_cast<uint4 *>(p.dx + t * p.lddx + 8 * c) = pack8(d);
        }
        rstd = rstd_next;
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nchunk) {
            float4 *o = reinterpret_cast<float4 *>(p.part + (int64_t)blockIdx.x * p.D + 8 * c);
            o[0] = make_float4(dg[i][0].x, dg[i][0].y, dg[i][1].x, dg[i][1].y);
            o[1] = make_float4(dg[i][2].x, dg[i][2].y, dg[i][3].x, dg[i][3].y);
        }
    }
    if (!p.one_row)
        griddep_launch_dependents();
    if (threadIdx.x == 0 && *wc.abort_flag)
        drain(ring, pending, parity, p.wait_limit_ns);
}

// dgamma[c] = sum over the rows of part: 32 columns per CTA, 64 slices of the
// rows side by side (slice s adds rows s, s + 64, ...), then the slices in
// order, eight by eight.
constexpr int DG_SLICES = 64;
constexpr int DG_THREADS = 8 * DG_SLICES;

__global__ void __launch_bounds__(DG_THREADS) norm_dgamma_kernel(const float4 *part, int rows, int D,
                                                                 float *dgamma)
{
    griddep_wait();
    __shared__ float4 s[DG_SLICES][8];
    __shared__ float s8[8][32];
    const int c4 = threadIdx.x & 7, slice = threadIdx.x >> 3;
    const float4 *col = part + blockIdx.x * 8 + c4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int r = slice; r < rows; r += DG_SLICES) {
        const float4 a = col[(int64_t)r * (D / 4)];
        v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
    }
    s[slice][c4] = v;
    __syncthreads();
    const float *f = reinterpret_cast<const float *>(&s[0][0]);
    const int c = threadIdx.x & 31, oct = threadIdx.x >> 5;
    if (oct < 8) {
        float a = f[(8 * oct) * 32 + c];
#pragma unroll
        for (int i = 1; i < 8; ++i)
            a += f[(8 * oct + i) * 32 + c];
        s8[oct][c] = a;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        float a = s8[0][c];
#pragma unroll
        for (int i = 1; i < 8; ++i)
            a += s8[i][c];
        dgamma[blockIdx.x * 32 + c] = a;
    }
    griddep_launch_dependents();
}

// Width and threads of a row of D columns: up to four chunks per thread,
// which share the row's reduction and the scales' division sequence.
struct RowShape {
    int width, threads;
};

RowShape row_shape(int64_t D)
{
    const int chunks = (int)(D / 8);
    const int width = chunks <= 32 ? ONE : (chunks <= 64 ? TWO : (chunks <= 4 * 256 ? FOUR : WIDE));
    return {width, (chunks + 32 * cpt_of(width) - 1) / (32 * cpt_of(width)) * 32};
}

// CTAs per SM, slots of a CTA's ring and shared memory for rows of `tensors`
// tensors.
struct RingShape {
    int per_sm, slots;
    size_t smem;
};

// Two slots: a row's reduction runs under the next row's copies. Forward: as
// many CTAs as fit (more slots for fewer CTAs were slower at every width from
// 256 to 18432). Backward: each CTA adds a row to dgamma's partial sums, so the
// fewest CTAs with 96 KB in flight (28672 x 2048 with dres: 4 CTAs 75 us, 6
// 78; 2 slots or 4 the same), but two, since one CTA leaves the memory idle at
// its barriers; where two do not fit, one with three slots (8192 columns with
// dres: 76 us, with two slots 79). The widest rows read gamma through L1, whose
// space a third slot or padding would take (12288 columns with dres: 88 us,
// with three slots 104).
RingShape ring_shape(int64_t D, int tensors, bool gamma_f32, bool bwd)
{
    const RowShape rs = row_shape(D);
    const int64_t gamma_bytes = stages_gamma(rs.width, bwd, tensors) ? (gamma_f32 ? 4 * D : 2 * D) : 0;
    constexpr int64_t SM_BYTES = 226 * 1024;  // of an SM
    constexpr int64_t OWN = 1024 + 512;       // of a CTA beside its dynamic part, 1 KB of it the system's
    constexpr int64_t IN_FLIGHT = 96 * 1024;
    const int64_t slot = 2 * D * tensors, fixed = gamma_bytes + BAR_BYTES;
    int per_sm = max_threads(rs.width) * min_ctas(rs.width, bwd) / rs.threads;
    if (bwd) {
        const int64_t want = std::max<int64_t>(2, (IN_FLIGHT + 2 * slot - 1) / (2 * slot));
        per_sm = (int)std::min<int64_t>(per_sm, want);
    }
    while (per_sm > 1 && (2 * slot + fixed + OWN) * per_sm > SM_BYTES)
        --per_sm;
    const int slots = per_sm == 1 && rs.width != WIDE && 3 * slot + fixed + OWN <= SM_BYTES ? 3 : 2;
    const int64_t smem = slots * slot + fixed, room = (SM_BYTES / per_sm - OWN) / 128 * 128;
    return {per_sm, slots, (size_t)(rs.width != WIDE && smem < room ? room : smem)};
}

int ring_grid(int64_t T, const RingShape &r)
{
    const int64_t cap = (int64_t)sm_count() * r.per_sm;
    return (int)(T < cap ? T : (cap > 0 ? cap : 1));
}

// The backward pass of few rows takes fewer CTAs than fit, since dgamma's second
// kernel adds up a row from each: about two rows each, and four CTAs per SM
// until every one of a full grid has four (us in a graph, as many CTAs as fit in
// brackets: 1031 x 2048 without dres 8.5 (10.4), 300 x 7168 with dres 9.1
// (10.1), 2048 x 512 with dres 7.4 (9.3)).
int bwd_grid(int64_t T, RingShape r)
{
    const int64_t sms = sm_count() > 0 ? sm_count() : 1;
    int64_t per_sm = (T + 2 * sms - 1) / (2 * sms);
    if (T < 4 * sms * r.per_sm)
        per_sm = std::min<int64_t>(per_sm, 4);
    r.per_sm = (int)std::min<int64_t>(per_sm, r.per_sm);
    return ring_grid(T, r);
}

// (every instantiation may take all of a CTA's shared memory)
template <auto K, typename P>
int launch_ring(const P &p, int grid, int threads, size_t smem, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(K, 226 * 1024, done))
        return FP8FG_ECUDA;
    return launch_pss(K, dim3((unsigned)grid), threads, smem, s, p);
}

template <int W>
int launch_fwd(const NormFwd &p, int grid, int threads, size_t smem, bool p2, cudaStream_t s)
{
    if (p.r)
        return p2 ? launch_ring<rmsnorm_fwd_kernel<W, true, true>>(p, grid, threads, smem, s)
                  : launch_ring<rmsnorm_fwd_kernel<W, true, false>>(p, grid, threads, smem, s);
    return p2 ? launch_ring<rmsnorm_fwd_kernel<W, false, true>>(p, grid, threads, smem, s)
              : launch_ring<rmsnorm_fwd_kernel<W, false, false>>(p, grid, threads, smem, s);
}

template <int W>
int launch_bwd(const NormBwd &p, int grid, int threads, size_t smem, cudaStream_t s)
{
    return p.dres ? launch_ring<rmsnorm_bwd_kernel<W, true>>(p, grid, threads, smem, s)
                  : launch_ring<rmsnorm_bwd_kernel<W, false>>(p, grid, threads, smem, s);
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
    p.inv_d = 1.0f / (float)D;
    p.eps = eps;
    p.gamma_f32 = gamma_kind == FP8FG_OUT_F32;
    const RowShape rs = row_shape(D);
    const RingShape ring = ring_shape(D, residual ? 2 : 1, p.gamma_f32, false);
    const int grid = ring_grid(T, ring);
    p.slots = ring.slots;
    p.one_row = T <= grid;
    p.status = status_word_ptr();
    p.wait_limit_ns = wait_limit_ns();
    p.skip_first_load = take_skip_first_load() ? 1 : 0;
    if (!p.status)
        return FP8FG_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (rs.width) {
    case ONE: return launch_fwd<ONE>(p, grid, rs.threads, ring.smem, pow2 != 0, s);
    case TWO: return launch_fwd<TWO>(p, grid, rs.threads, ring.smem, pow2 != 0, s);
    case FOUR: return launch_fwd<FOUR>(p, grid, rs.threads, ring.smem, pow2 != 0, s);
    default: return launch_fwd<WIDE>(p, grid, rs.threads, ring.smem, pow2 != 0, s);
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
    auto k = pow2 ? rmsnorm_t_kernel<true> : rmsnorm_t_kernel<false>;
    return launch_pss(k, grid, 256, 0, s, hp, ldh, rstd, gamma, f32, D, qT, ldqT, scalesT, ld_sT);
}

extern "C" int64_t fp8_rmsnorm_bwd_workspace(int64_t T, int64_t D)
{
    if (T <= 0 || D <= 0 || !norm_width_ok(D))
        return 0;
    int grid = 0;
    for (int tensors = 2; tensors <= 3; ++tensors)
        for (int f32 = 0; f32 < 2; ++f32)
            grid = std::max(grid, bwd_grid(T, ring_shape(D, tensors, f32 != 0, true)));
    return (int64_t)grid * D * 4;
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
    const RingShape ring = ring_shape(D, dres ? 3 : 2, gamma_kind == FP8FG_OUT_F32, true);
    const int grid = bwd_grid(T, ring);
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
    p.inv_d = 1.0f / (float)D;
    p.gamma_f32 = gamma_kind == FP8FG_OUT_F32;
    const RowShape rs = row_shape(D);
    p.slots = ring.slots;
    p.one_row = T <= grid;
    p.status = status_word_ptr();
    p.wait_limit_ns = wait_limit_ns();
    p.skip_first_load = take_skip_first_load() ? 1 : 0;
    if (!p.status)
        return FP8FG_ECUDA;
    int rc;
    switch (rs.width) {
    case ONE: rc = launch_bwd<ONE>(p, grid, rs.threads, ring.smem, s); break;
    case TWO: rc = launch_bwd<TWO>(p, grid, rs.threads, ring.smem, s); break;
    case FOUR: rc = launch_bwd<FOUR>(p, grid, rs.threads, ring.smem, s); break;
    default: rc = launch_bwd<WIDE>(p, grid, rs.threads, ring.smem, s); break;
    }
    if (rc != FP8FG_OK)
        return rc;
    return launch_pss(norm_dgamma_kernel, dim3((unsigned)(D / 32)), DG_THREADS, 0, s,
                      reinterpret_cast<const float4 *>(p.part), grid, (int)D, dgamma);
}
