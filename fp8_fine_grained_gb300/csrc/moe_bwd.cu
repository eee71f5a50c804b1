// Backward pass of the MoE combine out[t] = sum_j w[t][j] y[dest[t][j]]:
//     dy[dest[t][j]] = w[t][j] dout[t],   dw[t][j] = sum_n dout[t][n] y[dest[t][j]][n].
//
// A memory stream: k rows of y read and k rows of dy written per token, and dout
// once. One warp takes one slot (t, j): it reads the row of y and the token's
// dout, 8 columns to a lane, folds the product into eight FP32 sums a lane and
// stores dy's columns as it goes. The eight warps of a CTA take slots next to each
// other, so that a token's dout comes from L1 for all but the first of them. Where
// there are fewer slots than warps to run, 2, 4 or 8 warps share one, each a run of
// its columns, and join their parts of dw in shared memory.
//
// A row that several slots name (a forward call may) has the sum of their gradients,
// in slot order. Up to 1024 slots each warp looks for its row among all of them; where
// it is named again, the first of its slots adds them up. More slots find that out
// without atomics: every slot writes its number into claims[row], and a second kernel,
// started as the first ends, looks whether each slot still stands there. Where it does
// not, one warp adds up the row's slots and writes the row again. With no such row (an
// expert order has none) the second kernel reads 8 bytes a slot. (Looking against
// claims, 7168 and 2048 columns: 1024 slots 9.2 against 10.2 and 3.7 against 4.3 us, 2048
// slots 15.6 against 16.7 and 8.0 against 7.6, 4096 slots 33.0 against 23.4 and 16.7
// against 9.7.) A shared row is slow: one warp goes through all of dest for every 256
// columns (8192 slots of 7168 columns: 845 us with one such row, 42 without).
//
// Measured: 4096 tokens x 8 rows of 7168 columns 153 us (998 MB, 0.96 of HBM copy), with an
// FP32 dout 173 us (1057 MB, 0.90).
#include <cuda_bf16.h>

#include "host_common.h"
#include "ptx.cuh"

#include <type_traits>

namespace fp8fg {
namespace {

constexpr int BWD_THREADS = 256;
constexpr int BWD_WARPS = BWD_THREADS / 32;
constexpr int BWD_MAX_K = 16;
constexpr int BWD_UNROLL = 4;
constexpr int64_t BWD_FEW = 1024;  // slots that a warp looks through
constexpr unsigned ALL = 0xFFFFFFFFu;

struct CombineBwdArgs {
    const void *dout;
    int64_t lddo;
    const uint16_t *y;
    int64_t ldy, y_rows;
    const int32_t *dest;
    const float *w;
    int64_t slots;
    int k;
    int64_t chunks;  // 8 columns each
    uint16_t *dy;
    int64_t lddy;
    float *dw;
    int32_t *claims;
    int *status;
};

struct Eight {
    float v[8];
};

__device__ __forceinline__ Eight unpack(uint4 u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    Eight r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.v[2 * i] = bf16_lo(w[i]);
        r.v[2 * i + 1] = bf16_hi(w[i]);
    }
    return r;
}

__device__ __forceinline__ uint4 pack(const Eight &x)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.v[2 * i], x.v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// columns 8 c .. 8 c + 7 of dout's row t
template <bool F32>
__device__ __forceinline__ Eight load_dout(const CombineBwdArgs &a, int64_t t, int64_t c)
{
    if constexpr (F32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.dout) + t * a.lddo) + 2 * c;
        const float4 lo = p[0], hi = p[1];
        return {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
    } else {
        return unpack(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.dout) + t * a.lddo)[c]);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        v += __shfl_xor_sync(ALL, v, d);
    return v;
}

// dy's row r, columns 8 begin .. 8 end - 1: the sum over all slots that name it, by one warp.
template <bool F32>
__device__ __forceinline__ void add_up_row(const CombineBwdArgs &a, int64_t r, int64_t begin, int64_t end)
{
    const int lane = (int)lane_id();
    for (int64_t c = begin + lane; c - lane < end; c += 32) {
        Eight sum = {};
        for (int64_t i0 = 0; i0 < a.slots; i0 += 32) {
            unsigned hit = __ballot_sync(ALL, i0 + lane < a.slots && a.dest[i0 + lane] == r);
            for (; hit; hit &= hit - 1) {
                const int64_t i = i0 + __ffs(hit) - 1;
                if (c < end) {
                    const Eight d = load_dout<F32>(a, i / a.k, c);
                    const float w = a.w[i];
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        sum.v[q] = fmaf(w, d.v[q], sum.v[q]);
                }
            }
        }
        if (c < end)
            reinterpret_cast<uint4 *>(a.dy + r * a.lddy)[c] = pack(sum);
    }
}

template <bool F32, int SHARE, bool FEW>
__global__ void __launch_bounds__(BWD_THREADS) combine_bwd_kernel(const CombineBwdArgs a)
{
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float parts[SHARE > 1 ? BWD_WARPS : 1];
    constexpr int SLOTS = BWD_WARPS / SHARE;  // of a CTA at a time
    const int lane = (int)lane_id(), warp = threadIdx.x >> 5, part = warp % SHARE;
    // this warp's columns of a slot
    const int64_t each = (a.chunks + SHARE - 1) / SHARE, begin = min(part * each, a.chunks), end = min(begin + each, a.chunks);
    const int64_t stride = (int64_t)gridDim.x * SLOTS;
    for (int64_t s0 = (int64_t)blockIdx.x * SLOTS; s0 < a.slots; s0 += stride) {
        const int64_t s = s0 + warp / SHARE;
        const int64_t row = s < a.slots ? a.dest[s] : -1;
        float sum = 0.0f;
        if (row < 0 || row >= a.y_rows) {
            if (lane == 0 && part == 0 && s < a.slots) {
                if (row >= 0)
                    atomicCAS(a.status, 0, FP8FG_EDEVICE);
                a.dw[s] = 0.0f;
            }
        } else {
            const int64_t t = s / a.k;
            const float w = a.w[s];
            bool alone = true, first = true;
            if constexpr (FEW) {
                const int slots = (int)a.slots, mine = (int)row;
                int named = 0;
#pragma unroll 8
                for (int i = lane; i < slots; i += 32)
                    named += a.dest[i] == mine;
                alone = __reduce_add_sync(ALL, named) == 1;
                if (!alone)
                    for (int i = 0; i < (int)s; ++i)
                        first = first && a.dest[i] != mine;
            }
            const uint4 *y = reinterpret_cast<const uint4 *>(a.y + row * a.ldy);
            uint4 *dy = reinterpret_cast<uint4 *>(a.dy + row * a.lddy);
            float acc[8] = {};
            auto fold = [&](int64_t c, const Eight &d, const uint4 &u) {
                const Eight r = unpack(u);
                Eight g;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[i] = fmaf(d.v[i], r.v[i], acc[i]);
                    g.v[i] = w * d.v[i];
                }
                if (alone)
                    dy[c] = pack(g);
            };
            int64_t c = begin + lane;
            for (; c + 32 * (BWD_UNROLL - 1) < end; c += 32 * BWD_UNROLL) {
                uint4 u[BWD_UNROLL];
                Eight d[BWD_UNROLL];
#pragma unroll
                for (int i = 0; i < BWD_UNROLL; ++i)
                    u[i] = y[c + 32 * i];
#pragma unroll
                for (int i = 0; i < BWD_UNROLL; ++i)
                    d[i] = load_dout<F32>(a, t, c + 32 * i);
#pragma unroll
                for (int i = 0; i < BWD_UNROLL; ++i)
                    fold(c + 32 * i, d[i], u[i]);
            }
            if constexpr (SHARE == 1) {
                for (; c < end; c += 32)
                    fold(c, load_dout<F32>(a, t, c), y[c]);
            } else {  // (the last columns together too: they are most)
                uint4 u[BWD_UNROLL - 1];
                Eight d[BWD_UNROLL - 1];
#pragma unroll
                for (int i = 0; i < BWD_UNROLL - 1; ++i)
                    if (c + 32 * i < end) {
                        u[i] = y[c + 32 * i];
                        d[i] = load_dout<F32>(a, t, c + 32 * i);
                    }
#pragma unroll
                for (int i = 0; i < BWD_UNROLL - 1; ++i)
                    if (c + 32 * i < end)
                        fold(c + 32 * i, d[i], u[i]);
            }
            sum = warp_sum(((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7])));
            if (FEW && !alone && first)
                add_up_row<F32>(a, row, begin, end);
            if (lane == 0 && part == 0) {
                if (!FEW)
                    a.claims[row] = (int32_t)s;
                if (SHARE == 1)
                    a.dw[s] = sum;
            }
        }
        if constexpr (SHARE > 1) {
            if (lane == 0)
                parts[warp] = sum;
            __syncthreads();
            if (lane == 0 && part == 0 && row >= 0 && row < a.y_rows) {
                for (int i = 1; i < SHARE; ++i)
                    sum += parts[warp + i];
                a.dw[s] = sum;
            }
            __syncthreads();
        }
    }
}

constexpr int32_t MENDED = -2;

template <bool F32>
__global__ void __launch_bounds__(BWD_THREADS) combine_bwd_shared_rows_kernel(const CombineBwdArgs a)
{
    griddep_launch_dependents();
    griddep_wait();
    const int lane = (int)lane_id();
    const int64_t stride = (int64_t)gridDim.x * BWD_THREADS;
    for (int64_t s0 = (int64_t)blockIdx.x * BWD_THREADS + (threadIdx.x & ~31u); s0 < a.slots; s0 += stride) {
        const int64_t s = s0 + lane;
        int32_t row = s < a.slots ? a.dest[s] : -1;
        row = row >= a.y_rows ? -1 : row;
        // (the first that finds the row shared mends it; a slot that then reads
        // MENDED finds it taken)
        bool mend = row >= 0 && *(volatile int32_t *)(a.claims + row) != (int32_t)s;
        mend = mend && atomicExch(a.claims + row, MENDED) != MENDED;
        for (unsigned rest = __ballot_sync(ALL, mend); rest; rest &= rest - 1) {
            const int32_t r = __shfl_sync(ALL, row, __ffs(rest) - 1);
            add_up_row<F32>(a, r, 0, a.chunks);
        }
    }
}

template <bool F32>
int launch(const CombineBwdArgs &a, cudaStream_t s)
{
    const int64_t sms = sm_count() > 0 ? sm_count() : 1;
    // warps to a slot: until there are eight warps an SM, or a warp's columns are one round
    int share = 1;
    while (share < BWD_WARPS && a.slots * share < 8 * sms && a.chunks > 32 * share)
        share *= 2;
    const int64_t per = BWD_WARPS / share, want = (a.slots + per - 1) / per, cap = sms * 8 * 4;
    const dim3 grid((unsigned)(want < cap ? want : cap));
    const bool few = a.slots <= BWD_FEW;
    auto with = [&](auto sh) {
        constexpr int SHARE = decltype(sh)::value;
        return few ? launch_pss(combine_bwd_kernel<F32, SHARE, true>, grid, BWD_THREADS, 0, s, a)
                   : launch_pss(combine_bwd_kernel<F32, SHARE, false>, grid, BWD_THREADS, 0, s, a);
    };
    const int rc = share == 1   ? with(std::integral_constant<int, 1>())
                   : share == 2 ? with(std::integral_constant<int, 2>())
                   : share == 4 ? with(std::integral_constant<int, 4>())
                                : with(std::integral_constant<int, 8>());
    if (rc != FP8FG_OK || few)
        return rc;
    const int64_t looks = (a.slots + BWD_THREADS - 1) / BWD_THREADS;
    return launch_pss(combine_bwd_shared_rows_kernel<F32>, dim3((unsigned)(looks < cap ? looks : cap)), BWD_THREADS, 0, s,
                      a);
}

bool aligned4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

}  // namespace
}  // namespace fp8fg

using namespace fp8fg;

extern "C" int64_t fp8_moe_combine_bwd_workspace(int64_t T, int k, int64_t y_rows)
{
    return T > 0 && k > 0 && T > BWD_FEW / k && y_rows > 0 && y_rows < (1ll << 31) ? 4 * y_rows : 0;
}

extern "C" int fp8_moe_combine_bwd(const void *dout, int dout_kind, int64_t lddo, const void *y, int64_t ldy,
                                   int64_t y_rows, const int32_t *dest, const float *w, int64_t T, int k, int64_t N,
                                   void *dy, int64_t lddy, float *dw, void *workspace, int64_t workspace_bytes,
                                   void *stream)
{
    if (dout_kind != FP8FG_OUT_F32 && dout_kind != FP8FG_OUT_BF16)
        return FP8FG_EINVAL;
    if (T < 0 || N < 0 || y_rows < 0 || y_rows >= (1ll << 31) || k < 1 || k > BWD_MAX_K || T >= (1ll << 31) / k ||
        N % 8 != 0 || N >= (1ll << 31) || lddo < N || ldy < N || lddy < N)
        return FP8FG_EINVAL;
    if (T == 0)
        return FP8FG_OK;
    if (!dest || !w || !dw || (N > 0 && !dout) || (N > 0 && y_rows > 0 && (!y || !dy)))
        return FP8FG_EINVAL;
    const int64_t need = fp8_moe_combine_bwd_workspace(T, k, y_rows);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return FP8FG_EINVAL;
    const int64_t esz = dout_kind == FP8FG_OUT_F32 ? 4 : 2;
    if (!aligned16(dout) || !aligned16(y) || !aligned16(dy) || (lddo * esz) % 16 != 0 || ldy % 8 != 0 ||
        lddy % 8 != 0 || !aligned4(dest) || !aligned4(w) || !aligned4(dw) || !aligned4(workspace))
        return FP8FG_EALIGN;
    if (!device_supported())
        return FP8FG_EUNSUPPORTED;
    const CombineBwdArgs a = {dout, lddo, static_cast<const uint16_t *>(y), ldy, y_rows, dest, w, T * k, k, N / 8,
                              static_cast<uint16_t *>(dy), lddy, dw, static_cast<int32_t *>(workspace),
                              status_word_ptr()};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dout_kind == FP8FG_OUT_F32 ? launch<true>(a, s) : launch<false>(a, s);
}
