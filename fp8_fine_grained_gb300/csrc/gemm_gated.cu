// Gated feed-forward of E4M3 operands: both projections, the activation and
// the product in one kernel, with an E4M3 output in 1x128 groups.
//
//   G = X Wg^T, U = X Wu^T      (promoted block-scaled products, W = [Wg; Wu])
//   h = silu(G) * U             FP32, quantised by the group rule
//
// Three tilings, chosen by an estimate of their times (choose below):
//   persistent  the 128-row tiles of the block-scaled GEMM (gemm.cu, mode
//               GATED), for calls with enough tiles to fill the SMs;
//   ROWS        one tile of 128 tokens x 128 columns of h per cluster, the
//               contraction split over the cluster's S CTAs;
//   FEW         the same for at most 32 tokens, with the weight on the MMA's
//               128-row side and the tokens on its N side, so that no more
//               than 32 token rows are multiplied.
// A tile's weight is 128 gate rows and 128 up rows. With few rows the kernel
// is a stream of the weights, which one SM cannot draw at more than about 80
// GB/s: only the split gives a narrow weight (2048 columns are 16 tiles) enough
// CTAs. One token through 7168 x 18432 (144 tiles, no split) takes 43 us, 0.90
// of the copy bandwidth; 24 tokens through 7168 x 2048 take 29.0, 17.0, 11.5
// and 10.5 us with S = 1, 2, 4 and 6.
//
// The cluster tilings (12 warps):
//   warp 0      TMA producer: per 128-wide contraction block the 32 KB of
//               weight rows, the tokens' codes and their scales, and the two
//               weight-block scales by 4-byte cp.async, into a ring of stages.
//   warp 1      MMA issuer into one of BUFS partial buffers in TMEM.
//   warps 4..11 promotion, acc = fma(P, sX * sW, acc) in FP32 per block. FEW:
//               a thread owns one gate row (warps 4..7) or up row (8..11) and
//               the 32 tokens; ROWS: one token and the 128 gate or up columns.
//               Then the sums go to shared memory as [token][256]; after a
//               cluster barrier CTA r takes tokens r, r + S, ...: a warp per
//               token adds the S CTAs' sums in rank order (distributed shared
//               memory), applies the gate and quantises the token's 128
//               columns, one scale group, inside the warp.
// The order of every sum is fixed. Every wait on an mbarrier is bounded; a
// CTA that gave up still takes part in the two cluster barriers (every warp
// passes both inside its own role, since after setmaxnreg the roles' registers
// differ), and its garbage sums reach no address outside the outputs.
#include <cuda_bf16.h>

#include <atomic>

#include "gate.cuh"
#include "gated_args.h"
#include "group_rule.cuh"
#include "host_common.h"
#include "per_device.h"
#include "ptx.cuh"
#include "tensor_map.h"

namespace fp8fg {
namespace {

constexpr int BK = 128;
constexpr int BI = 128;                         // columns of h per tile
constexpr int MMA_K = 32;
constexpr int PROMO_WARPS = 8;
constexpr int PROMO_WARP0 = 4;
constexpr int THREADS = (PROMO_WARP0 + PROMO_WARPS) * 32;
constexpr int MAX_SPLIT = 8;                    // the portable cluster size
constexpr uint32_t W_BYTES = 2 * BI * BK;       // gate rows, then up rows

enum Tiling { FEW = 0, ROWS = 1 };

template <int TILING> struct Shape {
    static constexpr int TOK = TILING == FEW ? 32 : 128;      // tokens of a tile
    static constexpr uint32_t X_BYTES = TOK * BK;
    static constexpr int STAGES = TILING == FEW ? 6 : 4;
    static constexpr int BUFS = TILING == FEW ? 4 : 2;        // TMEM partial buffers
    static constexpr uint32_t BUF_COLS = TILING == FEW ? 2 * TOK : 2 * BI;
    static constexpr uint32_t TMEM_COLS = BUFS * BUF_COLS;
    static constexpr uint32_t SLOT = (4 * TOK + 16 + 127) / 128 * 128;  // token scales, two weight scales
    // the sums, [token][PITCH], reuse the idle ring: gate, then up columns. In
    // ROWS a warp writes 32 rows at one column, in FEW 32 columns of a row
    static constexpr uint32_t PITCH = TILING == FEW ? 2 * BI : 2 * BI + 4;
    static constexpr uint32_t w_off = 0;
    static constexpr uint32_t x_off = STAGES * W_BYTES;
    static constexpr uint32_t slot_off = x_off + STAGES * X_BYTES;
    static constexpr uint32_t full_off = slot_off + STAGES * SLOT;
    static constexpr uint32_t empty_off = full_off + 8 * STAGES;
    static constexpr uint32_t tempty_off = empty_off + 8 * STAGES;  // per stage (a buffer's block's stage)
    static constexpr uint32_t tfull_off = tempty_off + 8 * STAGES;
    static constexpr uint32_t tmem_ptr_off = tfull_off + 8 * BUFS;
    static constexpr uint32_t abort_off = tmem_ptr_off + 4;
    static constexpr uint32_t total = abort_off + 4;
    static_assert(TOK * PITCH * 4 <= slot_off, "sums inside the ring");
    static_assert(total <= 232448, "shared memory budget");
    static_assert(BUFS <= STAGES && TMEM_COLS <= 512, "buffers");
    // ROWS: 128 sums per thread need more registers than an even share;
    // setmaxnreg moves them from warps 0..3 to the promotion warps (the
    // launch's total bounds it)
    static constexpr bool REBALANCE = TILING == ROWS;
};
constexpr int LOW = 56, HIGH = 224;  // registers per thread after the move
constexpr int LAUNCH_MIN = (128 * LOW + PROMO_WARPS * 32 * HIGH + THREADS - 1) / THREADS;

struct ClusterParams {
    int64_t M, I, K;
    const float *sw;
    uint8_t *h;
    int64_t ldh;
    float *sh;
    int64_t ld_sh;
    uint16_t *gu;
    int64_t ld_gu;
    int token_tiles, split, pow2;
    int *status;
    uint64_t wait_limit_ns;
    int skip_first_load;
};

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 16 bytes at `addr` (an address of this CTA's shared memory) in CTA `rank`
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t rank)
{
    float4 v;
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// Tokens rank + S * (warp + 8 i) of the tile: the S CTAs' sums in rank order,
// the gate and the codes. NT tokens of a warp share one division sequence for
// their scales (lane n on token n); with one per token the divisions are a
// third of this part's instructions. ROWS, 333 tokens through 7168 x 2048: NT
// = 8 19.4 us, NT = 1 19.8; FEW has a token or two per warp and takes NT = 1.
template <uint32_t PITCH, int NT>
__device__ __forceinline__ void finish_tokens(const ClusterParams &p, uint32_t sbase, int rank, int warp, int lane,
                                              int nrows, int64_t m0, int64_t i0)
{
    const int step = p.split * PROMO_WARPS;  // between a warp's tokens
    const int64_t col = i0 + 4 * lane;
    for (int j0 = rank + p.split * warp; j0 < nrows; j0 += NT * step) {
        float v[NT][4], mine = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int j = j0 + n * step;
            if (j >= nrows)
                break;
            const uint32_t at = sbase + ((uint32_t)j * PITCH + 4 * lane) * 4;
            float4 g = ld_cluster(at, 0), u = ld_cluster(at + BI * 4, 0);
            for (int r = 1; r < p.split; ++r) {
                const float4 a = ld_cluster(at, r), b = ld_cluster(at + BI * 4, r);
                g.x += a.x, g.y += a.y, g.z += a.z, g.w += a.w;
                u.x += b.x, u.y += b.y, u.z += b.z, u.w += b.w;
            }
            if (p.gu) {
                const __nv_bfloat162 g0 = __floats2bfloat162_rn(g.x, g.y), g1 = __floats2bfloat162_rn(g.z, g.w);
                const __nv_bfloat162 u0 = __floats2bfloat162_rn(u.x, u.y), u1 = __floats2bfloat162_rn(u.z, u.w);
                uint2 o, q;
                o.x = *reinterpret_cast<const uint32_t *>(&g0), o.y = *reinterpret_cast<const uint32_t *>(&g1);
                q.x = *reinterpret_cast<const uint32_t *>(&u0), q.y = *reinterpret_cast<const uint32_t *>(&u1);
                *reinterpret_cast<uint2 *>(p.gu + (m0 + j) * p.ld_gu + col) = o;
                *reinterpret_cast<uint2 *>(p.gu + (m0 + j) * p.ld_gu + p.I + col) = q;
            }
            const float2 lo = silu_mul2(make_float2(g.x, g.y), make_float2(u.x, u.y));
            const float2 hi = silu_mul2(make_float2(g.z, g.w), make_float2(u.z, u.w));
            v[n][0] = lo.x, v[n][1] = lo.y, v[n][2] = hi.x, v[n][3] = hi.y;
            const float m = fmaxf(fmaxf(fabsf(v[n][0]), fabsf(v[n][1])), fmaxf(fabsf(v[n][2]), fabsf(v[n][3])));
            const uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
            mine = lane == n ? __uint_as_float(amax) : mine;
        }
        const ScalePair sp = p.pow2 ? group_scale_pow2(mine) : group_scale(mine);
        if (lane < NT && j0 + lane * step < nrows)
            p.sh[(i0 / BI) * p.ld_sh + m0 + j0 + lane * step] = sp.s;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int j = j0 + n * step;
            if (j >= nrows)
                break;
            const float inv = __shfl_sync(0xffffffffu, sp.inv, n);
            *reinterpret_cast<uint32_t *>(p.h + (m0 + j) * p.ldh + col) =
                cvt_e4m3x2(v[n][0] * inv, v[n][1] * inv) | (cvt_e4m3x2(v[n][2] * inv, v[n][3] * inv) << 16);
        }
    }
}

template <int TILING>
__global__ void __launch_bounds__(THREADS, 1)
    gated_cluster_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmS, const ClusterParams p)
{
    using SH = Shape<TILING>;
    constexpr int NS = SH::STAGES, NB = SH::BUFS, TOK = SH::TOK;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    // the swizzled stages assume the alignment requested above (the same for
    // every CTA): refuse to run if it is missing
    if (sbase & 1023u) {
        if (threadIdx.x == 0)
            atomicCAS(p.status, 0, FP8FG_EUNSUPPORTED);
        return;
    }
    const uint32_t full_bar = sbase + SH::full_off, empty_bar = sbase + SH::empty_off;
    const uint32_t tempty_bar = sbase + SH::tempty_off, tfull_bar = sbase + SH::tfull_off;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + SH::abort_off);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtl wc{abort_flag, p.status, p.wait_limit_ns};

    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(full_bar + 8 * s, 2);
            mbar_init(empty_bar + 8 * s, PROMO_WARPS);
            mbar_init(tempty_bar + 8 * s, PROMO_WARPS);
        }
        for (int b = 0; b < NB; ++b)
            mbar_init(tfull_bar + 8 * b, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmS);
    }
    if (warp == 1) {
        tmem_alloc(sbase + SH::tmem_ptr_off, SH::TMEM_COLS);
        tmem_relinquish();
    }
    griddep_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(smem + SH::tmem_ptr_off);

    const int rank = (int)blockIdx.x % p.split, tile = (int)blockIdx.x / p.split;
    const int64_t m0 = (int64_t)(tile % p.token_tiles) * TOK, i0 = (int64_t)(tile / p.token_tiles) * BI;
    const int num_kb = (int)(p.K / BK);
    const int k0 = (int)((int64_t)rank * num_kb / p.split), k1 = (int)((int64_t)(rank + 1) * num_kb / p.split);
    const int nrows = p.M - m0 < TOK ? (int)(p.M - m0) : TOK;

    if (warp == 0) {
        // ------------------------------------------------------ producer ----
        if constexpr (SH::REBALANCE)
            setmaxnreg_dec<LOW>();
        uint32_t stage = 0, phase = 0, filled_mask = 0, fill_parity = 0;
        bool skip = p.skip_first_load && blockIdx.x == 0;
        bool ok = true;
        const float *sw_gate = p.sw + (i0 / BI) * num_kb, *sw_up = p.sw + ((p.I + i0) / BI) * num_kb;
        for (int kb = k0; kb < k1; ++kb) {
            bool got = true;
            if (lane == 0)
                got = mbar_wait(empty_bar + 8 * stage, phase ^ 1, wc, FP8FG_ETIMEOUT);
            got = __shfl_sync(0xffffffffu, got ? 1 : 0, 0) != 0;
            if (!got) {
                ok = false;
                break;
            }
            if (skip) {
                skip = false;  // withhold this load: consumers must time out
            } else if (lane == 0) {
                const uint32_t fb = full_bar + 8 * stage;
                const uint32_t slot = sbase + SH::slot_off + stage * SH::SLOT;
                const uint32_t w_dst = sbase + SH::w_off + stage * W_BYTES;
                mbar_arrive_expect_tx(fb, W_BYTES + SH::X_BYTES + 4 * TOK);
                filled_mask |= 1u << stage;
                fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
                tma_load_3d(w_dst, &tmW, kb * BK, (int32_t)i0, 0, fb);  // gate rows, then up rows
                tma_load_2d(sbase + SH::x_off + stage * SH::X_BYTES, &tmX, kb * BK, (int32_t)m0, fb);
                tma_load_2d(slot, &tmS, (int32_t)m0, kb, fb);
                cp_async4(slot + 4 * TOK, sw_gate + kb);
                cp_async4(slot + 4 * TOK + 4, sw_up + kb);
                cp_async_mbar_arrive_noinc(fb);
            }
            __syncwarp();
            if (++stage == NS) {
                stage = 0;
                phase ^= 1;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!ok && lane == 0) {
            // every issued fill lands before the CTA exits
            for (int s = 0; s < NS; ++s) {
                if (!(filled_mask & (1u << s)))
                    continue;
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(full_bar + 8 * s, (fill_parity >> s) & 1u) &&
                       global_timer_ns() - t0 < p.wait_limit_ns) {
                }
            }
        }
        __syncwarp();
        cluster_sync();
        cluster_sync();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA ----
        if constexpr (SH::REBALANCE)
            setmaxnreg_dec<LOW>();
        constexpr uint32_t IDESC = TILING == FEW ? idesc_e4m3_f32(BI, TOK, false) : idesc_e4m3_f32(TOK, 2 * BI, false);
        bool ok = true, committed = false;
        uint32_t stage = 0, phase = 0, buf = 0, tphase = 0, last_buf = 0, last_par = 0;
        for (int g = 0; g < k1 - k0; ++g) {
            if (g >= NB) {
                // the buffer is free once block g - NB has been read out
                const int b = g - NB;
                const bool got = mbar_wait(tempty_bar + 8 * (uint32_t)(b % NS), (uint32_t)((b / NS) & 1), wc,
                                           FP8FG_ETIMEOUT);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
            }
            const bool got = mbar_wait(full_bar + 8 * stage, phase, wc, FP8FG_ETIMEOUT);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t w_addr = sbase + SH::w_off + stage * W_BYTES;
            const uint32_t x_addr = sbase + SH::x_off + stage * SH::X_BYTES;
            if (elect_one_sync()) {
                if constexpr (TILING == FEW) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int k = 0; k < BK / MMA_K; ++k)
                            mma_f8f6f4(tmem_base + buf * SH::BUF_COLS + h * TOK,
                                       smem_desc_sw128(w_addr + h * (BI * BK) + k * MMA_K, 0, 1024),
                                       smem_desc_sw128(x_addr + k * MMA_K, 0, 1024), IDESC, k > 0 ? 1u : 0u);
                } else {
#pragma unroll
                    for (int k = 0; k < BK / MMA_K; ++k)
                        mma_f8f6f4(tmem_base + buf * SH::BUF_COLS, smem_desc_sw128(x_addr + k * MMA_K, 0, 1024),
                                   smem_desc_sw128(w_addr + k * MMA_K, 0, 1024), IDESC, k > 0 ? 1u : 0u);
                }
                mma_commit(tfull_bar + 8 * buf);
            }
            __syncwarp();
            committed = true;
            last_buf = buf;
            last_par = tphase;
            if (++stage == NS) {
                stage = 0;
                phase ^= 1;
            }
            if (++buf == NB) {
                buf = 0;
                tphase ^= 1;
            }
        }
        if (!ok && committed && lane == 0) {
            // the last commit covers every MMA issued before it
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(tfull_bar + 8 * last_buf, last_par) && global_timer_ns() - t0 < p.wait_limit_ns) {
            }
        }
        __syncwarp();
        cluster_sync();
        cluster_sync();
        tc_fence_after();
        tmem_dealloc(tmem_base, SH::TMEM_COLS);
    } else if (warp < PROMO_WARP0) {
        if constexpr (SH::REBALANCE)
            setmaxnreg_dec<LOW>();  // completes warpgroup 0; no role
        cluster_sync();
        cluster_sync();
    } else {
        // ---------------------------------------------------- promotion ----
        if constexpr (SH::REBALANCE)
            setmaxnreg_inc<HIGH>();
        const int quarter = warp & 3, half = (warp - PROMO_WARP0) >> 2;
        constexpr int SUMS = TILING == FEW ? TOK : BI;  // per thread
        float2 acc[SUMS / 2];
#pragma unroll
        for (int j = 0; j < SUMS / 2; ++j)
            acc[j] = make_float2(0.0f, 0.0f);
        uint32_t stage = 0, phase = 0, buf = 0, tphase = 0;
        for (int g = 0; g < k1 - k0; ++g) {
            bool got = mbar_wait(full_bar + 8 * stage, phase, wc, FP8FG_ETIMEOUT);
            if (!__all_sync(0xffffffffu, got))
                break;
            const float *slot = reinterpret_cast<const float *>(smem + SH::slot_off + stage * SH::SLOT);
            const float sw = slot[TOK + half];
            const float sx = TILING == ROWS ? slot[quarter * 32 + lane] : 0.0f;
            got = mbar_wait(tfull_bar + 8 * buf, tphase, wc, FP8FG_ETIMEOUT);
            if (!__all_sync(0xffffffffu, got))
                break;
            tc_fence_after();
            const uint32_t taddr =
                tmem_base + ((uint32_t)(quarter * 32) << 16) + buf * SH::BUF_COLS + half * SUMS;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(tempty_bar + 8 * stage);
            };
            if constexpr (TILING == FEW) {
                const float2 sw2 = make_float2(sw, sw);
                uint32_t r[32];
                tmem_ld_chunk(taddr, r);
                tmem_wait_ld_chunk(r);
                release();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 s4 = reinterpret_cast<const float4 *>(slot)[j];
                    acc[2 * j] = __ffma2_rn(make_float2(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1])),
                                            __fmul2_rn(make_float2(s4.x, s4.y), sw2), acc[2 * j]);
                    acc[2 * j + 1] =
                        __ffma2_rn(make_float2(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])),
                                   __fmul2_rn(make_float2(s4.z, s4.w), sw2), acc[2 * j + 1]);
                }
                // the block's MMAs are complete and its scales read
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(empty_bar + 8 * stage);
            } else {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(empty_bar + 8 * stage);
                const float2 s2 = make_float2(sx * sw, sx * sw);
                auto fold = [&](int c, const uint32_t(&r)[16]) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        acc[8 * c + j] =
                            __ffma2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), s2,
                                       acc[8 * c + j]);
                };
                // (the schedule of the GEMM's promotion: the buffer goes back
                // to the MMA once all its columns are in registers)
                uint32_t r[4][16];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld_chunk(taddr + 16 * c, r[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_wait_ld_chunk(r[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    fold(c, r[c]);
                    tmem_ld_chunk(taddr + 16 * (4 + c), r[c]);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_wait_ld_chunk(r[c]);
                release();
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    fold(4 + c, r[c]);
            }
            if (++buf == NB) {
                buf = 0;
                tphase ^= 1;
            }
            if (++stage == NS) {
                stage = 0;
                phase ^= 1;
            }
        }
        // (the ring is idle: every fill has landed and every MMA is complete)
        float *sums = reinterpret_cast<float *>(smem);
        if constexpr (TILING == FEW) {
            sums += half * BI + quarter * 32 + lane;
#pragma unroll
            for (int j = 0; j < TOK; ++j)
                if (j < nrows)
                    sums[j * SH::PITCH] = (j & 1) ? acc[j >> 1].y : acc[j >> 1].x;
        } else if (quarter * 32 + lane < nrows) {
            sums += (quarter * 32 + lane) * SH::PITCH + half * BI;
#pragma unroll
            for (int j = 0; j < BI / 4; ++j)
                reinterpret_cast<float4 *>(sums)[j] =
                    make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y);
        }
        tc_fence_before();
        __syncwarp();
        cluster_sync();
        if (!*abort_flag)
            finish_tokens<SH::PITCH, TILING == FEW ? 1 : 8>(p, sbase, rank, warp - PROMO_WARP0, lane, nrows, m0, i0);
        // the other CTAs have read this one's sums
        __syncwarp();
        cluster_sync();
    }
}

template <int TILING>
void launch_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int64_t tiles, int split, cudaStream_t s)
{
    cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * split));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Shape<TILING>::total;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
}

template <int TILING>
bool set_attributes()
{
    static std::atomic<uint64_t> done{0};
    return allow_smem(gated_cluster_kernel<TILING>, Shape<TILING>::total, done);
}

// Clusters of `split` CTAs that run at once on device `dev` (the current one);
// 0 when the query fails. A cluster's CTAs share a GPC, so this is less than
// SMs / split; asked once per device, tiling and split.
template <int TILING>
int clusters_at_once(int dev, int split)
{
    static PerDevice known[MAX_SPLIT + 1];
    return known[split].get(dev, [&] {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        launch_config<TILING>(cfg, attr, sm_count(), split, nullptr);
        cfg.numAttrs = 1;  // the cluster dimension
        int n = 0;
        if (!set_attributes<TILING>() ||
            cudaOccupancyMaxActiveClusters(&n, gated_cluster_kernel<TILING>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        return n;
    });
}

template <int TILING>
int launch_clusters(const GatedArgs &g, int split, cudaStream_t s)
{
    using SH = Shape<TILING>;
    ClusterParams p{};
    p.M = g.M, p.I = g.I, p.K = g.K;
    p.sw = g.sw;
    p.h = g.h, p.ldh = g.ldh, p.sh = g.sh, p.ld_sh = g.ld_sh;
    p.gu = g.gu, p.ld_gu = g.ld_gu;
    p.token_tiles = (int)((g.M + SH::TOK - 1) / SH::TOK);
    p.split = split;
    p.pow2 = g.pow2;
    p.status = status_word_ptr();
    p.wait_limit_ns = wait_limit_ns();
    p.skip_first_load = take_skip_first_load() ? 1 : 0;
    CUtensorMap tw, tx, ts;
    const uint64_t dims[2] = {(uint64_t)g.I, 2}, strides[2] = {1, (uint64_t)g.I};
    const uint32_t box[2] = {BI, 2};
    if (!p.status ||
        !make_map_rows(&tw, g.wq, (uint64_t)g.K, (uint64_t)g.ldw, 2, dims, strides, BK, box) ||
        !make_map(&tx, g.xq, (uint64_t)g.K, (uint64_t)g.M, (uint64_t)g.ldx, BK, SH::TOK) ||
        !make_map_f32_row(&ts, g.sx, (uint64_t)g.M, (uint64_t)(g.K / BK), (uint64_t)g.ld_sx, SH::TOK))
        return FP8FG_ECUDA;
    auto k = gated_cluster_kernel<TILING>;
    if (!set_attributes<TILING>())
        return FP8FG_ECUDA;
    if constexpr (SH::REBALANCE) {
        // the setmaxnreg split must fit in the registers the launch holds
        // (asked once: the kernel has one binary)
        static std::atomic<int> regs{0};
        if (regs.load() == 0) {
            cudaFuncAttributes fa;
            if (cudaFuncGetAttributes(&fa, k) != cudaSuccess) {
                cudaGetLastError();
                return FP8FG_ECUDA;
            }
            regs.store(fa.numRegs);
        }
        if (regs.load() < LAUNCH_MIN)
            return FP8FG_EUNSUPPORTED;
    }
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    launch_config<TILING>(cfg, attr, (int64_t)p.token_tiles * (g.I / BI), split, s);
    if (cudaLaunchKernelEx(&cfg, k, tw, tx, ts, p) != cudaSuccess) {
        cudaGetLastError();
        return FP8FG_ECUDA;
    }
    return launch_status();
}

// The tiling of a call and its split of the contraction.
struct Plan {
    int tiling;  // Tiling, or PERSISTENT
    int split;
};
constexpr int PERSISTENT = -1;

template <int TILING>
bool consider(int dev, int64_t tiles, int64_t num_kb, double block_us, double fixed_us, double split_us, Plan &best,
              double &best_us)
{
    for (int split = 1; split <= MAX_SPLIT && split <= num_kb; ++split) {
        const int64_t at_once = clusters_at_once<TILING>(dev, split);
        if (at_once == 0)
            return false;
        const int64_t waves = (tiles + at_once - 1) / at_once;
        const double us = waves * ((num_kb + split - 1) / split * block_us + fixed_us + (split - 1) * split_us);
        if (us < best_us) {
            best_us = us;
            best = {TILING, split};
        }
    }
    return true;
}

// The shortest estimate: waves x (contraction blocks of a CTA x time per block
// + the fixed part of a tile + a term per CTA of the cluster). The constants
// are fits to measured times (us, loads from DRAM): 24 tokens through K x 1024
// with K = 1024 / 7168 and no split 7.7 / 29.1 (FEW); 333 tokens 10.6 / 28.6
// (ROWS) and 8.5 / 29.1 (persistent, which has no cluster barriers). Measured
// against every other tiling and split for 1 to 1500 tokens and widths of 128
// to 18432, the choice was the fastest or within 5 % of it: 333 tokens through
// 7168 x 2048 take 19.4 us split in two against 29.6 us in persistent tiles,
// through 2048 x 8192 28.7 (no split) against 22.7. The choice fixes the order of the sums,
// so it goes by the shape and the device alone: false (no plan) when the device
// does not say how many clusters it runs.
bool choose(int64_t M, int64_t I, int64_t K, Plan &best)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    const int64_t sms = sm_count() > 0 ? sm_count() : 1, num_kb = K / BK, cols = I / BI, rows = (M + 127) / 128;
    best = {PERSISTENT, 1};
    double best_us = (double)((rows * cols + sms - 1) / sms) * (num_kb * 0.43 + 5.0);
    if (M <= Shape<FEW>::TOK) {
        // (always: wide weights are bound by the memory, which the estimates
        // leave out; one token through 7168 x 18432: 43 us, persistent 56)
        best_us = 1e30;
        return consider<FEW>(dev, cols, num_kb, 0.45, 4.1, 0.15, best, best_us);
    }
    return rows * cols > sms || consider<ROWS>(dev, rows * cols, num_kb, 0.38, 7.6, 0.35, best, best_us);
}

}  // namespace
}  // namespace fp8fg

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
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    Plan plan;
    if (!choose(M, I, K, plan))
        return FP8FG_ECUDA;
    switch (plan.tiling) {
    case FEW: return launch_clusters<FEW>(g, plan.split, s);
    case ROWS: return launch_clusters<ROWS>(g, plan.split, s);
    default: return gated_gemm_tiles(g, s);
    }
}
