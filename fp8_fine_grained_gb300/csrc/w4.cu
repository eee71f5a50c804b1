// Products of few rows with 4-bit weights, and the quantiser of those weights.
//
//     y[r][n] = sum over groups g of s[n][g] * sum_{k in g} x[r][k] c[n][k]
//
// with c the value of a 4-bit code (E2M1, or a two's complement integer) and one
// FP32 scale per group of 32, 64 or 128 columns of a weight row; dense, or by
// expert with the rows in expert order. With the gate, the weight is a gate
// projection on top of an up projection and y = silu(G) * U.
//
// Decoding: every weight is used for a handful of rows, so the floor is the
// stream of the codes (K / 2 + 4 K / group bytes per weight row).
//
// Arithmetic. A code's value is exact in FP16. x is brought to FP16 exactly:
// within every 128 columns of a row by a power of two that takes the largest
// magnitude to [2^14, 2^15). (A bf16 value has 8 significant bits; those below
// 2^-31 of the block's largest are rounded to FP16's step of 2^-24, by half of it
// at most: 2^-39 of the largest.) The products are exact in FP32, in which the
// tensor cores add them up within a group; the group's sum times the product of
// its two scales is added up in FP32 registers.
//
// Shape. A unit is 16 or 32 weight rows (one or two m16n8k16 operands; with the
// gate, half of them gate rows and half the up rows below them) by up to 8 or 16
// rows of x. Units go to groups of ks warps, which share the unit's steps of
// 256 columns and join their sums in shared memory: with few units every warp of
// the device still has loads in flight. A warp's codes come by TMA into a ring of
// its own, which runs ahead over the ends of K and of the units; x is staged by
// the whole CTA, once for all the units of the same rows where it fits. Where it does
// not, a cluster of CTAs shares K.
//
// Bound by: the stream of the codes where it is long (64 tokens by 8 of 256 experts,
// 2048 -> 7168: 255 to 276 us on different machines, 1.74 GB, 0.93 to 1.0 of HBM copy);
// 5 us of launch, set-up, first loads and join where it is short (one token, 7168 -> 2 x
// 2048: 7.1 us for 15.6 MB); instructions for integer codes (9 for 8 codes, where E2M1
// takes 4: 5 tokens, 18432 -> 7168, groups of 64: 26.5 us for 74.6 MB, of which 5 us stage
// x and 2 us join the cluster), for 16 rows (twice the matrix instructions: 28672 x 7168 in
// 44.2 us where 8 rows take 28.4) and, beyond, for every tile of 16 rows anew (91.7 us for
// 32 rows, 162 for 64).
// Tried: loads by cp.async with addresses of each lane's own (337 instructions per
// 32 x 128 codes instead of 234), two CTAs of eight warps per SM with an x each (8
// experts' gate and up projections of one token 36.8 us instead of 26.3), tiles of 32
// rows (twice the time of two of 16).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "host_common.h"
#include "per_device.h"
#include "ptx.cuh"
#include "tensor_map.h"

#include <type_traits>
#include <utility>

namespace fp8fg {
namespace {

constexpr unsigned ALL = 0xFFFFFFFFu;
constexpr int STEP = 128;         // columns that share a scale of x
constexpr int WARPS = 16, THREADS = 32 * WARPS;
constexpr int LOAD = 256;         // columns of a stage of the ring
constexpr int MAX_RING = 4;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_STAGED = 64;    // rows of x that shared memory is asked for
constexpr int MAX_EXPERTS = 4096;

// Division of 0 <= n < 2^31 by a number that the host knows: one product.
struct Divisor {
    uint32_t d, mul, shift;
};

inline Divisor divisor(uint32_t d)
{
    // (rounding the reciprocal up is exact for n < 2^31 with 2^shift >= d)
    uint32_t shift = 0;
    while ((1ull << shift) < d)
        ++shift;
    return {d, (uint32_t)(((1ull << (31 + shift)) + d - 1) / d), shift};
}

__device__ __forceinline__ uint32_t div_by(uint32_t n, const Divisor &v)
{
    return (uint32_t)(((uint64_t)n * v.mul) >> 31 >> v.shift);
}

// Warps to a unit (their logarithm): the number with which the CTA's warps go
// through the fewest stages one after another, for `share` units a CTA, or a larger
// one that costs a tenth more at most. (Measured: 8 experts' gate and up projections
// of one token, 7 units of 28 stages a CTA: 32.4, 29.5, 27.1, 29.6 and 32.7 us with 1,
// 2, 4, 8 and 16 warps; 64 tokens' down projections, 339 units of 8 stages: 269, 267,
// 298, 407 us with 1 to 8.)
__host__ __device__ __forceinline__ int share_warps(int share, int loads, int log_cluster)
{
    const int most_loads = (loads + (1 << log_cluster) - 1) >> log_cluster;
    int log_ks = 0, least = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; 1 << i <= WARPS; ++i) {
        // (a turn costs about one stage beside its own: the join)
        const int turns = ((share << i) + WARPS - 1) / WARPS, cost = turns * (((most_loads + (1 << i) - 1) >> i) + 1);
        if (1 << i <= loads >> log_cluster && (i == 0 || 10 * (int64_t)cost <= 11 * (int64_t)least)) {
            least = cost < least ? cost : least;
            log_ks = i;
        }
    }
    return log_ks;
}

struct W4Args {
    const uint16_t *x;
    int64_t ldx, T;
    const int32_t *row_index, *offsets;
    int E;
    int64_t n_rows;
    const uint8_t *wq;
    const float *sw;
    int64_t wide;     // weight rows of an expert
    int64_t N, K;     // output columns; contraction
    int loads;        // stages of a unit: K / 256, rounded up
    int units;        // units of an expert's weight
    Divisor by_units, by_clusters;
    int ring;         // stages of a warp's ring
    int cluster, log_cluster;  // CTAs that share K
    int log_ks;       // warps that share a unit (without offsets)
    int x_halfs;      // capacity of the staged x
    int fit_rows;     // rows that fit whole (where a tile's do not, they are staged in pieces)
    void *y;
    int64_t ldy;
    int out_f32, gated;
    int *status;
    uint64_t limit_ns;
    int skip_first_load;
};

template <int G, int NT, int P>
struct Layout {
    static constexpr int ROWS = 16 * P;                            // of a unit
    static constexpr int CODES = ROWS * LOAD / 2;                  // bytes of a stage
    static constexpr int SCALES = LOAD / G;                        // of a row and stage
    static constexpr int STAGE = CODES + ROWS * SCALES * 4;
    static constexpr int TOKENS = 8 * NT;
    static constexpr int RED = WARPS * ROWS * TOKENS * 4;
    static constexpr int UNIT_SUMS = ROWS * TOKENS * 4;            // bytes
    static constexpr int PARTS = 16 * 1024 / UNIT_SUMS;  // units whose sums a cluster joins at once
};

__device__ __forceinline__ void cp_async4_or_zero(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}

template <int OFFSET>
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(v) : "r"(a), "n"(OFFSET));
    return v;
}

template <int OFFSET>
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a), "n"(OFFSET));
    return v;
}

// f(0), f(1), ... with constants
template <int... I, typename F>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>()), ...);
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A float at this CTA's shared address `a`, of CTA `rank` of the cluster.
__device__ __forceinline__ float cluster_float(uint32_t a, int rank)
{
    uint32_t p;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(p) : "memory");
    return v;
}

__device__ __forceinline__ void group_sync(int id, int threads)
{
    if (threads == 32)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// c = A B, or c + A B
template <bool FIRST>
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    const float z0 = FIRST ? 0.0f : c[0], z1 = FIRST ? 0.0f : c[1], z2 = FIRST ? 0.0f : c[2], z3 = FIRST ? 0.0f : c[3];
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%10, %11, %12, %13};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2), "f"(z3));
}

// The eight codes of a word as four FP16 pairs. E2M1: pair i holds codes 2i and
// 2i + 1. Integers: codes i and i + 4, so that a mask takes a pair out at once;
// 1024 + u (or 1024 + 16 u) stands in an FP16 whose low bits are u = code + 8.
template <int KIND>
__device__ __forceinline__ void decode(uint32_t w, uint32_t (&h)[4])
{
    if constexpr (KIND == FP8FG_E2M1) {
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(w));
    } else {
        // The published way to take 4-bit integers apart: a three-input operation masks a
        // nibble out into the low bits of an FP16 of exponent 1024, and one subtraction (with
        // a factor of 1/16 for a nibble in the next four bits) leaves its value. Here the
        // operation also flips the code's sign bit, so that two's complement comes out.
        // (in registers: a three-input operation takes one constant of its own)
        uint32_t low, high, low_base, high_base;
        asm("mov.b32 %0, 0x000F000F;" : "=r"(low));
        asm("mov.b32 %0, 0x00F000F0;" : "=r"(high));
        asm("mov.b32 %0, 0x64086408;" : "=r"(low_base));
        asm("mov.b32 %0, 0x64806480;" : "=r"(high_base));
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t v = w >> (4 * i);
            uint32_t lo, hi;  // (v & mask) ^ base
            asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(lo) : "r"(v), "r"(low), "r"(low_base));
            asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(hi) : "r"(v), "r"(high), "r"(high_base));
            asm("add.rn.f16x2 %0, %1, %2;" : "=r"(h[i]) : "r"(lo), "r"(0xE408E408u));  // - 1032
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h[i + 1]) : "r"(hi), "r"(0x2C002C00u), "r"(0xD480D480u));  // / 16 - 72
        }
    }
}

// Where unit u belongs: rows [row0, row0 + count) of expert e, whose units end
// before unit `end`; the unit's place among them.
struct Tile {
    int e, count, end, unit, row0;
};

// The experts' rows and units, added up: [E + 1] each, in shared memory.
struct Tables {
    const int32_t *rows, *units;
};

template <int TOKENS>
__device__ __forceinline__ Tile tile_of(const W4Args &a, const Tables &tab, int u)
{
    int lo = 0, hi = a.E;  // units[lo] <= u < units[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.units[mid] <= u)
            lo = mid;
        else
            hi = mid;
    }
    const int i = u - tab.units[lo], tile = (int)div_by(i, a.by_units);
    Tile k;
    k.e = lo;
    k.unit = i - tile * a.units;
    k.end = u - k.unit + a.units;
    k.row0 = tab.rows[lo] + tile * TOKENS;
    k.count = min(TOKENS, tab.rows[lo + 1] - k.row0);
    return k;
}

// tile_of, from the tile of another unit, which is mostly the same.
template <int TOKENS>
__device__ __forceinline__ void seek(const W4Args &a, const Tables &tab, int u, Tile &k)
{
    if (u < k.end && u >= k.end - a.units)
        k.unit = u - (k.end - a.units);
    else
        k = tile_of<TOKENS>(a, tab, u);
}

// Units [pos, end) that a CTA goes through without a change of the staged x: rows
// [row0, row0 + rows), those of the units' tiles, follow each other.
struct Segment {
    int end, rows, row0;
};

template <int TOKENS>
__device__ __forceinline__ Segment segment_at(const W4Args &a, const Tables &tab, int pos, Tile k, int u_end,
                                              int most_units)
{
    Segment g;  // (k: the tile of unit pos)
    g.row0 = k.row0;
    for (;;) {
        g.end = min(min(k.end, u_end), pos + most_units);
        g.rows = k.row0 - g.row0 + k.count;
        if (g.end != k.end || g.end >= u_end)
            return g;
        k = tile_of<TOKENS>(a, tab, g.end);
        if (k.row0 - g.row0 + k.count > a.fit_rows)
            return g;
    }
}

// Wait for the copies in flight into `ahead` stages of the ring, `stage` (of `parity`)
// and those behind it: nothing may land in shared memory that the CTA has left. The stage
// that was given up on is one of them: its wait ends early where another warp's ran out.
// Every copy was asked for before this began, so that one limit covers them all (a copy
// that never comes costs it once).
__device__ __forceinline__ void drain(uint32_t full_at, int stage, uint32_t parity, int ahead, int ring, uint64_t limit_ns)
{
    const uint64_t t0 = global_timer_ns();
    for (int i = 0; i < ahead; ++i) {
        while (!mbar_try_wait(full_at + 8 * stage, parity) && global_timer_ns() - t0 < limit_ns)
            ;
        if (++stage == ring) {
            stage = 0;
            parity ^= 1;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // (scales of a stage whose codes never come)
}

// Columns [c0, c0 + 128 here) of rows [row0, row0 + rows) of x into shared memory, in
// FP16 with a power of two for every 128 columns: sixteen lanes a step, eight
// columns each, in the order in which decode gives the codes. begin, then load and
// store in turn while there is something left.
template <int KIND>
struct XStage {
    static constexpr int BATCH = 4, HALVES = THREADS / 16;  // loads of a thread in flight; half-warps
    uint4 v[BATCH];
    int to[BATCH];  // row << 20 | step, or -1
    int row0, rows, c0, here, r, s, row_of;
    const uint16_t *row_at;

    __device__ __forceinline__ void begin(int row0_, int rows_, int c0_, int here_)
    {
        row0 = row0_;
        rows = rows_;
        c0 = c0_;
        here = here_;
        r = 0;
        s = threadIdx.x >> 4;
        row_of = -1;
    }

    __device__ __forceinline__ void load(const W4Args &a)
    {
        const int hl = threadIdx.x & 15;
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            for (; s >= here && r < rows; ++r)
                s -= here;
            to[b] = r < rows ? r << 20 | s : -1;
            v[b] = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                if (row_of != r) {
                    int64_t t = row0 + r;
                    if (a.row_index) {
                        t = a.row_index[row0 + r];
                        if (t < 0 || t >= a.T) {
                            atomicCAS(a.status, 0, FP8FG_EDEVICE);
                            t = 0;
                        }
                    }
                    row_of = r;
                    row_at = a.x + t * a.ldx + c0 + hl * 8;
                }
                if (c0 + s * STEP + hl * 8 < (int)a.K)
                    v[b] = *reinterpret_cast<const uint4 *>(row_at + s * STEP);
            }
            s += HALVES;
        }
    }

    // (row r of the staged x begins at r * pitch; its scales at r * (pitch / 128))
    __device__ __forceinline__ bool store(int pitch, __half *xs, float *sx)
    {
        const int hl = threadIdx.x & 15;
        const unsigned mates = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            if (to[b] < 0)
                return false;
            const uint32_t u[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
            // the largest exponent of the block's finite values: of the magnitudes' bits, two
            // values at a time
            uint32_t m = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                m = __vmaxu2(m, u[q] & 0x7FFF7FFFu);
            if ((m & 0xFFFFu) >= 0x7F80u || m >= 0x7F800000u) {  // infinities and NaN do not count
                m = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t w = u[q] & 0x7FFF7FFFu;
                    m = __vmaxu2(m, w & ~__vcmpgeu2(w, 0x7F807F80u));
                }
                m = __vmaxu2(m, 141u << 7);  // (a factor of 1 at least, which leaves them infinite)
            }
            uint32_t e = max(m & 0xFFFFu, m >> 16);
#pragma unroll
            for (int d = 8; d; d >>= 1)
                e = max(e, __shfl_xor_sync(mates, e, d));
            e = max(e >> 7, 15u);  // (the factors stay normal numbers)
            const float up = __uint_as_float((268u - e) << 23);
            uint32_t h[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // (integers take their codes in pairs i and i + 4)
                const float lo = KIND == FP8FG_E2M1 ? bf16_lo(u[q]) : q & 1 ? bf16_hi(u[q / 2]) : bf16_lo(u[q / 2]);
                const float hi = KIND == FP8FG_E2M1 ? bf16_hi(u[q]) : q & 1 ? bf16_hi(u[2 + q / 2]) : bf16_lo(u[2 + q / 2]);
                const __half2 p = __floats2half2_rn(lo * up, hi * up);
                h[q] = *reinterpret_cast<const uint32_t *>(&p);
            }
            const int at_r = to[b] >> 20, at_s = to[b] & 0xFFFFF;
            *reinterpret_cast<uint4 *>(xs + at_r * pitch + at_s * STEP + hl * 8) = make_uint4(h[0], h[1], h[2], h[3]);
            if (hl == 0)
                sx[at_r * (pitch / STEP) + at_s] = __uint_as_float((e - 14u) << 23);
        }
        return true;
    }
};

// One element of y: a sum, or with the gate silu(v) * up.
__device__ __forceinline__ void write_out(const W4Args &a, float v, float up, int64_t at)
{
    if (a.gated)
        v = v / (1.0f + expf(-v)) * up;
    if (a.out_f32)
        static_cast<float *>(a.y)[at] = v;
    else
        static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v);
}

template <int KIND, int G, int NT, int P>
__global__ void __launch_bounds__(THREADS, 1)
    w4_matvec_kernel(const W4Args a, const __grid_constant__ CUtensorMap codes)
{
    using Lay = Layout<G, NT, P>;
    constexpr int TOKENS = Lay::TOKENS, SC = Lay::SCALES, CODES = Lay::CODES, ROWS = Lay::ROWS;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int32_t warp_sums[WARPS];
    __shared__ __align__(8) uint64_t full[WARPS][MAX_RING];
    __shared__ int abort_flag;
    const int lane = (int)lane_id(), warp = threadIdx.x >> 5;
    // rings of codes, rings of scales, sums to be joined, rows and units before each
    // expert [E + 1], sums to be joined in the cluster, scales of the staged x, the staged x
    const int ring = a.ring;
    float *red = reinterpret_cast<float *>(smem + WARPS * ring * Lay::STAGE);
    int32_t *first_row = reinterpret_cast<int32_t *>(red + Lay::RED / 4), *first_unit = first_row + (a.E + 4) / 4 * 4;
    const Tables tab = {first_row, first_unit};
    float *parts = reinterpret_cast<float *>(first_unit + (a.E + 4) / 4 * 4);  // (only in a cluster)
    float *sx = parts + (a.cluster > 1 ? Lay::PARTS * Lay::UNIT_SUMS / 4 : 0);
    __half *xs = reinterpret_cast<__half *>(sx + (a.x_halfs / STEP + 3) / 4 * 4);
    const uint32_t ring_at = smem_u32(smem) + warp * ring * CODES;
    const uint32_t scales_at = smem_u32(smem) + (WARPS * CODES + warp * ROWS * SC * 4) * ring;
    const uint32_t xs_at = smem_u32(xs), sx_at = smem_u32(sx), full_at = smem_u32(&full[warp][0]);
    const WaitCtl ctl = {&abort_flag, a.status, a.limit_ns};

    // every stage: the codes' copy, and each lane's copies of scales
    if (lane < ring)
        mbar_init(full_at + 8 * lane, 33);
    if (threadIdx.x == 0) {
        abort_flag = 0;
        tma_prefetch_desc(&codes);
    }
    fence_mbar_init();
    griddep_launch_dependents();
    griddep_wait();

    // rows and units of every expert, added up
    if (!a.offsets) {
        if (threadIdx.x == 0) {
            first_row[0] = first_unit[0] = 0;
            first_row[1] = (int)a.n_rows;
            first_unit[1] = (int)((a.n_rows + TOKENS - 1) / TOKENS * a.units);
        }
        __syncthreads();
    } else {
        const int each = (a.E + THREADS - 1) / THREADS;
        const int lo = min((int)threadIdx.x * each, a.E), hi = min(lo + each, a.E);
        int sum = 0, next = lo < a.E ? a.offsets[lo] : 0;
        bool bad = false;
        for (int e = lo; e < hi; ++e) {
            const int from = next;
            next = a.offsets[e + 1];
            bad |= from < 0 || next < from || next > a.n_rows || (e == 0 && from != 0);
            first_row[e] = from;
            first_unit[e] = sum;
            sum += (int)((int64_t)(next - from + TOKENS - 1) / TOKENS * a.units);
        }
        int upto = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(ALL, upto, d);
            upto += lane >= d ? v : 0;
        }
        if (lane == 31)
            warp_sums[warp] = upto;
        if (__syncthreads_or(bad)) {  // malformed offsets: nothing is computed
            if (threadIdx.x == 0)
                atomicCAS(a.status, 0, FP8FG_EDEVICE);
            return;
        }
        int before = upto - sum, all = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            before += w < warp ? warp_sums[w] : 0;
            all += warp_sums[w];
        }
        for (int e = lo; e < hi; ++e)
            first_unit[e] += before;
        if (lo < a.E && hi == a.E) {
            first_row[a.E] = next;
            first_unit[a.E] = all;
        }
        __syncthreads();
    }
    // this cluster's run of units, even to one, and this CTA's share of K
    const int clusters = (int)gridDim.x >> a.log_cluster, cluster_id = (int)blockIdx.x >> a.log_cluster;
    const int rank = (int)blockIdx.x & (a.cluster - 1);
    const int all_units = first_unit[a.E], even = (int)div_by(all_units, a.by_clusters), more = all_units - even * clusters;
    const int u_begin = even * cluster_id + min(cluster_id, more), u_end = u_begin + even + (cluster_id < more);
    const int l_begin = (a.loads * rank) >> a.log_cluster, l_stop = (a.loads * (rank + 1)) >> a.log_cluster;

    const int log_ks = a.offsets ? share_warps(even + (more > 0), a.loads, a.log_cluster) : a.log_ks;
    const int ks = 1 << log_ks, groups = WARPS >> log_ks, group = warp >> log_ks, part = warp & (ks - 1);
    const int outs = a.gated ? ROWS / 2 : ROWS, log_outs = (P == 2 ? 5 : 4) - a.gated;  // output columns of a unit
    const int spitch = (int)(a.K / G);

    const int most_units = a.cluster > 1 ? Lay::PARTS : 1 << 30;

    // (the first rows of x are asked for before the codes, whose loads would be ahead
    // of them in every queue)
    const int span = (l_stop - l_begin) * LOAD;
    Tile k = {};
    Segment seg = {u_begin, 0, 0};
    XStage<KIND> xst;
    if (u_begin < u_end) {
        k = tile_of<TOKENS>(a, tab, u_begin);
        seg = segment_at<TOKENS>(a, tab, u_begin, k, u_end, most_units);
        xst.begin(seg.row0, seg.rows, l_begin * LOAD, span / STEP);
        if (seg.rows <= a.fit_rows)
            xst.load(a);
    }

    // the loads: stage ld_step of unit ld_u; the segment's units go to the groups in
    // turn, starting with the first
    int ld_u = u_begin + group, ld_end = seg.end, ld_step = l_begin + part, ld_n0 = 0;
    const float *ld_scales = a.sw;
    Tile ld_tile = k;
    bool skip = a.skip_first_load && blockIdx.x == 0 && warp == 0;
    auto aim = [&] {
        while (ld_u >= ld_end) {
            if (ld_end >= u_end)
                return;
            ld_u = ld_end + group;
            seek<TOKENS>(a, tab, ld_end, ld_tile);
            ld_end = segment_at<TOKENS>(a, tab, ld_end, ld_tile, u_end, most_units).end;
        }
        seek<TOKENS>(a, tab, ld_u, ld_tile);
        ld_n0 = ld_tile.unit * outs;
        // (rows behind the last are read as it is, and their sums never written)
        const int r = lane & (ROWS - 1), up = a.gated && r >= ROWS / 2;
        const int n = min(ld_n0 + (up ? r - ROWS / 2 : r), (int)a.N - 1);
        ld_scales = a.sw + ((int64_t)ld_tile.e * a.wide + n + (up ? (int)a.N : 0)) * spitch;
    };
    int ahead = 0;  // stages filled and not yet read
    bool dead = false;
    auto fill = [&](int st) {
        if (ld_u >= ld_end || dead)
            return;
        ++ahead;
        const uint32_t bar = full_at + 8 * st;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar, CODES);
            if (!skip)
                tma_load_4d(ring_at + st * CODES, &codes, ld_step * (LOAD / 2), ld_n0, 0, ld_tile.e, bar);
            skip = false;
        }
        // 32 lanes, ROWS rows: with 16 of them, a lane takes every other scale
        constexpr int SKIP = 32 / ROWS;
#pragma unroll
        for (int i0 = 0; i0 < SC; i0 += SKIP) {
            const int i = i0 + (SKIP == 2 ? lane >> 4 : 0), g = ld_step * SC + i;
            cp_async4_or_zero(scales_at + ((st * ROWS + (lane & (ROWS - 1))) * SC + i) * 4,
                              ld_scales + min(g, spitch - 1), g < spitch);
        }
        cp_async_mbar_arrive_noinc(bar);
        ld_step += ks;
        if (ld_step >= l_stop) {
            ld_step = l_begin + part;
            ld_u += groups;
            aim();
        }
    };
    aim();
    for (int i = 0; i < ring; ++i)
        fill(i);

    // this lane's words of a stage: row lane / 4, whose 16-byte piece q the copy puts at
    // piece q ^ (row % 8)
    const uint32_t word_at = ring_at + (lane / 4) * 128 + (lane / 4) * 16 + (lane & 3) * 4;

    int stage = 0;
    uint32_t parity = 0;
    bool fresh = true;  // the segment's x is still to be stored
    for (int pos = u_begin; pos < u_end;) {
        // columns of x that fit: each row has its values, 32 to spare (rows then start half
        // a shared-memory line apart)
        const bool whole = seg.rows <= a.fit_rows;
        const int cols = whole ? span : min((a.x_halfs / seg.rows - 32) / LOAD * LOAD, span);
        const int xpitch = cols + 32, spx = cols / STEP;
        if (whole && fresh) {
            while (xst.store(xpitch, xs, sx))
                xst.load(a);
            __syncthreads();
        }
        for (int u0 = pos; u0 < seg.end; u0 += groups) {
            const int u = u0 + group;
            const bool has = u < seg.end;
            seek<TOKENS>(a, tab, has ? u : pos, k);
            // (columns of the product beyond the tile's rows are computed from its last row
            // and not written)
            uint32_t x_row[NT], x_scale[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r0 = k.row0 - seg.row0, last = k.count - 1;
                x_row[n] = xs_at + 2 * ((r0 + min(n * 8 + lane / 4, last)) * xpitch + (lane & 3) * 8);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    x_scale[n][q] = sx_at + 4 * (r0 + min(n * 8 + 2 * (lane & 3) + q, last)) * spx;
            }
            float acc[P][NT][4] = {};
            for (int c0 = 0; c0 < span; c0 += cols) {
                if (!whole) {
                    __syncthreads();
                    xst.begin(seg.row0, seg.rows, l_begin * LOAD + c0, min(cols, span - c0) / STEP);
                    do
                        xst.load(a);
                    while (xst.store(xpitch, xs, sx));
                    __syncthreads();
                }
                // stages of this CTA's share, counted from its first
                const int l0 = c0 / LOAD, l_end = has ? min(l0 + cols / LOAD, l_stop - l_begin) : 0;
                for (int l = l0 + ((part - l0) & (ks - 1)); l < l_end; l += ks) {
                    // (a load that does not come ends the loads; the sums are then worth
                    // nothing, and the status word says so)
                    if (!dead && !__all_sync(ALL, mbar_wait(full_at + 8 * stage, parity, ctl, FP8FG_ETIMEOUT))) {
                        dead = true;
                        drain(full_at, stage, parity, ahead, ring, a.limit_ns);
                    }
                    const uint32_t at = word_at + stage * CODES;
                    const uint32_t scales = scales_at + (stage * ROWS + lane / 4) * (SC * 4);
                    const uint32_t x_at = (l - l0) * (2 * LOAD), sx_of = (l - l0) * (LOAD / STEP * 4);
                    uint32_t x_now[NT], sx_now[NT][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        x_now[n] = x_row[n] + x_at;
                        sx_now[n][0] = x_scale[n][0] + sx_of;
                        sx_now[n][1] = x_scale[n][1] + sx_of;
                    }
                    float c[P][NT][4];
                    each(std::make_integer_sequence<int, LOAD / 32>(), [&](auto q_) {
                        constexpr int q = decltype(q_)::value, col = q * 32;  // 32 columns
                        uint4 xb[NT];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            xb[n] = lds128<2 * col>(x_now[n]);
                        const uint32_t w = at ^ (q << 4);
                        each(std::make_integer_sequence<int, P>(), [&](auto p_) {
                            constexpr int p = decltype(p_)::value;
                            uint32_t h0[4], h1[4];
                            decode<KIND>(lds32<p * 2048>(w), h0);
                            decode<KIND>(lds32<p * 2048 + 1024>(w), h1);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                if (n > 0 && n * 8 >= k.count)
                                    break;
                                mma_f16<col % G == 0>(c[p][n], h0[0], h1[0], h0[1], h1[1], xb[n].x, xb[n].y);
                                mma_f16<false>(c[p][n], h0[2], h1[2], h0[3], h1[3], xb[n].z, xb[n].w);
                            }
                        });
                        if constexpr ((col + 32) % G == 0) {
                            constexpr int g = col / G, half = col / STEP;
                            float sw[P][2];
                            each(std::make_integer_sequence<int, P>(), [&](auto p_) {
                                constexpr int p = decltype(p_)::value;
                                sw[p][0] = __uint_as_float(lds32<(p * 16 * SC + g) * 4>(scales));
                                sw[p][1] = __uint_as_float(lds32<((p * 16 + 8) * SC + g) * 4>(scales));
                            });
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                if (n > 0 && n * 8 >= k.count)
                                    break;
                                const float x0 = __uint_as_float(lds32<half * 4>(sx_now[n][0]));
                                const float x1 = __uint_as_float(lds32<half * 4>(sx_now[n][1]));
#pragma unroll
                                for (int p = 0; p < P; ++p) {
                                    // (the two scales first: the sum of the codes' products alone leaves
                                    // FP32's range where x is large and the weight's scale small)
                                    acc[p][n][0] = fmaf(c[p][n][0], sw[p][0] * x0, acc[p][n][0]);
                                    acc[p][n][1] = fmaf(c[p][n][1], sw[p][0] * x1, acc[p][n][1]);
                                    acc[p][n][2] = fmaf(c[p][n][2], sw[p][1] * x0, acc[p][n][2]);
                                    acc[p][n][3] = fmaf(c[p][n][3], sw[p][1] * x1, acc[p][n][3]);
                                }
                            }
                        }
                    });
                    __syncwarp();
                    --ahead;
                    fill(stage);
                    if (++stage == ring) {
                        stage = 0;
                        parity ^= 1;
                    }
                }
            }
            if (!has)
                continue;
            // the group's sums, joined in the order of the warps' shares
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        *reinterpret_cast<float2 *>(red + (size_t)(warp * ROWS + p * 16 + q * 8 + lane / 4) * TOKENS +
                                                    n * 8 + 2 * (lane & 3)) =
                            make_float2(acc[p][n][2 * q], acc[p][n][2 * q + 1]);
            group_sync(1 + group, 32 * ks);
            const float *from0 = red + (size_t)group * ks * ROWS * TOKENS;
            const int64_t n0 = (int64_t)k.unit * outs;
            const int here = (int)min((int64_t)outs, a.N - n0);
            if (a.cluster > 1) {  // kept for the cluster's join
                for (int i = part * 32 + lane; i < ROWS * TOKENS; i += 32 * ks) {
                    float v = 0.0f;
#pragma unroll 4
                    for (int q = 0; q < ks; ++q)
                        v += from0[q * ROWS * TOKENS + i];
                    parts[(u - pos) * ROWS * TOKENS + i] = v;
                }
            } else {
                for (int i = part * 32 + lane; i < outs * k.count; i += 32 * ks) {
                    const int t = i >> log_outs, r = i & (outs - 1);
                    if (r >= here)
                        continue;
                    float v = 0.0f, up = 0.0f;
#pragma unroll 4
                    for (int q = 0; q < ks; ++q) {
                        const float *from = from0 + (q * ROWS + r) * TOKENS + t;
                        v += from[0];
                        if (a.gated)
                            up += from[ROWS / 2 * TOKENS];
                    }
                    write_out(a, v, up, (int64_t)(k.row0 + t) * a.ldy + n0 + r);
                }
            }
            group_sync(1 + group, 32 * ks);
        }
        if (a.cluster > 1) {
            // the CTAs' sums, joined in the order of their shares, units in turn
            cluster_sync();
            const uint32_t parts_at = smem_u32(parts);
            const int log_per = log_outs + (NT == 2 ? 4 : 3), units = (seg.end - pos - rank + a.cluster - 1) >> a.log_cluster;
            for (int i = threadIdx.x; i < units << log_per; i += THREADS) {
                const int u = pos + rank + (i >> log_per) * a.cluster;
                const int t = i >> log_outs & (TOKENS - 1), r = i & (outs - 1);
                const Tile of = tile_of<TOKENS>(a, tab, u);
                const int64_t n = (int64_t)of.unit * outs + r;
                if (t >= of.count || n >= a.N)
                    continue;
                const uint32_t at = parts_at + 4 * (((u - pos) * ROWS + r) * TOKENS + t);
                float v = 0.0f, up = 0.0f;
#pragma unroll 4
                for (int q = 0; q < a.cluster; ++q) {
                    v += cluster_float(at, q);
                    if (a.gated)
                        up += cluster_float(at + ROWS / 2 * TOKENS * 4, q);
                }
                write_out(a, v, up, (int64_t)(of.row0 + t) * a.ldy + n);
            }
            cluster_sync();
        }
        pos = seg.end;
        if (pos < u_end) {
            const int row0 = seg.row0, rows = seg.rows;
            seek<TOKENS>(a, tab, pos, k);
            seg = segment_at<TOKENS>(a, tab, pos, k, u_end, most_units);
            fresh = seg.row0 != row0 || seg.rows != rows;  // (else the same rows are staged)
            if (fresh) {
                xst.begin(seg.row0, seg.rows, l_begin * LOAD, span / STEP);
                if (seg.rows <= a.fit_rows)
                    xst.load(a);
                __syncthreads();
            }
        }
    }
}

// ------------------------------------------------------------ quantiser ----

struct W4QuantArgs {
    const uint16_t *w;
    int64_t ldw, rows, K;
    uint8_t *q;
    float *scales;
};

// A lane takes 8 columns (16 bytes in, 4 out), G / 8 lanes a group: the group's
// largest magnitude over the lanes, the scale and its reciprocal by division, one
// product per value and one rounding to nearest even. Once per weight; 32 x 4096 x 7168
// in groups of 128: 610 us, 2.38 GB, 0.57 of HBM copy (integers 706 us, 0.50), with a 64-bit
// division and one load in flight a thread and turn.
template <int KIND, int G>
__global__ void __launch_bounds__(256) w4_quant_kernel(const W4QuantArgs a)
{
    griddep_launch_dependents();
    griddep_wait();
    constexpr float MOST = KIND == FP8FG_E2M1 ? 6.0f : 7.0f;
    const int64_t per_row = a.K / 8, total = a.rows * per_row;
    // (a group's lanes run together to the loop's end: total and the stride are
    // multiples of the group's lanes)
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per_row, c = i - r * per_row;
        const uint4 v = *reinterpret_cast<const uint4 *>(a.w + r * a.ldw + c * 8);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        float f[8], amax = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f[2 * q] = bf16_lo(u[q]);
            f[2 * q + 1] = bf16_hi(u[q]);
            amax = fmaxf(amax, fmaxf(fabsf(f[2 * q]), fabsf(f[2 * q + 1])));
        }
        constexpr int LANES = G / 8;
        const unsigned mates = (LANES == 32 ? ALL : (1u << LANES) - 1) << (lane_id() & ~(LANES - 1));
#pragma unroll
        for (int d = LANES / 2; d; d >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(mates, amax, d));
        float inv = __fdiv_rn(MOST, amax), s = __fdiv_rn(amax, MOST);
        if (amax == 0.0f || isinf(inv))
            inv = s = 1.0f;
        uint32_t word = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float lo = f[2 * q] * inv, hi = f[2 * q + 1] * inv;
            if constexpr (KIND == FP8FG_E2M1) {
                uint32_t b;
                asm("{\n\t.reg .b8 p;\n\tcvt.rn.satfinite.e2m1x2.f32 p, %1, %2;\n\tcvt.u32.u8 %0, p;\n\t}" : "=r"(b) : "f"(hi), "f"(lo));
                word |= b << (8 * q);
            } else {
                const int x = max(-7, min(7, __float2int_rn(lo))), y = max(-7, min(7, __float2int_rn(hi)));
                word |= (uint32_t)((x & 15) | (y & 15) << 4) << (8 * q);
            }
        }
        *reinterpret_cast<uint32_t *>(a.q + (r * a.K + c * 8) / 2) = word;
        if (c % LANES == 0)
            a.scales[r * (a.K / G) + c / LANES] = s;
    }
}

bool aligned4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

bool w4_format_ok(int kind, int group, int64_t K)
{
    return (kind == FP8FG_E2M1 || kind == FP8FG_INT4) && (group == 32 || group == 64 || group == 128) && K % group == 0;
}

template <typename F>
int by_format(int kind, int group, F f)
{
    using std::integral_constant;
    auto with = [&](auto kd) {
        if (group == 32)
            return f(kd, integral_constant<int, 32>());
        if (group == 64)
            return f(kd, integral_constant<int, 64>());
        return f(kd, integral_constant<int, 128>());
    };
    return kind == FP8FG_E2M1 ? with(integral_constant<int, FP8FG_E2M1>()) : with(integral_constant<int, FP8FG_INT4>());
}

constexpr int W4_SMEM = 225 * 1024;

// Shared memory of a CTA beside the staged x.
template <typename Lay>
int fixed_smem(int ring, int cluster, int E)
{
    return WARPS * ring * Lay::STAGE + Lay::RED + (E + 4) / 4 * 32 + (cluster > 1 ? Lay::PARTS * Lay::UNIT_SUMS : 0) +
           16;
}

// Values of x that fit beside that: 2 bytes each, and 4 for every 128 of them.
template <typename Lay>
int64_t x_room(int ring, int cluster, int E)
{
    return (W4_SMEM - fixed_smem<Lay>(ring, cluster, E)) / (2 * STEP + 4) * STEP;
}

// With which `rows` rows of x fit whole (and a stage's columns of any tile's rows, for
// tiles that have more): the smallest cluster, and with that the deepest ring; the
// largest and the shallowest where none do.
struct Split {
    int ring, cluster;
    bool fits;
};

template <typename Lay>
Split split_for(int most, int least, int64_t rows, const W4Args &a)
{
    for (int cluster = 1;; cluster *= 2) {
        const int64_t span = (int64_t)((a.loads + cluster - 1) / cluster) * LOAD;
        for (int ring = most; ring >= least; --ring) {
            const int64_t room = x_room<Lay>(ring, cluster, a.E);
            if (room >= rows * (span + 32) && room >= Lay::TOKENS * (LOAD + 32))
                return {ring, cluster, true};
        }
        if (cluster == MAX_CLUSTER || 2 * cluster > a.loads)
            return {least, cluster, false};
    }
}

template <int KIND, int G, int NT, int P>
int launch_w4(W4Args a, const Split &split, const uint8_t *wq, cudaStream_t s)
{
    using Lay = Layout<G, NT, P>;
    auto kernel = w4_matvec_kernel<KIND, G, NT, P>;
    static std::atomic<uint64_t> allowed{0};
    if (!allow_smem(kernel, W4_SMEM, allowed))
        return FP8FG_ECUDA;
    const int outs = a.gated ? Lay::ROWS / 2 : Lay::ROWS;
    const int64_t units = (a.N + outs - 1) / outs;
    const int64_t tiles = (a.n_rows + Lay::TOKENS - 1) / Lay::TOKENS + (a.E < a.n_rows ? a.E : a.n_rows) - 1;
    if (tiles * units >= (1ll << 30))
        return FP8FG_EINVAL;
    a.units = (int)units;
    a.ring = split.ring;
    a.cluster = split.cluster;
    a.log_cluster = split.cluster == 8 ? 3 : split.cluster / 2;
    const int64_t room = x_room<Lay>(a.ring, a.cluster, a.E), rows = a.n_rows < MAX_STAGED ? a.n_rows : MAX_STAGED;
    if (room < Lay::TOKENS * (LOAD + 32))
        return FP8FG_EINVAL;  // (no size leads here)
    const int64_t all = rows * ((a.loads + a.cluster - 1) / a.cluster * LOAD + 32);
    a.x_halfs = (int)(room < all ? room : (all + STEP - 1) / STEP * STEP);
    a.fit_rows = (int)(a.x_halfs / ((a.loads + a.cluster - 1) / a.cluster * LOAD + 32));
    const int smem = fixed_smem<Lay>(a.ring, a.cluster, a.E) + (a.x_halfs / STEP + 3) / 4 * 16 + a.x_halfs * 2;
    // [columns][output rows][gate, up][experts]; a box is a unit's rows by a stage's columns
    const uint64_t dims[3] = {(uint64_t)a.N, a.gated ? 2u : 1u, (uint64_t)a.E};
    const uint64_t strides[3] = {1, (uint64_t)a.N, (uint64_t)a.wide};
    const uint32_t box[3] = {(uint32_t)outs, a.gated ? 2u : 1u, 1};
    CUtensorMap codes;
    if (!make_map_rows(&codes, wq, (uint64_t)a.K / 2, (uint64_t)a.K / 2, 3, dims, strides, LOAD / 2, box))
        return FP8FG_ECUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.cluster);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = a.cluster > 1 ? attr : attr + 1;
    cfg.numAttrs = 1;
    int64_t cap = sm_count() > 0 ? sm_count() : 1;
    if (a.cluster > 1) {  // as many as run at once (each CTA takes an SM's shared memory, whatever its x)
        static PerDevice running[4];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess)
            return FP8FG_ECUDA;
        cap = running[a.log_cluster].get(dev, [&] {
            cfg.dynamicSmemBytes = W4_SMEM;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                n = 0;
            }
            cfg.dynamicSmemBytes = smem;
            return n;
        });
        if (cap < 1)
            return FP8FG_ECUDA;
        cfg.numAttrs = 2;
    }
    const int64_t want = tiles * units;
    const unsigned clusters = (unsigned)(want < cap ? want : cap);
    a.by_units = divisor((uint32_t)units);
    a.by_clusters = divisor(clusters);
    if (!a.offsets)
        a.log_ks = share_warps((int)((a.n_rows + Lay::TOKENS - 1) / Lay::TOKENS * units + clusters - 1) / (int)clusters,
                               a.loads, a.log_cluster);
    cfg.gridDim = dim3(clusters * a.cluster);
    if (cudaLaunchKernelEx(&cfg, kernel, a, codes) != cudaSuccess) {
        cudaGetLastError();
        return FP8FG_ECUDA;
    }
    return launch_status();
}

}  // namespace
}  // namespace fp8fg

using namespace fp8fg;

extern "C" int fp8fg_w4_quant(const void *w, int64_t rows, int64_t K, int64_t ldw, int kind, int group, uint8_t *q,
                              float *scales, void *stream)
{
    if (rows < 0 || K < 0 || !w4_format_ok(kind, group, K) || ldw < K || rows >= (1ll << 40) || K >= (1ll << 22))
        return FP8FG_EINVAL;
    if (rows == 0 || K == 0)
        return FP8FG_OK;
    if (!w || !q || !scales)
        return FP8FG_EINVAL;
    if (!aligned16(w) || !aligned16(q) || ldw % 8 != 0 || !aligned4(scales))
        return FP8FG_EALIGN;
    if (!device_supported())
        return FP8FG_EUNSUPPORTED;
    const W4QuantArgs a = {static_cast<const uint16_t *>(w), ldw, rows, K, q, scales};
    const int64_t want = (rows * (K / 8) + 255) / 256, cap = 16ll * (sm_count() > 0 ? sm_count() : 1);
    const dim3 grid((unsigned)(want < cap ? want : cap));
    return by_format(kind, group, [&](auto kd, auto g) {
        return launch_pss(w4_quant_kernel<decltype(kd)::value, decltype(g)::value>, grid, 256, 0,
                          static_cast<cudaStream_t>(stream), a);
    });
}

extern "C" int fp8fg_w4_matvec(const void *x, int64_t ldx, int64_t T, const int32_t *row_index,
                               const int32_t *expert_offsets, int32_t n_experts, int64_t n_rows, const uint8_t *wq,
                               const float *sw, int kind, int group, int64_t N, int64_t K, int gated, void *y, int out,
                               int64_t ldy, void *stream)
{
    if ((out != FP8FG_OUT_F32 && out != FP8FG_OUT_BF16) || (gated != 0 && gated != 1) || T < 0 || n_rows < 0 || N < 0 ||
        K <= 0 || K >= (1ll << 22) || !w4_format_ok(kind, group, K) || n_experts < 1 || n_experts > MAX_EXPERTS || ldx < K ||
        ldy < N || N >= (1ll << 30) || n_rows >= (1ll << 31) || T >= (1ll << 31))
        return FP8FG_EINVAL;
    if (!expert_offsets && (n_experts != 1 || row_index))
        return FP8FG_EINVAL;
    if (!row_index && T < n_rows)
        return FP8FG_EINVAL;
    if (n_rows == 0 || N == 0)
        return FP8FG_OK;
    if (T == 0 || !x || !wq || !sw || !y)
        return FP8FG_EINVAL;
    const int64_t esz = out == FP8FG_OUT_F32 ? 4 : 2;
    if (!aligned16(x) || !aligned16(wq) || ldx % 8 != 0 || !aligned4(sw) || !aligned4(row_index) ||
        !aligned4(expert_offsets) || reinterpret_cast<uintptr_t>(y) % (uintptr_t)esz != 0)
        return FP8FG_EALIGN;
    if (!device_supported())
        return FP8FG_EUNSUPPORTED;
    W4Args a = {};
    a.x = static_cast<const uint16_t *>(x);
    a.ldx = ldx;
    a.T = T;
    a.row_index = row_index;
    a.offsets = expert_offsets;
    a.E = n_experts;
    a.n_rows = n_rows;
    a.wq = wq;
    a.sw = sw;
    a.wide = gated ? 2 * N : N;
    a.N = N;
    a.K = K;
    a.loads = (int)((K + LOAD - 1) / LOAD);
    a.y = y;
    a.ldy = ldy;
    a.out_f32 = out == FP8FG_OUT_F32;
    a.gated = gated;
    a.status = status_word_ptr();
    a.limit_ns = wait_limit_ns();
    a.skip_first_load = take_skip_first_load();
    // tiles of 8 rows, or 16 where that saves reading the weight again (of an expert
    // whose rows are few on average, some have more)
    const int64_t share = (n_rows + n_experts - 1) / n_experts;
    const bool small = expert_offsets ? share <= 4 || n_rows <= 8 : n_rows <= 8;
    // Units of 32 rows leave up to one in six SMs idle where there are fewer than six an SM,
    // units of 16 fewer. The limit is higher than it has to be. K = 7168, one row, us with
    // units of 16 and 32: 2048 weight rows 5.7 and 6.6, 7168 8.9 and 9.4, 8192 9.9 and 9.5,
    // 12288 14.8 and 11.8, 24320 23.0 and 21.4, 28672 22.9 and 22.1, 58368 42.4 and 36.9. Eight
    // rows do not fit beside units of 32 there.
    const bool narrow = a.wide * (n_rows < n_experts ? n_rows : n_experts) < 6ll * 32 * sm_count();
    return by_format(kind, group, [&](auto kd, auto g) {
        constexpr int KIND = decltype(kd)::value, G = decltype(g)::value;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        auto pick = [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            // (an expert has a token once at most, as a rule)
            const int64_t most = T < n_rows ? T : n_rows, rows = most < 8 * NT ? most : 8 * NT;
            const Split wide = split_for<Layout<G, NT, 2>>(2, 2, rows, a);
            if (narrow || !wide.fits || wide.cluster > 1)
                return launch_w4<KIND, G, NT, 1>(a, split_for<Layout<G, NT, 1>>(4, 2, rows, a), wq, s);
            return launch_w4<KIND, G, NT, 2>(a, wide, wq, s);
        };
        return small ? pick(std::integral_constant<int, 1>()) : pick(std::integral_constant<int, 2>());
    });
}
