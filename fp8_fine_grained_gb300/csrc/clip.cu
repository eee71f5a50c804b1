// Global norm of a list of gradient tensors, and the tensors scaled so that
// it does not exceed max_norm.
//
//   norm = sqrt(sum over all tensors of g^2)
//   coef = min(1, max_norm / (norm + eps))
//   out  = g * coef
//
// Two streams over the data: the norm has to be known before the first
// element is written. 400 M FP32 elements take 728 us (4.8 GB, 6.6 TB/s or 0.97
// of the measured copy). The first kernel leaves one FP64 partial sum per CTA;
// every CTA of the second adds those up in the same order (a few KB from L2),
// so the result does not depend on the schedule and no third launch is needed.
// The second kernel walks the chunks backwards: what the first one read last
// is still in L2.
//
// The tensors' pointers and sizes travel in the kernels' parameters (no device
// table to copy). A tensor is cut into chunks of bytes whose vector loads start
// on a 16-byte boundary of its own; the elements before the first boundary
// belong to chunk 0. Chunks are dealt round-robin to the CTAs, a whole chunk in
// flight in each (UNROLL 16-byte loads per thread). CTAs per SM of the sums and
// of the scaling, with chunks of 64 and 32 KB, us in a loop of calls (one
// run of all four):
//                              2, 2    3, 2    2, 3    3, 3
//   400 M FP32 elements         744     734     778     763
//   30 M, in 120 tensors       63.3    63.1    59.2    59.1
//   1.5 M, in 120 tensors      10.9     9.5     9.6     9.5
// so the scaling takes 3 up to 256 MB (what the sums leave in L2 is then still a
// good part of it) and 2 beyond. Other chunks for 400 M: 32 and 32 KB 776, 32
// and 16 KB 777, 64 and 64 KB 760.
#include <cuda_bf16.h>

#include "host_common.h"
#include "ptx.cuh"

namespace fp8fg {
namespace {

constexpr int THREADS = 256;
constexpr int CTAS_PER_SM = 3;
constexpr int64_t SCALE_WIDE_BYTES = 256ll << 20;  // the scaling's third CTA up to here
constexpr int SUM_UNROLL = 16, SCALE_UNROLL = 8;
constexpr int chunk_bytes(int unroll) { return unroll * THREADS * 16; }
constexpr int MAX_TENSORS = 1024;  // per launch: 24 bytes + 4 each in the 32 KB of kernel parameters

template <int N>
struct Table {
    const void *g[N];
    void *out[N];
    int64_t n[N];            // elements; negative: bf16
    uint32_t first[N + 1];   // first chunk of each tensor
    int count;
    bool in_place;           // every tensor: out == g
};

struct Piece {
    const uint8_t *g;
    uint8_t *out;
    int64_t begin, end;  // elements of the chunk's vector part and tail
    int head;            // elements before `begin` that belong to it (chunk 0)
    bool bf16;
};

__host__ __device__ __forceinline__ int head_elements(const void *p, int esz)
{
    return (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / esz;
}

// Piece of a chunk. `cur` is the tensor of the CTA's previous chunk, mostly
// this one's too; else the last tensor with first <= chunk is searched for.
template <int N, int UNROLL>
__device__ __forceinline__ Piece piece_of(const Table<N> &tab, uint32_t chunk, int &cur)
{
    if (chunk < tab.first[cur] || chunk >= tab.first[cur + 1]) {
        int lo = 0, hi = tab.count;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tab.first[mid] <= chunk)
                lo = mid;
            else
                hi = mid;
        }
        cur = lo;
    }
    Piece q;
    q.bf16 = tab.n[cur] < 0;
    const int64_t n = q.bf16 ? -tab.n[cur] : tab.n[cur];
    q.g = static_cast<const uint8_t *>(tab.g[cur]);
    q.out = static_cast<uint8_t *>(tab.out[cur]);
    int64_t head = head_elements(q.g, q.bf16 ? 2 : 4);
    head = head < n ? head : n;
    const int64_t per = chunk_bytes(UNROLL) / (q.bf16 ? 2 : 4), at = (int64_t)(chunk - tab.first[cur]) * per;
    q.head = at == 0 ? (int)head : 0;
    q.begin = head + at;
    q.end = q.begin + per < n ? q.begin + per : n;
    return q;
}

// (The kernels here may start before the stream's previous kernel ends: nothing
// is read by the read-only path, which promises data that does not change while
// the grid runs.)
__device__ __forceinline__ float load_one(const uint8_t *p, int64_t i, bool bf16)
{
    return bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i])
                : reinterpret_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_one(uint8_t *p, int64_t i, bool bf16, float v)
{
    if (bf16)
        reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        reinterpret_cast<float *>(p)[i] = v;
}

__device__ __forceinline__ uint4 ld16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// s += the squares of 16 bytes
__device__ __forceinline__ float2 sq16(const uint4 &v, bool bf16, float2 s)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (bf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
            s = __ffma2_rn(f, f, s);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float2 f = make_float2(__uint_as_float(w[i]), __uint_as_float(w[i + 1]));
            s = __ffma2_rn(f, f, s);
        }
    }
    return s;
}

__device__ __forceinline__ uint4 mul16(const uint4 &v, bool bf16, float c)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bf16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(bf16_lo(w[i]) * c, bf16_hi(w[i]) * c);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            w[i] = __float_as_uint(__uint_as_float(w[i]) * c);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over the block, the same in every thread and for every launch.
__device__ __forceinline__ double block_sum(double v, double *part)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w)
        v += part[w];
    return v;
}

// Squares are FP32, summed in FP32 inside a chunk (eight sums of at most 16
// terms per thread, then those) and in FP64 beyond it.
template <int N>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM)
    sumsq_kernel(const __grid_constant__ Table<N> tab, double *partial)
{
    griddep_launch_dependents();
    griddep_wait();
    __shared__ double part[THREADS / 32];
    const uint32_t chunks = tab.first[tab.count];
    constexpr int UNROLL = SUM_UNROLL;
    double total = 0.0;
    int cur = 0;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Piece q = piece_of<N, UNROLL>(tab, c, cur);
        const int esz = q.bf16 ? 2 : 4, per = 16 / esz;
        const int64_t len = q.end - q.begin;
        const int vecs = len > 0 ? (int)(len / per) : 0;
        const uint8_t *src = q.g + q.begin * esz;
        uint4 v[UNROLL];
#pragma unroll
        for (int j = 0; j < UNROLL; ++j) {
            const int i = j * THREADS + threadIdx.x;
            v[j] = i < vecs ? ld16(src + i * 16) : make_uint4(0, 0, 0, 0);
        }
        float2 s2[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            s2[j] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < UNROLL; ++j)
            s2[j & 3] = sq16(v[j], q.bf16, s2[j & 3]);
        float s = ((s2[0].x + s2[0].y) + (s2[1].x + s2[1].y)) + ((s2[2].x + s2[2].y) + (s2[3].x + s2[3].y));
        const int tail = len > 0 ? (int)(len - (int64_t)vecs * per) : 0;
        if ((int)threadIdx.x < tail) {
            const float v = load_one(q.g, q.begin + (int64_t)vecs * per + threadIdx.x, q.bf16);
            s = fmaf(v, v, s);
        }
        if ((int)threadIdx.x < q.head) {
            const float v = load_one(q.g, threadIdx.x, q.bf16);
            s = fmaf(v, v, s);
        }
        total += (double)s;
    }
    total = block_sum(total, part);
    if (threadIdx.x == 0)
        partial[blockIdx.x] = total;
}

template <int N>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM)
    scale_kernel(const __grid_constant__ Table<N> tab, const double *partial, int n_partial,
                 float max_norm, float eps, float *norm_out)
{
    griddep_wait();
    __shared__ double part[THREADS / 32];
    double total = 0.0;
    for (int i = threadIdx.x; i < n_partial; i += THREADS)
        total += partial[i];
    total = block_sum(total, part);
    // root in FP32, of the sum brought into its range
    const float norm = total > 1e30 ? sqrtf((float)(total * 0x1p-200)) * 0x1p100f : sqrtf((float)total);
    const float ratio = max_norm / (norm + eps);
    const float coef = ratio > 1.0f ? 1.0f : ratio;  // a NaN norm gives NaN
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) {
        norm_out[0] = norm;
        norm_out[1] = coef;
    }
    if (coef == 1.0f && tab.in_place)
        return;
    constexpr int UNROLL = SCALE_UNROLL;
    const uint32_t chunks = tab.first[tab.count];
    int cur = 0;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Piece q = piece_of<N, UNROLL>(tab, chunks - 1 - c, cur);
        if (coef == 1.0f && q.out == q.g)
            continue;
        const int esz = q.bf16 ? 2 : 4, per = 16 / esz;
        const int64_t len = q.end - q.begin;
        // vector stores need the output on the input's 16-byte grid
        const bool same = ((reinterpret_cast<uintptr_t>(q.g) ^ reinterpret_cast<uintptr_t>(q.out)) & 15) == 0;
        const int vecs = len > 0 && same ? (int)(len / per) : 0;
        const uint8_t *src = q.g + q.begin * esz;
        uint8_t *dst = q.out + q.begin * esz;
        uint4 v[UNROLL];
#pragma unroll
        for (int j = 0; j < UNROLL; ++j) {
            const int i = j * THREADS + threadIdx.x;
            if (i < vecs)
                v[j] = ld16(src + i * 16);
        }
#pragma unroll
        for (int j = 0; j < UNROLL; ++j) {
            const int i = j * THREADS + threadIdx.x;
            if (i < vecs)
                __stcs(reinterpret_cast<uint4 *>(dst + i * 16), mul16(v[j], q.bf16, coef));
        }
        for (int64_t i = q.begin + (int64_t)vecs * per + threadIdx.x; i < q.end; i += THREADS)
            store_one(q.out, i, q.bf16, load_one(q.g, i, q.bf16) * coef);
        if ((int)threadIdx.x < q.head)
            store_one(q.out, threadIdx.x, q.bf16, load_one(q.g, threadIdx.x, q.bf16) * coef);
    }
    griddep_launch_dependents();  // (not on entry: the sums of a following call would start among these CTAs)
}

// CTAs of a launch: all resident at once.
int64_t grid_cap(int per_sm)
{
    const int sms = sm_count();
    return (int64_t)(sms > 0 ? sms : 1) * per_sm;
}

unsigned grid_of(int64_t chunks, int per_sm)
{
    const int64_t cap = grid_cap(per_sm);
    return (unsigned)(chunks < cap ? (chunks > 0 ? chunks : 1) : cap);
}

int64_t chunks_of(const fp8fg_grad &t, int unroll)
{
    const int esz = t.kind == FP8FG_OUT_BF16 ? 2 : 4;
    const int64_t body = (t.n - head_elements(t.g, esz)) * esz, per = chunk_bytes(unroll);
    return t.n == 0 ? 0 : (body > per ? (body + per - 1) / per : 1);
}

// Tensors [0, take) of one launch; their chunks fit in 31 bits
template <int N>
void fill(Table<N> &tab, const fp8fg_grad *t, int take, int unroll)
{
    uint32_t first = 0;
    tab.in_place = true;
    for (int i = 0; i < take; ++i) {
        tab.in_place = tab.in_place && (t[i].out == t[i].g || t[i].n == 0);
        tab.g[i] = t[i].g;
        tab.out[i] = t[i].out;
        tab.n[i] = t[i].kind == FP8FG_OUT_BF16 ? -t[i].n : t[i].n;
        tab.first[i] = first;
        first += (uint32_t)chunks_of(t[i], unroll);
    }
    tab.first[take] = first;
    tab.count = take;
}

// The smaller parameter block of a short list copies faster at the launch.
template <int N>
int launch_sumsq(const fp8fg_grad *t, int take, double *partial, int *used, cudaStream_t s)
{
    Table<N> tab;
    fill(tab, t, take, SUM_UNROLL);
    const unsigned grid = grid_of(tab.first[take], CTAS_PER_SM);
    *used = (int)grid;
    return launch_pss(sumsq_kernel<N>, dim3(grid), THREADS, 0, s, tab, partial);
}

template <int N>
int launch_scale(const fp8fg_grad *t, int take, const double *partial, int n_partial, float max_norm, float eps,
                 float *norm, cudaStream_t s)
{
    Table<N> tab;
    fill(tab, t, take, SCALE_UNROLL);
    const int64_t chunks = tab.first[take];
    const unsigned grid = grid_of(chunks, chunks * chunk_bytes(SCALE_UNROLL) <= SCALE_WIDE_BYTES ? CTAS_PER_SM : 2);
    return launch_pss(scale_kernel<N>, dim3(grid), THREADS, 0, s, tab, partial, n_partial, max_norm, eps, norm);
}

}  // namespace
}  // namespace fp8fg

using namespace fp8fg;

extern "C" int64_t fp8fg_grad_clip_workspace(int64_t count)
{
    if (count < 0)
        return 0;
    const int64_t launches = count > 0 ? (count + MAX_TENSORS - 1) / MAX_TENSORS : 1;
    return launches * grid_cap(CTAS_PER_SM) * 8;
}

extern "C" int fp8fg_grad_clip(const fp8fg_grad *grads, int64_t count, float max_norm, float eps, float *norm,
                               void *workspace, int64_t workspace_bytes, void *stream)
{
    if (count < 0 || count >= (1ll << 20) || !(max_norm >= 0.0f) || !(eps >= 0.0f) || !norm || !workspace ||
        (count > 0 && !grads))
        return FP8FG_EINVAL;
    if ((reinterpret_cast<uintptr_t>(norm) & 3u) != 0 || (reinterpret_cast<uintptr_t>(workspace) & 7u) != 0)
        return FP8FG_EALIGN;
    for (int64_t i = 0; i < count; ++i) {
        const fp8fg_grad &t = grads[i];
        if ((t.kind != FP8FG_OUT_F32 && t.kind != FP8FG_OUT_BF16) || t.n < 0 || t.n >= (1ll << 42) ||
            (t.n > 0 && (!t.g || !t.out)))
            return FP8FG_EINVAL;
        const uintptr_t mask = t.kind == FP8FG_OUT_BF16 ? 1u : 3u;
        if (t.n > 0 && (((reinterpret_cast<uintptr_t>(t.g) | reinterpret_cast<uintptr_t>(t.out)) & mask) != 0))
            return FP8FG_EALIGN;
    }
    if (!device_supported())
        return FP8FG_EUNSUPPORTED;
    if (workspace_bytes < fp8fg_grad_clip_workspace(count))
        return FP8FG_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    double *partial = static_cast<double *>(workspace);
    // launches of at most MAX_TENSORS tensors and 2^31 chunks
    int n_partial = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int64_t at = 0;
        do {
            const int take = (int)(count - at < MAX_TENSORS ? count - at : MAX_TENSORS);
            int64_t chunks = 0;
            for (int i = 0; i < take; ++i)
                chunks += chunks_of(grads[at + i], SCALE_UNROLL);
            if (chunks >= (1ll << 31))
                return FP8FG_EINVAL;
            int rc;
            if (pass == 0) {
                int used = 0;
                auto sums = take <= 64    ? launch_sumsq<64>
                            : take <= 256 ? launch_sumsq<256>
                                          : launch_sumsq<MAX_TENSORS>;
                rc = sums(grads + at, take, partial + n_partial, &used, s);
                n_partial += used;
            } else {
                float *out = at == 0 ? norm : nullptr;
                auto scaled = take <= 64    ? launch_scale<64>
                              : take <= 256 ? launch_scale<256>
                                            : launch_scale<MAX_TENSORS>;
                rc = scaled(grads + at, take, partial, n_partial, max_norm, eps, out, s);
            }
            if (rc != FP8FG_OK)
                return rc;
            at += take;
        } while (at < count);
    }
    return FP8FG_OK;
}
