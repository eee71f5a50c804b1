// The router of a mixture-of-experts layer, forward and backward.
//
// Forward: of every token's E logits the k best experts and their weights. The
// score s of an expert is the sigmoid or the softmax of its logit; a bias enters
// the choice (s + b), not the weight; the experts stand in groups, of which the
// best are kept (a group's value is the sum of its one or two best choices).
// Equal experts and groups go by the lower index:
//   - Without a bias the logits order the experts as their scores do, so they
//     are compared themselves: the order is that of real numbers. Sums of a group's
//     two best scores are computed in FP32 with a known error, and compared once more
//     in FP64 in rows where a kept group and a dropped one are closer than that: by 2
//     less the sum where it is above 1, by its logarithm where it underflows.
//   - With a bias the choices are computed in FP32 with a known error, and a row in
//     which two neighbours of the order (the chosen experts and the next one, or
//     the last kept group and the first dropped) are closer than that error is
//     decided once more in FP64, for the experts near the border alone (one to a
//     lane). Two experts of the same logit and bias are equal and not close. With
//     256 experts under one row in a hundred takes that path; all experts in FP64
//     (FP64 runs at a 64th of FP32's rate here) take 30 us for one row and are left
//     for rows in which more than 32 experts are close.
// Backward: the gradient of the logits from that of the weights; the choice and
// the bias get none. It needs the chosen logits alone, except where a softmax is
// not divided by its chosen part: there the whole row is read for its sum.
//
// A warp takes one token: its logits stand in the lanes' registers, expert i of
// lane l is 32 i + l. The chosen ones are found without k reductions in turn: the k
// largest of the lanes' own largest keys give a border, the dozen keys at or above it
// go to one lane each and are ranked against each other. Bound by the launch and the
// chain of shuffles (one token, 256 experts in 8 groups: 3.7 us, 2 of them the launch)
// and by some 1200 instructions a row where there are many (4096 tokens: 10 to 12 us for
// 4.5 MB, by how many rows FP64 decides; backward 4.0 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <type_traits>

#include "host_common.h"
#include "ptx.cuh"

namespace fp8fg {
namespace {

constexpr int ROUTE_WARPS = 4;
constexpr int ROUTE_MAX_E = 1024;
constexpr int ROUTE_MAX_K = 16;
constexpr int ROUTE_MAX_GROUPS = 32;
constexpr unsigned ALL = 0xFFFFFFFFu;

struct RouteArgs {
    const void *logits;
    int64_t ld;
    const float *bias;
    int64_t T;
    int E, k, score, groups, top_groups, group_top, renorm;
    uint32_t by_members;  // 2^22 / (E / groups), rounded up: exact quotients below 1024
    int log_lanes;        // lanes to a group
    float scale;
    int32_t *ids;
    float *gates;
};

template <typename L>
__device__ __forceinline__ float to_f32(L v)
{
    return (float)v;
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v)
{
    return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half v)
{
    return __half2float(v);
}

// A float as an unsigned number of the same order; 0 is below every number, and
// stands for minus infinity and NaN (an expert that cannot be chosen).
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (!(v > -CUDART_INF_F))
        return 0;
    const uint32_t u = __float_as_uint(v + 0.0f);  // (-0 is 0)
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// The group of expert e.
__device__ __forceinline__ int group_of(const RouteArgs &a, int e) { return (int)((uint32_t)e * a.by_members >> 22); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        v += __shfl_xor_sync(ALL, v, d);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        v = fmaxf(v, __shfl_xor_sync(ALL, v, d));
    return v;
}

// The least and the largest of the lanes' values (no NaN among them).
__device__ __forceinline__ float warp_least(float v)
{
    float r;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float warp_most(float v)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// exp(v - top); 1 for v = top, infinite or not
template <typename F>
__device__ __forceinline__ F exp_below(F v, F top)
{
    return v == top ? F(1) : exp(v - top);
}

template <typename F>
__device__ __forceinline__ F sigmoid(F v)
{
    return F(1) / (F(1) + exp(-v));
}

// A sigmoid for comparisons: off by less than 2^-21 (an exponential within 2^-22
// of itself with its argument's rounding, of which the sigmoid moves by a quarter
// and 0.28 times, and a reciprocal within 2^-23).
__device__ __forceinline__ float rough_sigmoid(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// The warp's values in descending order.
__device__ __forceinline__ uint32_t warp_sorted(uint32_t v)
{
    const int lane = (int)lane_id();
#pragma unroll
    for (int run = 2; run <= 32; run <<= 1)
#pragma unroll
        for (int d = run >> 1; d; d >>= 1) {
            const uint32_t w = __shfl_xor_sync(ALL, v, d);
            v = ((lane & d) == 0) == ((lane & run) == 0) ? max(v, w) : min(v, w);
        }
    return v;
}

// The weights of the chosen experts before the scale, lane j holding slot j's
// logit l (`in`: the slot is used). A softmax that is not divided by its chosen
// part takes the row's largest logit and its sum of exponentials.
__device__ __forceinline__ float slot_weight(float l, bool in, int score, bool renorm, float row_max, float row_sum)
{
    if (score == FP8FG_SOFTMAX) {
        if (!renorm)
            return in ? exp_below(l, row_max) / row_sum : 0.0f;
        const float top = warp_max(in ? l : -CUDART_INF_F);
        const float e = in ? exp_below(l, top) : 0.0f;
        return e / warp_sum(e);
    }
    if (!renorm)
        return in ? sigmoid(l) : 0.0f;
    // sigmoid(l) = exp(l - m) / (1 + exp(l)) exp(m), and exp(m) cancels in the
    // quotient: with m the largest logit, where that is below zero, the sum is
    // above a half whatever the logits are
    const float m = fminf(0.0f, warp_max(in ? l : -CUDART_INF_F));
    const float s = !in ? 0.0f : l > 0.0f ? sigmoid(l) : exp_below(l, m) / (1.0f + expf(l));
    return s / warp_sum(s);
}

// The order of a row in FP64, for rows that FP32 cannot order: lane j returns
// slot j's expert or -1.
template <typename L, int NE>
__device__ __noinline__ int choose_exactly(const RouteArgs &a, const L *row, double *buf)
{
    const int lane = (int)lane_id(), members = a.E / a.groups;
    const double low = -CUDART_INF;
    double s[NE], top = low;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 32 * i + lane;
        s[i] = e < a.E ? (double)to_f32(row[e]) : low;
        if (!(s[i] > low))
            s[i] = low;
        top = fmax(top, s[i]);
    }
    if (a.score == FP8FG_SOFTMAX) {
        double sum = 0;
        for (int d = 16; d; d >>= 1)
            top = fmax(top, __shfl_xor_sync(ALL, top, d));
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            s[i] = s[i] > low ? exp_below(s[i], top) : low;
            sum += s[i] > low ? s[i] : 0;
        }
        for (int d = 16; d; d >>= 1)
            sum += __shfl_xor_sync(ALL, sum, d);
#pragma unroll
        for (int i = 0; i < NE; ++i)
            s[i] /= sum;
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            s[i] = s[i] > low ? sigmoid(s[i]) : low;
    }
    unsigned kept = ALL;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 32 * i + lane;
        if (a.bias && e < a.E)
            s[i] += (double)a.bias[e];
        if (!(s[i] > low))
            s[i] = low;
        if (e < a.E)
            buf[e] = s[i];
    }
    __syncwarp();
    if (a.groups > 1) {
        double mine = low;  // lane g: group g's value
        for (int g = 0; g < a.groups; ++g) {
            double first = low, second = low;
            for (int m = lane; m < members; m += 32) {
                const double v = buf[g * members + m];
                second = fmax(second, fmin(first, v));
                first = fmax(first, v);
            }
            for (int d = 16; d; d >>= 1) {
                const double f = __shfl_xor_sync(ALL, first, d), t = __shfl_xor_sync(ALL, second, d);
                second = fmax(fmax(second, t), fmin(first, f));
                first = fmax(first, f);
            }
            if (lane == g)
                mine = a.group_top == 2 && second > low ? first + second : first;
        }
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double v = __shfl_sync(ALL, mine, g);
            rank += v > mine || (v == mine && g < lane);
        }
        kept = __ballot_sync(ALL, lane < a.groups && rank < a.top_groups);
    }
    int chosen = -1;
    for (int j = 0; j < a.k; ++j) {
        double best = low;
        int at = ROUTE_MAX_E;
        for (int e = lane; e < a.E; e += 32) {
            const double v = (kept >> (e / members)) & 1u ? buf[e] : low;
            if (v > best) {
                best = v;
                at = e;
            }
        }
        for (int d = 16; d; d >>= 1) {
            const double v = __shfl_xor_sync(ALL, best, d);
            const int i = __shfl_xor_sync(ALL, at, d);
            if (v > best || (v == best && i < at)) {
                best = v;
                at = i;
            }
        }
        if (!(best > low))
            break;
        if (lane == j)
            chosen = at;
        __syncwarp();
        if (lane == 0)
            buf[at] = low;
        __syncwarp();
    }
    return chosen;
}

// A double as an integer of the same order.
__device__ __forceinline__ long long order_key(double v)
{
    const long long u = __double_as_longlong(v + 0.0);
    return u ^ (u < 0 ? 0x7FFFFFFFFFFFFFFFll : 0);
}

// The choice of expert e in FP64.
template <typename L>
__device__ __forceinline__ double exact_choice(const RouteArgs &a, const L *row, int e, double top, double sum)
{
    const double l = (double)to_f32(row[e]), s = a.score == FP8FG_SOFTMAX ? exp_below(l, top) / sum : sigmoid(l);
    return a.bias ? s + (double)a.bias[e] : s;
}

// The order of a row whose FP32 choices `keys` are too close to each other
// somewhere: the experts near the border compared in FP64, and with `regroup` the
// groups too; without it, bit g << shift of `kept` says whether group g is kept. Lane j
// returns slot j's expert or -1; -2 in every lane where there are too many for that.
template <typename L, int NE>
__device__ __noinline__ int choose_near(const RouteArgs &a, const L *row, const uint32_t *keys, int32_t *list, float off,
                                        bool regroup, unsigned kept, int shift)
{
    const int lane = (int)lane_id(), members = a.E / a.groups;
    double top = -CUDART_INF, sum = 0;
    if (a.score == FP8FG_SOFTMAX) {
        for (int e = lane; e < a.E; e += 32)
            top = fmax(top, (double)to_f32(row[e]));  // (fmax passes a NaN over)
        for (int d = 16; d; d >>= 1)
            top = fmax(top, __shfl_xor_sync(ALL, top, d));
        for (int e = lane; e < a.E; e += 32) {
            const double l = (double)to_f32(row[e]);
            sum += l > -CUDART_INF ? exp_below(l, top) : 0;
        }
        for (int d = 16; d; d >>= 1)
            sum += __shfl_xor_sync(ALL, sum, d);
    }
    auto near = [&](float v) { return off + 0x1p-22f * fabsf(v); };

    if (regroup) {
        // lane g: group g's value, of its two best experts
        long long value = order_key(-CUDART_INF);
        bool close = false;
        if (lane < a.groups) {
            uint32_t k1 = 0, k2 = 0, k3 = 0;
            int e1 = 0, e2 = 0;
            for (int e = lane * members; e < (lane + 1) * members; ++e) {
                const uint32_t key = keys[e];
                if (key > k1) {
                    k3 = k2;
                    k2 = k1;
                    e2 = e1;
                    k1 = key;
                    e1 = e;
                } else if (key > k2) {
                    k3 = k2;
                    k2 = key;
                    e2 = e;
                } else {
                    k3 = max(k3, key);
                }
            }
            if (k1) {
                const float border = key_value(a.group_top == 2 && k2 ? k2 : k1);
                close = k3 && border - key_value(k3) <= near(border);
                const double c1 = exact_choice(a, row, e1, top, sum);
                double v = c1;
                if (k2) {
                    const double c2 = exact_choice(a, row, e2, top, sum);
                    v = a.group_top == 2 ? c1 + c2 : fmax(c1, c2);
                }
                value = order_key(v);
            }
        }
        if (__any_sync(ALL, close))
            return -2;
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const long long v = __shfl_sync(ALL, value, g);
            rank += v > value || (v == value && g < lane);
        }
        kept = __ballot_sync(ALL, lane < a.groups && rank < a.top_groups);
        shift = 0;
    }

    // the k-th choice in FP32, and the experts that may stand before it
    uint32_t key[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 32 * i + lane;
        key[i] = e < a.E && (kept >> (group_of(a, e) << shift) & 1u) ? keys[e] : 0;
    }
    uint32_t last = 0xFFFFFFFFu;
    for (int found = 0; found < a.k;) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            best = key[i] < last ? max(best, key[i]) : best;
        best = __reduce_max_sync(ALL, best);
        if (!best)
            break;
        unsigned same = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            same += key[i] == best;
        found += (int)__reduce_add_sync(ALL, same);
        last = best;
    }
    const float v = key_value(last), border = v - near(v);
    int count = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const bool in = key[i] && last != 0xFFFFFFFFu && !(key_value(key[i]) < border);
        const unsigned who = __ballot_sync(ALL, in);
        const int at = count + __popc(who & ((1u << lane) - 1));
        if (in && at < 32)
            list[at] = 32 * i + lane;
        count += __popc(who);
    }
    if (count > 32)
        return -2;
    __syncwarp();
    const int e = lane < count ? list[lane] : ROUTE_MAX_E;
    const long long mine = lane < count ? order_key(exact_choice(a, row, e, top, sum)) : order_key(-CUDART_INF);
    int rank = 0;
    for (int j = 0; j < count; ++j) {
        const long long w = __shfl_sync(ALL, mine, j);
        const int x = __shfl_sync(ALL, e, j);
        rank += w > mine || (w == mine && x < e);
    }
    __syncwarp();
    if (lane < count)
        list[rank] = e;
    __syncwarp();
    return lane < a.k && lane < count ? list[lane] : -1;
}

// log(sigmoid(v)), and log(sigmoid(v) + sigmoid(w)) of v >= w.
__device__ __forceinline__ double log_sigmoid(double v) { return fmin(v, 0.0) - log1p(exp(-fabs(v))); }

__device__ __forceinline__ double log_of_sum(double v, double w)
{
    const double p = log_sigmoid(v);
    return p > -CUDART_INF ? p + log1p(exp(log_sigmoid(w) - p)) : p;
}

// What the sum of the scores of a group's two best logits (keys, 0 for none) is compared
// by, as a real number: scores that underflow or come close to 1 count too. First an
// integer of the sum's order, then, where that is the same, the logits: of two that FP64
// cannot add up the larger one is in front.
struct SumOrder {
    long long value;
    unsigned long long logits;
};

// An integer of the order of a positive sum, 0 for 1; below 1e-300 that of its logarithm.
template <typename F>
__device__ __forceinline__ long long order_of_sum(double sum, F log_of_it)
{
    const long long one = order_key(1.0);
    return sum >= 1e-300 ? order_key(sum) - one : order_key(log_of_it()) - order_key(-690.0) - one;
}

__device__ __forceinline__ SumOrder sum_order(int score, uint32_t first, uint32_t second, float row_max)
{
    if (!first)
        return {order_key(-CUDART_INF), 0};
    const double v = (double)key_value(first), w = second ? (double)key_value(second) : -CUDART_INF;
    const unsigned long long logits = (unsigned long long)first << 32 | second;
    if (score == FP8FG_SOFTMAX) {
        if (row_max == CUDART_INF_F)  // (infinite logits share the row; the others' scores are 0)
            return {order_key((double)((v == CUDART_INF) + (w == CUDART_INF))), 0};
        const double top = (double)row_max;
        return {order_of_sum(exp(v - top) + exp(w - top), [&] { return v - top + log1p(exp(w - v)); }), logits};
    }
    if (v == -w)
        return {0, 0};  // the sum is 1
    const double ev = exp(-fabs(v)), ew = exp(-fabs(w)), rv = 1 / (1 + ev), rw = 1 / (1 + ew);
    const double sum = (v > 0 ? rv : ev * rv) + (w > 0 ? rw : ew * rw);
    if (sum <= 1)
        return {order_of_sum(sum, [&] { return log_of_sum(v, w); }), logits};
    // above 1: by 2 less the sum, that of the complements
    return {-order_of_sum((v > 0 ? ev * rv : rv) + (w > 0 ? ew * rw : rw), [&] { return log_of_sum(-w, -v); }), logits};
}

// The groups to keep by their sums of two scores, lane `g << log_lanes` and those behind
// it holding the keys of group g's two best logits: bit g << log_lanes of the result.
__device__ __noinline__ unsigned keep_by_sums(const RouteArgs &a, uint32_t first, uint32_t second, float row_max)
{
    const int g = (int)lane_id() >> a.log_lanes;
    const SumOrder sum = sum_order(a.score, first, second, row_max);
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
        const long long v = __shfl_sync(ALL, sum.value, h << a.log_lanes);
        const unsigned long long w = __shfl_sync(ALL, sum.logits, h << a.log_lanes);
        rank += v > sum.value || (v == sum.value && (w > sum.logits || (w == sum.logits && h < g)));
    }
    return __ballot_sync(ALL, g < a.groups && rank < a.top_groups);
}

template <typename L, int NE>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) route_kernel(const RouteArgs a)
{
    extern __shared__ double smem[];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = (int)lane_id(), warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp;
    if (t >= a.T)
        return;
    double *buf = smem + (size_t)warp * max(a.E, 64);  // (keys, and a list of 32 experts)
    const L *row = static_cast<const L *>(a.logits) + t * a.ld;

    float l[NE], b[NE];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NE; ++i)
        b[i] = a.bias && 32 * i + lane < a.E ? a.bias[32 * i + lane] : 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 32 * i + lane;
        l[i] = e < a.E ? to_f32(row[e]) : -CUDART_INF_F;
        nan |= isnan(l[i]);
    }
    nan = __any_sync(ALL, nan);

    // what the experts are compared by: the logits, or the choices
    const bool sums = a.groups > 1 && a.group_top == 2;
    const bool by_logit = !a.bias;
    const bool need_sum = a.score == FP8FG_SOFTMAX && (!by_logit || sums || !a.renorm);
    float row_max = 0.0f, row_sum = 1.0f;
    uint32_t key[NE];
    float e_of[NE];
    if (need_sum) {
        row_max = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            row_max = fmaxf(row_max, l[i]);  // (fmaxf passes a NaN over)
        row_max = warp_max(row_max);
        row_sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            e_of[i] = l[i] > -CUDART_INF_F ? exp_below(l[i], row_max) : 0.0f;
            row_sum += e_of[i];
        }
        row_sum = warp_sum(row_sum);
    }
    // (the error of a choice: below 2^-21 for a sigmoid, below 2^-18 of the
    // largest score for a softmax, whose sum adds up to 1024 terms; and half a
    // step of the sum with the bias. Two of them may be off in opposite ways.)
    const float off = a.score == FP8FG_SOFTMAX ? 0x1p-17f / row_sum : 0x1p-20f;
    const auto rough_score = [&](float v) {
        return a.score == FP8FG_SOFTMAX ? __fdividef(exp_below(v, row_max), row_sum) : rough_sigmoid(v);
    };
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 32 * i + lane;
        float c = l[i];
        if (!by_logit && c > -CUDART_INF_F) {
            c = a.score == FP8FG_SOFTMAX ? __fdividef(e_of[i], row_sum) : rough_sigmoid(c);
            c += b[i];
        }
        key[i] = order_key(c);
    }

    uint32_t *keys = reinterpret_cast<uint32_t *>(buf);
    if (!by_logit || a.groups > 1) {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (32 * i + lane < a.E)
                keys[32 * i + lane] = key[i];
        __syncwarp();
    }
    bool close = false, regroup = false;
    unsigned kept = 1;  // (one group)
    if (a.groups > 1) {
        // 2^log_lanes lanes to a group: each its best two, then those of all
        const int g = lane >> a.log_lanes, p = lane & ((1 << a.log_lanes) - 1), members = a.E / a.groups;
        uint32_t first = 0, second = 0;
        if (g < a.groups)
#pragma unroll 4
            for (int m = p; m < members; m += 1 << a.log_lanes) {
                const uint32_t v = keys[g * members + m];
                second = max(second, min(first, v));
                first = max(first, v);
            }
        for (int d = 1; d < 1 << a.log_lanes; d <<= 1) {
            const uint32_t f = __shfl_xor_sync(ALL, first, d), t = __shfl_xor_sync(ALL, second, d);
            second = max(max(second, t), min(first, f));
            first = max(first, f);
        }
        float best = first ? key_value(first) : -CUDART_INF_F, next = sums && second ? key_value(second) : 0.0f;
        if (by_logit && sums) {
            best = first ? rough_score(best) : best;
            next = second ? rough_score(next) : 0.0f;
        } else if (!by_logit) {  // (by a quarter, exactly: two of the largest or lowest numbers have a sum)
            best *= 0.25f;
            next *= 0.25f;
        }
        const float mine = best + next;
        int rank = 0;
#pragma unroll 4
        for (int h = 0; h < a.groups; ++h) {
            const float v = __shfl_sync(ALL, mine, h << a.log_lanes);
            rank += v > mine || (v == mine && h < g);
        }
        const bool keep = g < a.groups && rank < a.top_groups;
        kept = __ballot_sync(ALL, keep);
        if (a.top_groups < a.groups && (sums || !by_logit)) {
            // (a group's value is off by less than two scores' errors, half a step of each of
            // its two choices, however small their sum, and half a step of the sum; infinite
            // ones are exact)
            const float size = fabsf(best) + fabsf(next), err = fmaf(0x1p-22f, size, by_logit ? off : 0.25f * off);
            const bool finite = size < CUDART_INF_F;
            // the least that a kept group can be worth, the most that a dropped one can
            const float least = warp_least(keep && finite ? mine - err : CUDART_INF_F);
            const float most = warp_most(g < a.groups && !keep && finite ? mine + err : -CUDART_INF_F);
            regroup = least <= most;
        }
        if (by_logit && regroup) {
            regroup = false;
            kept = keep_by_sums(a, first, second, row_max);
        }
        // (beside an infinite logit the others' scores are equal)
        if (by_logit && sums && a.score == FP8FG_SOFTMAX && row_max == CUDART_INF_F) {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                key[i] = key[i] && key[i] != order_key(CUDART_INF_F) ? order_key(0.0f) : key[i];
        }
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (32 * i + lane < a.E && !(kept >> (group_of(a, 32 * i + lane) << a.log_lanes) & 1u))
                key[i] = 0;
    }

    // The chosen experts, and one more where the order can be in doubt. The last of
    // as many largest keys of the lanes is not above the last of the whole row's, so
    // keys below it are out; mostly a dozen are left, and stand one to a lane.
    const int picks = min(by_logit ? a.k : a.k + 1, 32);
    uint32_t most = key[0];
#pragma unroll
    for (int i = 1; i < NE; ++i)
        most = max(most, key[i]);
    const uint32_t least = max(__shfl_sync(ALL, warp_sorted(most), picks - 1), 1u);
    uint2 *list = reinterpret_cast<uint2 *>(buf) + (max(a.E, 64) + 1) / 2;  // behind the keys
    int count = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const unsigned who = __ballot_sync(ALL, key[i] >= least);
        const int at = count + __popc(who & ((1u << lane) - 1));
        if (key[i] >= least && at < 32)
            list[at] = make_uint2(key[i], 32 * i + lane);
        count += __popc(who);
    }
    __syncwarp();
    uint2 mine = make_uint2(0, 0);  // lane j: the j-th key, its expert
    if (count <= 32) {
        if (lane < count)
            mine = list[lane];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < count; ++j) {
            const uint32_t w = __shfl_sync(ALL, mine.x, j);
            rank += w > mine.x || (w == mine.x && j < lane);  // (the list is in the experts' order within a register)
        }
        __syncwarp();
        if (lane < count)
            list[rank] = mine;
        __syncwarp();
        mine = lane < min(count, picks) ? list[lane] : make_uint2(0, 0);
    } else {  // many equal keys: one after another
        for (int j = 0; j < picks; ++j) {
            uint32_t best = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = 32 * i + lane;
                }
            const uint32_t top = __reduce_max_sync(ALL, best);
            if (top == 0)
                break;
            const unsigned e = __reduce_min_sync(ALL, best == top ? (unsigned)at : ALL);
            if (lane == j)
                mine = make_uint2(top, e);
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (32 * i + lane == (int)e)
                    key[i] = 0;
        }
    }
    int chosen = mine.x && lane < a.k ? (int)mine.y : -1;
    if (!by_logit) {
        const uint32_t before = __shfl_up_sync(ALL, mine.x, 1);
        const int e = (int)mine.y, before_e = __shfl_up_sync(ALL, e, 1);
        if (lane > 0 && mine.x && key_value(before) - key_value(mine.x) <= off + 0x1p-22f * fabsf(key_value(mine.x)))
            close |= to_f32(row[e]) != to_f32(row[before_e]) || (a.bias && a.bias[e] != a.bias[before_e]);
        close = __any_sync(ALL, close);
    }
    if (close || regroup) {
        __syncwarp();
        chosen = choose_near<L, NE>(a, row, keys, reinterpret_cast<int32_t *>(keys + a.E), off, regroup, kept,
                                    a.log_lanes);
        if (__any_sync(ALL, chosen == -2)) {
            __syncwarp();
            chosen = choose_exactly<L, NE>(a, row, buf);
        }
    }

    const bool in = chosen >= 0;
    float g = a.scale * slot_weight(in ? to_f32(row[chosen]) : -CUDART_INF_F, in, a.score, a.renorm, row_max, row_sum);
    if (lane < a.k) {
        a.ids[t * a.k + lane] = chosen;
        a.gates[t * a.k + lane] = nan ? CUDART_NAN_F : in ? g : 0.0f;
    }
}

struct RouteBwdArgs {
    const float *dgates;
    const int32_t *ids;
    const void *logits;
    int64_t ld, T;
    int E, k, score, renorm;
    float scale;
    void *dlogits;
    int64_t ldd;
    int *status;
};

template <typename L>
__device__ __forceinline__ L from_f32(float v)
{
    return (L)v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v)
{
    return __float2half_rn(v);
}

template <typename L, int NE>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) route_bwd_kernel(const RouteBwdArgs a)
{
    extern __shared__ float rows[];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = (int)lane_id(), warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp;
    if (t >= a.T)
        return;
    const L *row = static_cast<const L *>(a.logits) + t * a.ld;
    L *out = static_cast<L *>(a.dlogits) + t * a.ldd;
    float *d_of = rows + (size_t)warp * a.E;  // the slots' part of the row's gradient

    int e = -1;
    float dg = 0.0f;
    if (lane < a.k) {
        e = a.ids[t * a.k + lane];
        dg = a.dgates[t * a.k + lane];
        if (e >= a.E) {
            atomicCAS(a.status, 0, FP8FG_EDEVICE);
            e = -1;
        }
    }
    const bool in = e >= 0;
    const float l = in ? to_f32(row[e]) : 0.0f;
    for (int i = lane; i < a.E; i += 32)
        d_of[i] = 0.0f;

    const bool whole = a.score == FP8FG_SOFTMAX && !a.renorm;
    float v[NE], row_max = 0.0f, row_sum = 1.0f;
    if (whole) {
        row_max = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            v[i] = 32 * i + lane < a.E ? to_f32(row[32 * i + lane]) : -CUDART_INF_F;
            row_max = fmaxf(row_max, v[i]);
        }
        row_max = warp_max(row_max);
        row_sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            v[i] = v[i] == -CUDART_INF_F ? 0.0f : exp_below(v[i], row_max);  // (a NaN stays one)
            row_sum += v[i];
        }
        row_sum = warp_sum(row_sum);
        row_sum = row_sum == 0.0f ? 1.0f : row_sum;  // (every expert masked: no gradient)
    }
    const float w = slot_weight(l, in, a.score, a.renorm, row_max, row_sum);
    const float mean = a.renorm || whole ? warp_sum(in ? dg * w : 0.0f) : 0.0f;
    float d = 0.0f;
    if (in) {
        if (a.score == FP8FG_SOFTMAX)
            d = a.renorm ? w * (dg - mean) : dg;
        else
            d = (a.renorm ? dg - mean : dg) * w * sigmoid(-l);
        d *= a.scale;
    }
    // slots of one expert add up, in slot order in each of them
    float sum = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const int ej = __shfl_sync(ALL, e, j);
        const float dj = __shfl_sync(ALL, d, j);
        if (ej == e)
            sum += dj;
    }
    __syncwarp();
    if (in)
        d_of[e] = sum;
    __syncwarp();
    if (whole) {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int x = 32 * i + lane;
            if (x < a.E)
                out[x] = from_f32<L>(v[i] / row_sum * (d_of[x] - a.scale * mean));
        }
    } else {
        for (int x = lane; x < a.E; x += 32)
            out[x] = from_f32<L>(d_of[x]);
    }
}

template <typename F>
int by_width(int E, F f)
{
    if (E <= 32)
        return f(std::integral_constant<int, 1>());
    if (E <= 64)
        return f(std::integral_constant<int, 2>());
    if (E <= 128)
        return f(std::integral_constant<int, 4>());
    if (E <= 256)
        return f(std::integral_constant<int, 8>());
    if (E <= 512)
        return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

template <typename F>
int by_type(int type, F f)
{
    if (type == FP8FG_F32)
        return f(float());
    if (type == FP8FG_BF16)
        return f(__nv_bfloat16());
    return f(__half());
}

int64_t type_size(int type) { return type == FP8FG_F32 ? 4 : 2; }

bool route_args_ok(int type, int64_t ld, int64_t T, int E, int k, int score, int renorm, float scale)
{
    return (type == FP8FG_F32 || type == FP8FG_BF16 || type == FP8FG_F16) && T >= 0 && T < (1ll << 31) && E >= 1 &&
           E <= ROUTE_MAX_E && k >= 1 && k <= ROUTE_MAX_K && k <= E && ld >= E &&
           (score == FP8FG_SIGMOID || score == FP8FG_SOFTMAX) && (renorm == 0 || renorm == 1) && isfinite(scale);
}

bool aligned_to(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)n == 0; }

}  // namespace
}  // namespace fp8fg

using namespace fp8fg;

extern "C" int fp8fg_moe_route(const void *logits, int type, int64_t ld, const float *bias, int64_t T, int E, int k,
                               int score, int groups, int top_groups, int group_top, int renorm, float scale,
                               int32_t *ids, float *gates, void *stream)
{
    if (!route_args_ok(type, ld, T, E, k, score, renorm, scale))
        return FP8FG_EINVAL;
    if (groups < 1 || groups > ROUTE_MAX_GROUPS || E % groups || top_groups < 1 || top_groups > groups ||
        group_top < 1 || group_top > 2 || k > top_groups * (E / groups))
        return FP8FG_EINVAL;
    if (T == 0)
        return FP8FG_OK;
    if (!logits || !ids || !gates)
        return FP8FG_EINVAL;
    if (!aligned_to(logits, type_size(type)) || !aligned_to(bias, 4) || !aligned_to(ids, 4) || !aligned_to(gates, 4))
        return FP8FG_EALIGN;
    if (!device_supported())
        return FP8FG_EUNSUPPORTED;
    const uint32_t members = (uint32_t)(E / groups);
    int log_lanes = 0;
    while (2 << log_lanes <= 32 / groups)
        ++log_lanes;
    const RouteArgs a = {logits,    ld,     bias,      T,     E,   k,    score, groups, top_groups,
                         group_top, renorm, ((1u << 22) + members - 1) / members, log_lanes, scale, ids, gates};
    const dim3 grid((unsigned)((T + ROUTE_WARPS - 1) / ROUTE_WARPS));
    const size_t smem = (size_t)ROUTE_WARPS * (E > 64 ? E : 64) * sizeof(double);
    return by_type(type, [&](auto l) {
        return by_width(E, [&](auto n) {
            return launch_pss(route_kernel<decltype(l), decltype(n)::value>, grid, ROUTE_WARPS * 32, smem,
                              static_cast<cudaStream_t>(stream), a);
        });
    });
}

extern "C" int fp8fg_moe_route_bwd(const float *dgates, const int32_t *ids, const void *logits, int type, int64_t ld,
                                   int64_t T, int E, int k, int score, int renorm, float scale, void *dlogits,
                                   int64_t ldd, void *stream)
{
    if (!route_args_ok(type, ld, T, E, k, score, renorm, scale) || ldd < E)
        return FP8FG_EINVAL;
    if (T == 0)
        return FP8FG_OK;
    if (!dgates || !ids || !logits || !dlogits)
        return FP8FG_EINVAL;
    if (!aligned_to(logits, type_size(type)) || !aligned_to(dlogits, type_size(type)) || !aligned_to(dgates, 4) ||
        !aligned_to(ids, 4))
        return FP8FG_EALIGN;
    if (!device_supported())
        return FP8FG_EUNSUPPORTED;
    const RouteBwdArgs a = {dgates, ids, logits, ld, T, E, k, score, renorm, scale, dlogits, ldd, status_word_ptr()};
    const dim3 grid((unsigned)((T + ROUTE_WARPS - 1) / ROUTE_WARPS));
    const size_t smem = (size_t)ROUTE_WARPS * E * sizeof(float);
    return by_type(type, [&](auto l) {
        return by_width(E, [&](auto n) {
            return launch_pss(route_bwd_kernel<decltype(l), decltype(n)::value>, grid, ROUTE_WARPS * 32, smem,
                              static_cast<cudaStream_t>(stream), a);
        });
    });
}
