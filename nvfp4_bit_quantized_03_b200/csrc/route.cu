// Routing of tokens to the experts of a mixture layer: the k experts of every token and their
// weights, the gradient of the weights, and the plan of the expert-ordered rows.
//
// Scores of a token's logits l: softmax s_e = exp(l_e - max l) / sum or sigmoid s_e = 1 / (1 +
// exp(-l_e)).  Experts are chosen by v_e = s_e + bias_e (the bias balances the load and does not
// enter the weights), optionally only among the experts of the top_groups groups whose two best v
// have the largest sum; ties go to the lowest index.  Weights w_j = scale * s_j, divided by the sum
// of the chosen scores when renormalised.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "bounds_check.cuh"
#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kRouteThreads = 128;
constexpr uint32_t kDevIndex = 8u;  // NVFP4_DEVSTAT_INDEX

// ---- order-preserving keys -----------------------------------------------------------------
// Unsigned integers in the order of the values (-0 and +0 equal); 0 is below every key and marks
// what cannot be chosen.
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ unsigned long long order_key(double v)
{
    const unsigned long long b = __double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k)
{
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(
        kAll, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return (static_cast<unsigned long long>(hi) << 32) | lo;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ float warp_maxf(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t* p)
{
    return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}

__device__ __forceinline__ float log_sigmoid(float x)
{
    return fminf(x, 0.0f) - log1pf(expf(-fabsf(x)));
}

// The r-th best of the warp's keys, r = 0 .. rounds - 1, best first: lane r of the result holds the
// expert (lane * NPL + i of its owner), -1 when nothing is left.  With `gap` also the smallest
// difference between consecutive values, up to the one after the last.
template <int NPL, typename Key>
__device__ __forceinline__ int select_best(Key (&key)[NPL], int rounds, int lane, float* gap)
{
    int mine = -1;
    float before = 0.0f;
    for (int r = 0; r < rounds + (gap ? 1 : 0); ++r) {
        Key best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const Key top = warp_max(best);
        if (top == 0) break;
        if constexpr (sizeof(Key) == 4) {
            if (gap) {
                const float v = key_value(top);
                if (r > 0) *gap = fminf(*gap, before - v);
                before = v;
            }
        }
        const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1;
        const int chosen = __shfl_sync(kAll, at, owner);
        if (r < rounds && lane == r) mine = owner * NPL + chosen;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (lane == owner && i == chosen) key[i] = 0;
    }
    return mine;
}

struct RouteArgs {
    const void* logits;
    const float* bias;
    int64_t ld;
    int T, E, k, groups, top_groups;
    bool sigmoid, renorm;
    float scale;
    int32_t* experts;
    float* weights;
    int* dev_status;
};

// Choice by scores in type F (float, or double where a float comparison is too close to call).
// x: the lane's logits (-inf: cannot be chosen), mx their warp maximum.  values: the warp's shared
// buffer of E group-search values.  Returns the chosen expert of lane j; close: a comparison was
// closer than the error of F (never set for double).
template <int NPL, typename F>
__device__ __forceinline__ int choose(const RouteArgs& a, const float (&x)[NPL], float mx, int lane,
                                      F* values, bool& close, bool& bad)
{
    using Key = decltype(order_key(F(0)));
    F s[NPL];
    F sum = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        if (sizeof(F) == 8)
            s[i] = a.sigmoid ? F(1) / (F(1) + F(exp(-double(x[i])))) : F(exp(double(x[i]) - double(mx)));
        else
            s[i] = a.sigmoid ? F(1) / (F(1) + F(expf(-x[i]))) : F(expf(x[i] - mx));
        sum += s[i];
    }
    if (!a.sigmoid) {
        sum = warp_sum(sum);
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] = s[i] / sum;
    }
    Key key[NPL];
    float largest = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane * NPL + i;
        key[i] = 0;
        if (e < a.E && x[i] > -INFINITY) {
            if (a.bias) s[i] += F(__ldg(a.bias + e));
            nan |= !(s[i] < F(INFINITY));
            if (s[i] > -F(INFINITY)) {
                key[i] = order_key(s[i]);
                largest = fmaxf(largest, fabsf(float(s[i])));
            }
        }
    }
    bad = __any_sync(kAll, nan);
    if (bad) return -1;
    // An FP32 score is off by at most 5 half-steps of 2^-24 (exp 2 ulp, sum, quotient, bias), of a
    // value no larger than 1 + largest; a softmax sum adds log2(32 NPL) more.  Differences below
    // 2^-19 of that are decided in FP64.
    const float tol = sizeof(F) == 8 ? 0.0f : 0x1p-19f * (1.0f + warp_maxf(largest));
    float gap = INFINITY;
    if (a.groups > 1) {
        const int size = a.E / a.groups;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane * NPL + i;
            if (e < a.E) values[e] = key[i] ? s[i] : -F(INFINITY);
        }
        __syncwarp();
        Key gkey[1] = {0};
        if (lane < a.groups) {
            F m1 = -F(INFINITY), m2 = -F(INFINITY);
            for (int i = 0; i < size; ++i) {
                const F v = values[lane * size + (i + lane) % size];
                if (v > m1) {
                    m2 = m1;
                    m1 = v;
                } else if (v > m2) {
                    m2 = v;
                }
            }
            if (m1 > -F(INFINITY)) gkey[0] = order_key(m2 > -F(INFINITY) ? m1 + m2 : m1);
        }
        __syncwarp();
        // sums of two have twice the error
        float ggap = INFINITY;
        const int g = select_best<1>(gkey, a.top_groups, lane, sizeof(F) == 8 ? nullptr : &ggap);
        gap = 0.5f * ggap;
        const unsigned kept = __reduce_or_sync(kAll, g >= 0 ? 1u << g : 0u);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane * NPL + i;
            if (e < a.E && !((kept >> (e / size)) & 1u)) key[i] = 0;
        }
    }
    const int mine = select_best<NPL>(key, a.k, lane, sizeof(F) == 8 ? nullptr : &gap);
    close = sizeof(F) == 4 && gap < tol;
    return mine;
}

// A warp per token; lane l holds the logits of experts l * NPL .. l * NPL + NPL - 1.
template <int NPL, typename T>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteArgs a)
{
    extern __shared__ double group_values[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * (kRouteThreads / 32) + warp;
    if (t >= a.T) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    float x[NPL];
    bool bad = false;
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane * NPL + i;
        x[i] = e < a.E ? load_logit(row + e) : -INFINITY;
        bad |= !(x[i] < INFINITY);
        mx = fmaxf(mx, x[i]);
    }
    bad = __any_sync(kAll, bad);
    mx = warp_maxf(mx);
    int expert = -1;
    if (!bad && mx > -INFINITY) {
        if (!a.bias && a.groups == 1) {
            // scores rise with the logits: the logits themselves are compared, exactly
            uint32_t key[NPL];
#pragma unroll
            for (int i = 0; i < NPL; ++i) key[i] = x[i] > -INFINITY ? order_key(x[i]) : 0u;
            expert = select_best<NPL>(key, a.k, lane, nullptr);
        } else {
            double* values = group_values + warp * a.E;
            bool close = false;
            expert = choose<NPL, float>(a, x, mx, lane, reinterpret_cast<float*>(values), close, bad);
            if (close && !bad) {
                bool never;
                expert = choose<NPL, double>(a, x, mx, lane, values, never, bad);
            }
        }
    }
    if (bad) {
        expert = -1;
        if (lane == 0 && a.dev_status) atomicOr(a.dev_status, static_cast<int>(kDevNonfinite));
    }
    const bool chosen = expert >= 0;
    const float l = chosen ? load_logit(row + expert) : -INFINITY;
    float w = 0.0f;
    if (a.renorm) {
        // shares exp(q - max q) / sum of the chosen log-scores q (up to a common constant): no
        // underflow however small the scores are
        const float q = a.sigmoid && chosen ? log_sigmoid(l) : l;
        const float top = warp_maxf(q);
        const float p = chosen ? expf(q - top) : 0.0f;
        const float sum = warp_sum(p);
        if (chosen) w = a.scale * (p / sum);
    } else if (a.sigmoid) {
        if (chosen) w = a.scale * (1.0f / (1.0f + expf(-l)));
    } else {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) sum += expf(x[i] - mx);
        sum = warp_sum(sum);
        if (chosen) w = a.scale * (expf(l - mx) / sum);
    }
    if (lane < a.k) {
        a.experts[static_cast<int64_t>(t) * a.k + lane] = expert;
        a.weights[static_cast<int64_t>(t) * a.k + lane] = w;
    }
}

struct RouteBackwardArgs {
    const void* logits;
    int64_t ld;
    const int32_t* experts;
    const float* dweights;
    int T, E, k;
    bool sigmoid, renorm;
    float scale;
    void* dlogits;
    int64_t ldd;
    int* dev_status;
};

// With S the chosen experts, p_j = s_j / sum_S s and g_j the gradient of w_j times the scale:
//   softmax, renormalised: dl_i = p_i (g_i - sum_S g p)          on S
//   softmax:               dl_e = s_e ([e in S] g_e - sum_S g s) everywhere
//   sigmoid, renormalised: dl_i = p_i (1 - s_i) (g_i - sum_S g p) on S
//   sigmoid:               dl_i = g_i s_i (1 - s_i)               on S
// A warp per token; lane j holds the j-th chosen expert.  A row without one has zero gradient.
template <int NPL, typename T>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(const RouteBackwardArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * (kRouteThreads / 32) + warp;
    if (t >= a.T) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    int expert = -1;
    float g = 0.0f, l = -INFINITY;
    if (lane < a.k) {
        expert = a.experts[static_cast<int64_t>(t) * a.k + lane];
        if (expert < -1 || expert >= a.E) {
            if (a.dev_status) atomicOr(a.dev_status, static_cast<int>(kDevIndex));
            expert = -1;
        }
        if (expert >= 0) {
            l = load_logit(row + expert);
            g = a.scale * a.dweights[static_cast<int64_t>(t) * a.k + lane];
        }
    }
    const bool chosen = expert >= 0;
    float out[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) out[i] = 0.0f;
    if (__any_sync(kAll, chosen)) {
        // 1 - sigmoid(l) = sigmoid(-l), without cancellation
        const float rest = a.sigmoid ? 1.0f / (1.0f + expf(l)) : 1.0f;
        float d = 0.0f;  // this lane's expert's part
        if (a.renorm) {
            const float q = a.sigmoid && chosen ? log_sigmoid(l) : l;
            const float top = warp_maxf(q);
            float p = chosen && q > -INFINITY ? expf(q - top) : 0.0f;
            const float sum = warp_sum(p);
            p = sum > 0.0f ? p / sum : 0.0f;
            const float mean = warp_sum(g * p);
            if (p > 0.0f) d = p * rest * (g - mean);
        } else if (a.sigmoid) {
            if (chosen) d = g * rest * (1.0f / (1.0f + expf(-l)));
        } else {
            float x[NPL];
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const int e = lane * NPL + i;
                x[i] = e < a.E ? load_logit(row + e) : -INFINITY;
                mx = fmaxf(mx, x[i]);
            }
            mx = warp_maxf(mx);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                x[i] = x[i] > -INFINITY ? expf(x[i] - mx) : 0.0f;
                sum += x[i];
            }
            sum = warp_sum(sum);
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            const float s = chosen && l > -INFINITY ? expf(l - mx) * inv : 0.0f;
            const float mean = warp_sum(g * s);
            d = g * s;
#pragma unroll
            for (int i = 0; i < NPL; ++i) out[i] = -(x[i] * inv) * mean;
        }
        for (int j = 0; j < a.k; ++j) {
            const int e = __shfl_sync(kAll, expert, j);
            const float dj = __shfl_sync(kAll, d, j);
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (e == lane * NPL + i) out[i] += dj;
        }
    }
    T* drow = static_cast<T*>(a.dlogits) + t * a.ldd;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane * NPL + i;
        if (e < a.E) {
            if constexpr (sizeof(T) == 4)
                drow[e] = out[i];
            else
                drow[e] = __bfloat16_as_ushort(__float2bfloat16_rn(out[i]));
        }
    }
}

// ---- the plan of the expert-ordered rows ---------------------------------------------------
// A stable counting sort of the pairs (t, j) by expert, regions padded to 128 rows.  A CTA takes
// kPlanPairs consecutive pairs, a warp an eighth of them in order.
constexpr int kPlanThreads = 256, kPlanWarps = kPlanThreads / 32;

struct PlanArgs {
    const int32_t* experts;
    int64_t pairs;
    int k, E;
    int64_t rows;
    int32_t* offsets;
    int32_t* pair_row;
    int32_t* row_token;
    int32_t* counts;  // [chunks][E] pairs of every chunk and expert (null: one chunk)
    int* dev_status;
};

__device__ __forceinline__ int pair_expert(const PlanArgs& a, int64_t i)
{
    const int e = a.experts[i];
    if (e >= 0 && e < a.E) return e;
    if (e != -1 && a.dev_status) atomicOr(a.dev_status, static_cast<int>(kDevIndex));
    return -1;
}

__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(const PlanArgs a)
{
    __shared__ int count[kMaxExperts];
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads) count[e] = 0;
    __syncthreads();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanPairs;
    for (int i = threadIdx.x; i < kPlanPairs; i += kPlanThreads)
        if (first + i < a.pairs) {
            const int e = pair_expert(a, first + i);
            if (e >= 0) atomicAdd(&count[e], 1);
        }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads)
        a.counts[static_cast<int64_t>(blockIdx.x) * a.E + e] = count[e];
}

__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(const PlanArgs a)
{
    __shared__ int next[kPlanWarps][kMaxExperts];  // pairs of each warp, then its next row
    __shared__ int total[kMaxExperts], before[kMaxExperts], start[kMaxExperts + 1];
    __shared__ int warp_sums[kPlanWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunk = blockIdx.x, chunks = gridDim.x;
    for (int i = threadIdx.x; i < kPlanWarps * kMaxExperts; i += kPlanThreads)
        next[i / kMaxExperts][i % kMaxExperts] = 0;
    __syncthreads();
    // the warp's share of the chunk, in order
    constexpr int kPerWarp = kPlanPairs / kPlanWarps;
    const int64_t first = static_cast<int64_t>(chunk) * kPlanPairs + warp * kPerWarp;
    int mine[kPerWarp / 32];
#pragma unroll
    for (int i = 0; i < kPerWarp / 32; ++i) {
        const int64_t p = first + 32 * i + lane;
        mine[i] = p < a.pairs ? pair_expert(a, p) : -1;
        if (mine[i] >= 0) atomicAdd(&next[warp][mine[i]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads) {
        int sum = 0, prior = 0;
        if (a.counts) {
            for (int c = 0; c < chunks; ++c) {
                const int n = a.counts[static_cast<int64_t>(c) * a.E + e];
                if (c < chunk) prior += n;
                sum += n;
            }
        } else {
            for (int w = 0; w < kPlanWarps; ++w) sum += next[w][e];
        }
        total[e] = sum;
        before[e] = prior;
    }
    __syncthreads();
    // region starts: exclusive scan of the padded counts, kMaxExperts / kPlanThreads per thread
    constexpr int kPer = kMaxExperts / kPlanThreads;
    int padded[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        padded[i] = e < a.E ? (total[e] + 127) / 128 * 128 : 0;
        sum += padded[i];
    }
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kAll, scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == 31) warp_sums[warp] = scan;
    __syncthreads();
    for (int w = 0; w < warp; ++w) scan += warp_sums[w];
    int at = scan - sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        if (e <= a.E) start[e] = at;
        at += padded[i];
    }
    if (threadIdx.x == kPlanThreads - 1 && a.E == kMaxExperts) start[a.E] = at;
    __syncthreads();
    if (chunk == 0)
        for (int e = threadIdx.x; e <= a.E; e += kPlanThreads) a.offsets[e] = start[e];
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads) {
        int row = start[e] + before[e];
        for (int w = 0; w < kPlanWarps; ++w) {
            const int n = next[w][e];
            next[w][e] = row;
            row += n;
        }
    }
    __syncthreads();
    // place 32 pairs at a time: equal experts in lane order
#pragma unroll
    for (int i = 0; i < kPerWarp / 32; ++i) {
        const int64_t p = first + 32 * i + lane;
        const unsigned same = __match_any_sync(kAll, mine[i]);
        int row = -1;
        if (mine[i] >= 0) row = next[warp][mine[i]] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (mine[i] >= 0 && lane == 31 - __clz(same)) next[warp][mine[i]] = row + 1;
        __syncwarp();
        if (p < a.pairs) {
            a.pair_row[p] = row;
            if (row >= 0 && row < a.rows) a.row_token[row] = static_cast<int32_t>(p / a.k);
        }
    }
    // rows without a token: the ends of the regions, and everything behind the last
    for (int e = chunk; e < a.E; e += chunks)
        for (int r = start[e] + total[e] + threadIdx.x; r < start[e + 1]; r += kPlanThreads)
            a.row_token[r] = -1;
    for (int64_t r = start[a.E] + static_cast<int64_t>(chunk) * kPlanThreads + threadIdx.x; r < a.rows;
         r += static_cast<int64_t>(chunks) * kPlanThreads)
        a.row_token[r] = -1;
}

template <typename T>
cudaError_t launch_route_t(const RouteArgs& a, cudaStream_t s)
{
    const int warps = kRouteThreads / 32;
    const int grid = (a.T + warps - 1) / warps;
    const size_t smem = a.groups > 1 ? sizeof(double) * warps * a.E : 0;
    if (a.E <= 32)       route_kernel<1, T><<<grid, kRouteThreads, smem, s>>>(a);
    else if (a.E <= 64)  route_kernel<2, T><<<grid, kRouteThreads, smem, s>>>(a);
    else if (a.E <= 128) route_kernel<4, T><<<grid, kRouteThreads, smem, s>>>(a);
    else if (a.E <= 256) route_kernel<8, T><<<grid, kRouteThreads, smem, s>>>(a);
    else                 route_kernel<16, T><<<grid, kRouteThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_route_backward_t(const RouteBackwardArgs& a, cudaStream_t s)
{
    const int warps = kRouteThreads / 32;
    const int grid = (a.T + warps - 1) / warps;
    if (a.E <= 32)       route_backward_kernel<1, T><<<grid, kRouteThreads, 0, s>>>(a);
    else if (a.E <= 64)  route_backward_kernel<2, T><<<grid, kRouteThreads, 0, s>>>(a);
    else if (a.E <= 128) route_backward_kernel<4, T><<<grid, kRouteThreads, 0, s>>>(a);
    else if (a.E <= 256) route_backward_kernel<8, T><<<grid, kRouteThreads, 0, s>>>(a);
    else                 route_backward_kernel<16, T><<<grid, kRouteThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route(const void* logits, bool bf16, int64_t T, int64_t E, int64_t ld,
                         const float* bias, bool sigmoid, bool renorm, int groups, int top_groups,
                         int k, float scale, int32_t* experts, float* weights, int* dev_status,
                         cudaStream_t s)
{
    RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.ld = ld;
    a.T = static_cast<int>(T);
    a.E = static_cast<int>(E);
    a.k = k;
    a.groups = groups;
    a.top_groups = top_groups;
    a.sigmoid = sigmoid;
    a.renorm = renorm;
    a.scale = scale;
    a.experts = experts;
    a.weights = weights;
    a.dev_status = dev_status;
    return bf16 ? launch_route_t<uint16_t>(a, s) : launch_route_t<float>(a, s);
}

cudaError_t launch_route_backward(const void* logits, bool bf16, int64_t T, int64_t E, int64_t ld,
                                  const int32_t* experts, const float* dweights, bool sigmoid,
                                  bool renorm, int k, float scale, void* dlogits, int64_t ldd,
                                  int* dev_status, cudaStream_t s)
{
    RouteBackwardArgs a;
    a.logits = logits;
    a.ld = ld;
    a.experts = experts;
    a.dweights = dweights;
    a.T = static_cast<int>(T);
    a.E = static_cast<int>(E);
    a.k = k;
    a.sigmoid = sigmoid;
    a.renorm = renorm;
    a.scale = scale;
    a.dlogits = dlogits;
    a.ldd = ldd;
    a.dev_status = dev_status;
    return bf16 ? launch_route_backward_t<uint16_t>(a, s) : launch_route_backward_t<float>(a, s);
}

cudaError_t launch_plan(const int32_t* experts, int64_t pairs, int k, int E, int64_t rows,
                        int32_t* offsets, int32_t* pair_row, int32_t* row_token, int32_t* counts,
                        int* dev_status, cudaStream_t s)
{
    PlanArgs a;
    a.experts = experts;
    a.pairs = pairs;
    a.k = k;
    a.E = E;
    a.rows = rows;
    a.offsets = offsets;
    a.pair_row = pair_row;
    a.row_token = row_token;
    a.dev_status = dev_status;
    const int chunks = static_cast<int>((pairs + kPlanPairs - 1) / kPlanPairs);
    a.counts = chunks > 1 ? counts : nullptr;
    if (chunks > 1) {
        plan_count_kernel<<<chunks, kPlanThreads, 0, s>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    plan_place_kernel<<<chunks, kPlanThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace nvfp4
