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
// Unsigned integers in the order of the values (-0 and +0 equal).  Keys below kFirstKey (-inf, and 0
// for what has been taken or excluded) cannot be chosen; a +inf or NaN is at or above kBadKey.
constexpr uint32_t kFirstKey = 0x00800000u, kBadKey = 0xFF800000u;
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

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(uint16_t v)
{
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// A buffer and its size in bytes, which the debug build holds every access against.
struct Buffer {
    const void* base;
    int64_t bytes;
    int* dev_status;

    template <typename T>
    __device__ __forceinline__ T ldg(const T* p) const { return ldg_checked(p, base, bytes, dev_status); }
    template <typename T>
    __device__ __forceinline__ T load(const T* p) const { return ld_checked(p, base, bytes, dev_status); }
    template <typename T>
    __device__ __forceinline__ void store(T* p, const T& v) const
    {
        st_checked(p, v, base, bytes, dev_status);
    }
};

template <typename T>
__device__ __forceinline__ float load_logit(const T* p, const Buffer& in) { return to_float(in.ldg(p)); }

// The lane's NPL values of a row of E (-inf behind its end), in loads of up to 16 bytes when the
// rows allow them (`wide`).
template <int NPL, typename T>
__device__ __forceinline__ void load_values(const T* row, int lane, int E, bool wide, float (&x)[NPL],
                                            const Buffer& in)
{
    constexpr int BYTES = NPL * static_cast<int>(sizeof(T));
    if (wide && (lane + 1) * NPL <= E) {
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int c = 0; c < BYTES / 16; ++c) {
                const uint4 v = in.ldg(reinterpret_cast<const uint4*>(row + lane * NPL) + c);
                if constexpr (sizeof(T) == 4) {
                    x[4 * c] = __uint_as_float(v.x);
                    x[4 * c + 1] = __uint_as_float(v.y);
                    x[4 * c + 2] = __uint_as_float(v.z);
                    x[4 * c + 3] = __uint_as_float(v.w);
                } else {
                    unpack8(v, x + 8 * c);
                }
            }
            return;
        } else if constexpr (BYTES == 8) {
            const uint2 v = in.ldg(reinterpret_cast<const uint2*>(row + lane * NPL));
            if constexpr (sizeof(T) == 4) {
                x[0] = __uint_as_float(v.x);
                x[1] = __uint_as_float(v.y);
            } else {
                x[0] = bf16_lo(v.x);
                x[1] = bf16_hi(v.x);
                x[2] = bf16_lo(v.y);
                x[3] = bf16_hi(v.y);
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane * NPL + i;
        x[i] = e < E ? load_logit(row + e, in) : -INFINITY;
    }
}

__device__ __forceinline__ float log_sigmoid(float x)
{
    return fminf(x, 0.0f) - log1pf(expf(-fabsf(x)));
}

// The r-th best of the warp's keys, r = 0 .. rounds - 1, best first: lane r of the result holds the
// expert (lane * NPL + i of its owner), -1 when nothing is left.  Exact for any key.
template <int NPL, typename Key>
__device__ __forceinline__ int select_best(Key (&key)[NPL], int rounds, int lane)
{
    int mine = -1;
    for (int r = 0; r < rounds; ++r) {
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
        const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1;
        const int chosen = __shfl_sync(kAll, at, owner);
        if (lane == r) mine = owner * NPL + chosen;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (lane == owner && i == chosen) key[i] = 0;
    }
    return mine;
}

// The same, faster, on 32-bit keys whose lowest log2(NPL) bits give way to the place in the lane
// (NPL - 1 - i, so that equal keys come in the order of their places).  Each lane sorts its keys
// once (Batcher's odd-even merge sort); a round then compares the lanes' first ones, and the lowest
// lane that holds the best writes it down and moves up.
template <int NPL>
__device__ __forceinline__ void pack_and_sort(uint32_t (&key)[NPL])
{
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        key[i] = (key[i] & ~(NPL - 1u)) | static_cast<uint32_t>(NPL - 1 - i);
#pragma unroll
    for (int p = 1; p < NPL; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j + q < NPL; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < NPL && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t a = key[i + j], b = key[i + j + q];
                        key[i + j] = max(a, b);
                        key[i + j + q] = min(a, b);
                    }
}
// close: two consecutive values (the one after the last round included) are no further apart than
// `error` times 1 + the larger magnitude.
template <int NPL>
__device__ __forceinline__ int take_best(uint32_t (&key)[NPL], int rounds, int lane, uint2* found,
                                         float error, bool& close)
{
    constexpr uint32_t kPlace = NPL - 1u;
    const uint32_t lower = (1u << lane) - 1u;
#pragma unroll 3
    for (int r = 0; r <= rounds; ++r) {
        const uint32_t first = key[0] & ~kPlace;
        const uint32_t top = __reduce_max_sync(kAll, first);
        const unsigned holders = __ballot_sync(kAll, first == top);
        if (first == top && !(holders & lower)) {
            found[r] = make_uint2(top, lane * NPL + (kPlace - (key[0] & kPlace)));
#pragma unroll
            for (int i = 0; i + 1 < NPL; ++i) key[i] = key[i + 1];
            key[NPL - 1] = 0;
        }
    }
    __syncwarp();
    // lane r looks at the values of rounds r and r + 1
    int mine = -1;
    bool near = false;
    if (lane < rounds) {
        const uint2 a = found[lane];
        const uint32_t next = found[lane + 1].x;
        if (a.x >= kFirstKey) mine = static_cast<int>(a.y);
        if (next >= kFirstKey) {
            const float u = key_value(a.x), v = key_value(next);
            near = !(u - v > error * (1.0f + fmaxf(fabsf(u), fabsf(v))));
        }
    }
    close = __any_sync(kAll, near);
    return mine;
}

struct RouteArgs {
    const void* logits;
    const float* bias;
    int64_t ld;
    int T, E, k, groups, top_groups;
    bool sigmoid, renorm;
    bool wide;         // logits (and bias) can be read 16 bytes at a time
    int group_lanes;   // lanes that hold one group, a power of two; 0: groups end inside lanes
    float scale;
    int32_t* experts;
    float* weights;
    int* dev_status;

    template <typename L>
    __device__ __forceinline__ Buffer logits_buffer() const
    {
        return Buffer{logits, matrix_bytes(T, E, ld, sizeof(L)), dev_status};
    }
    __device__ __forceinline__ Buffer bias_buffer() const
    {
        return Buffer{bias, static_cast<int64_t>(4) * E, dev_status};
    }
    // of a T x k output
    __device__ __forceinline__ Buffer per_pair(const void* base) const
    {
        return Buffer{base, static_cast<int64_t>(4) * T * k, dev_status};
    }
};

// Fast choice by FP32 scores s + bias.  close: some comparison was too close to call, and the choice
// has to be made in FP64.  An FP32 score is off by at most 10 units of 2^-23 (exp by its
// intrinsic: 2 + 1.2 |d| units at an argument d, times s; the sum of up to 512; the quotient; the
// bias), and the keys give way up to 15 units of the value to the place: two values are told
// apart from 2^-18 of 1 + the larger on, sums of two from twice that.  bad: a value was NaN or
// +inf.
constexpr float kScoreError = 0x1p-18f;

template <int NPL>
__device__ __forceinline__ int choose_fast(const RouteArgs& a, const float (&x)[NPL], float mx,
                                           int lane, uint2* found, bool& close, bool& bad)
{
    constexpr uint32_t kPlace = NPL - 1u;
    float s[NPL];
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] = __fdividef(1.0f, 1.0f + __expf(-x[i]));
    } else {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            s[i] = __expf(x[i] - mx);
            sum += s[i];
        }
        const float inv = 1.0f / warp_sum(sum);
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] *= inv;
    }
    if (a.bias) {
        float b[NPL];
        load_values<NPL>(a.bias, lane, a.E, a.wide, b, a.bias_buffer());
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] += b[i];
    }
    uint32_t key[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) key[i] = order_key(x[i] > -INFINITY ? s[i] : -INFINITY);
    pack_and_sort<NPL>(key);
    bad = __any_sync(kAll, (key[0] & ~kPlace) >= kBadKey);
    if (bad) return -1;
    bool close_groups = false;
    if (a.groups > 1) {
        // the group's two best: the lane's own, then across the group's lanes
        uint32_t m1 = key[0], m2 = NPL > 1 ? key[NPL > 1 ? 1 : 0] : 0u;
        for (int d = 1; d < a.group_lanes; d <<= 1) {
            const uint32_t o1 = __shfl_xor_sync(kAll, m1, d), o2 = __shfl_xor_sync(kAll, m2, d);
            m2 = max(min(m1, o1), max(m2, o2));
            m1 = max(m1, o1);
        }
        const float v1 = key_value(m1 & ~kPlace), v2 = key_value(m2 & ~kPlace);
        const bool any = m1 >= kFirstKey, two = m2 >= kFirstKey;
        const float score = any ? (two ? v1 + v2 : v1) : -INFINITY;
        // rank of this lane's group among all
        const int mine = lane / a.group_lanes;
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const float o = __shfl_sync(kAll, score, g * a.group_lanes);
            rank += (o > score || (o == score && g < mine)) ? 1 : 0;
        }
        const bool kept = rank < a.top_groups;
        const uint32_t okey = any ? order_key(score) : 0u;
        const uint32_t low = __reduce_min_sync(kAll, kept && any ? okey : 0xFFFFFFFFu);
        const uint32_t high = __reduce_max_sync(kAll, kept || mine >= a.groups ? 0u : okey);
        const uint32_t size =
            __reduce_max_sync(kAll, any ? __float_as_uint(fabsf(v1) + (two ? fabsf(v2) : 0.0f)) : 0u);
        if (high && low != 0xFFFFFFFFu)
            close_groups = !(key_value(low) - key_value(high) >
                             2.0f * kScoreError * (1.0f + __uint_as_float(size)));
        if (!kept) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) key[i] = 0;
        }
    }
    const int mine = take_best<NPL>(key, a.k, lane, found, kScoreError, close);
    close |= close_groups;
    return mine;
}

// The choice in FP64, for groups of any size: for comparisons too close for FP32, and for every token
// where groups end inside lanes.  values: the warp's shared buffer of E.  Bound by instruction issue
// (73 % of the slots): 2785 instructions a token of 160 experts.  B200, 16384 tokens, sigmoid, bias, 4 of 8 groups, k 8, FP64
// for all: 160 experts 56 us, 192 57, 320 133, 384 140 (against the fast choice at 128 16, at 256 21).
template <int NPL>
__device__ __forceinline__ int choose_exact(const RouteArgs& a, const float (&x)[NPL], float mx,
                                         int lane, double* values, bool& bad)
{
    double s[NPL], sum = 0.0;
    unsigned long long key[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        s[i] = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(x[i])))
                         : exp(static_cast<double>(x[i]) - static_cast<double>(mx));
        sum += s[i];
    }
    if (!a.sigmoid) {
        sum = warp_sum(sum);
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] /= sum;
    }
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        key[i] = 0;
        if (x[i] > -INFINITY) {  // false behind the last expert too
            if (a.bias) s[i] += a.bias_buffer().ldg(a.bias + lane * NPL + i);
            nan |= !(s[i] < INFINITY);
            if (s[i] > -INFINITY) key[i] = order_key(s[i]);
        }
    }
    bad = __any_sync(kAll, nan);
    if (bad) return -1;
    if (a.groups > 1) {
        const int size = a.E / a.groups;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane * NPL + i;
            if (e < a.E) values[e] = key[i] ? s[i] : -INFINITY;
        }
        __syncwarp();
        unsigned long long gkey[1] = {0};
        if (lane < a.groups) {
            double m1 = -INFINITY, m2 = -INFINITY;
            for (int i = 0; i < size; ++i) {
                const double v = values[lane * size + i];
                if (v > m1) {
                    m2 = m1;
                    m1 = v;
                } else if (v > m2) {
                    m2 = v;
                }
            }
            if (m1 > -INFINITY) gkey[0] = order_key(m2 > -INFINITY ? m1 + m2 : m1);
        }
        __syncwarp();
        const int g = select_best<1>(gkey, a.top_groups, lane);
        const unsigned kept = __reduce_or_sync(kAll, g >= 0 ? 1u << g : 0u);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane * NPL + i;
            if (e < a.E && !((kept >> (e / size)) & 1u)) key[i] = 0;
        }
    }
    return select_best<NPL>(key, a.k, lane);
}

// A warp per token; lane l holds the logits of experts l * NPL .. l * NPL + NPL - 1, so that the
// lowest lane with a value has the lowest index and a row is read in 16-byte loads.  B200: 16384 x
// 256 FP32 logits, sigmoid, bias, 4 of 8 groups, k 8: 21-22 us (51 us with the rounds searching unsorted
// keys and exact scores; 26 with the FP64 choice in a function of its own, which keeps the logits in
// local memory).  A token takes 848 instructions (scores 160, sort 40, groups 90, k + 1 rounds of about
// 20, weights 100), together 12 us of issue: the slots are 77 % busy for the 16.5 us that an SM has
// work, the rest of them waits in the rounds' chain of reduce, ballot and shift; launch, first loads and
// the last CTAs are the other 5 us.  Without bias and groups, k 8: FP32 11.6 us, bf16 11.0; one token 2.6
// us, a launch.
template <int NPL, typename T>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteArgs a)
{
    extern __shared__ double group_values[];
    __shared__ uint2 found[kRouteThreads / 32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * (kRouteThreads / 32) + warp;
    if (t >= a.T) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    const Buffer in = a.logits_buffer<T>();
    float x[NPL];
    load_values<NPL>(row, lane, a.E, a.wide, x, in);
    bool bad = false;
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        bad |= !(x[i] < INFINITY);
        mx = fmaxf(mx, x[i]);
    }
    bad = __any_sync(kAll, bad);
    mx = key_value(__reduce_max_sync(kAll, order_key(mx)));
    int expert = -1;
    if (!bad && mx > -INFINITY) {
        if (!a.bias && a.groups == 1) {
            // scores rise with the logits: the logits themselves are compared.  The packed keys
            // hold a bf16 exactly; FP32 logits that differ in their last bits only are told apart
            // by the whole keys.
            uint32_t key[NPL];
#pragma unroll
            for (int i = 0; i < NPL; ++i) key[i] = order_key(x[i]);
            pack_and_sort<NPL>(key);
            bool equal;
            expert = take_best<NPL>(key, a.k, lane, found[warp], 0.0f, equal);
            if (sizeof(T) == 4 && equal) {
#pragma unroll
                for (int i = 0; i < NPL; ++i) key[i] = x[i] > -INFINITY ? order_key(x[i]) : 0u;
                expert = select_best<NPL>(key, a.k, lane);
            }
        } else {
            bool close = a.group_lanes == 0;
            if (!close) expert = choose_fast<NPL>(a, x, mx, lane, found[warp], close, bad);
            if (close && !bad)
                expert = choose_exact<NPL>(a, x, mx, lane, group_values + warp * a.E, bad);
        }
    }
    if (bad) {
        expert = -1;
        if (lane == 0 && a.dev_status) atomicOr(a.dev_status, static_cast<int>(kDevNonfinite));
    }
    const bool chosen = expert >= 0;
    const float l = chosen ? load_logit(row + expert, in) : -INFINITY;
    float w = 0.0f;
    if (a.renorm) {
        float p = a.sigmoid && chosen ? 1.0f / (1.0f + expf(-l)) : 0.0f;
        float sum = a.sigmoid ? warp_sum(p) : 0.0f;
        if (sum < 0x1p-100f) {
            // softmax, or sigmoids near underflow: shares exp(q - max q) / sum of the chosen
            // log-scores q (up to a common constant), exact however small the scores are
            const float q = a.sigmoid && chosen ? log_sigmoid(l) : l;
            const float top = warp_maxf(q);
            p = chosen ? expf(q - top) : 0.0f;
            sum = warp_sum(p);
        }
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
        const int64_t at = static_cast<int64_t>(t) * a.k + lane;
        a.per_pair(a.experts).store(a.experts + at, expert);
        a.per_pair(a.weights).store(a.weights + at, w);
    }
}

struct RouteBackwardArgs {
    const void* logits;
    int64_t ld;
    const int32_t* experts;
    const float* dweights;
    int T, E, k;
    bool sigmoid, renorm;
    bool wide;  // logits and dlogits can be read and written 16 bytes at a time
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
// Renormalised weights need only the chosen logits, so a row is written and, but for them, not
// read.  B200, 8192 x 128 bf16, k 8: 4.2 us (softmax; not renormalised 4.6), of which a launch is 2.
template <int NPL, typename T>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(const RouteBackwardArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * (kRouteThreads / 32) + warp;
    if (t >= a.T) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    const Buffer in{a.logits, matrix_bytes(a.T, a.E, a.ld, sizeof(T)), a.dev_status};
    const int64_t pairs_bytes = static_cast<int64_t>(4) * a.T * a.k;
    int expert = -1;
    float g = 0.0f, l = -INFINITY;
    if (lane < a.k) {
        expert = ld_checked(a.experts + static_cast<int64_t>(t) * a.k + lane, a.experts, pairs_bytes,
                            a.dev_status);
        if (expert < -1 || expert >= a.E) {
            if (a.dev_status) atomicOr(a.dev_status, static_cast<int>(kDevIndex));
            expert = -1;
        }
        if (expert >= 0) {
            l = load_logit(row + expert, in);
            g = a.scale * ld_checked(a.dweights + static_cast<int64_t>(t) * a.k + lane, a.dweights,
                                     pairs_bytes, a.dev_status);
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
            load_values<NPL>(row, lane, a.E, a.wide, x, in);
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < NPL; ++i) mx = fmaxf(mx, x[i]);
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
    const Buffer to{a.dlogits, matrix_bytes(a.T, a.E, a.ldd, sizeof(T)), a.dev_status};
    if constexpr (NPL * sizeof(T) >= 16) {
        if (a.wide && (lane + 1) * NPL <= a.E) {
            constexpr int PER = 16 / sizeof(T);
#pragma unroll
            for (int c = 0; c < NPL / PER; ++c) {
                uint32_t w[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if constexpr (sizeof(T) == 4) {
                        w[h] = __float_as_uint(out[PER * c + h]);
                    } else {
                        const __nv_bfloat162 v =
                            __floats2bfloat162_rn(out[PER * c + 2 * h], out[PER * c + 2 * h + 1]);
                        w[h] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                }
                to.store(reinterpret_cast<uint4*>(drow + lane * NPL) + c,
                         make_uint4(w[0], w[1], w[2], w[3]));
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane * NPL + i;
        if (e < a.E) {
            if constexpr (sizeof(T) == 4)
                to.store(drow + e, out[i]);
            else
                to.store(drow + e, __bfloat16_as_ushort(__float2bfloat16_rn(out[i])));
        }
    }
}

// ---- the plan of the expert-ordered rows ---------------------------------------------------
// A stable counting sort of the pairs (t, j) by expert, regions padded to 128 rows.  A CTA takes
// kPlanPairs consecutive pairs, a warp an eighth of them in order; more pairs are counted by a pass
// ahead, whose counts a scan, or with few chunks each CTA for itself, adds up.  Integer counts only,
// so the order of the atomics does not show.  A chain of short latencies: B200, 131072 pairs of 256
// experts 11.4 us in all, one token 3.2 us.
constexpr int kPlanThreads = 256, kPlanWarps = kPlanThreads / 32;

struct PlanArgs {
    const int32_t* experts;
    int64_t pairs;
    int k, E;
    int64_t rows;
    int32_t* offsets;
    int32_t* pair_row;
    int32_t* row_token;
    // [chunks][E] pairs of every chunk and expert (null: one chunk).  With `scanned` those of the
    // chunks before, and a row more with those of all.
    int32_t* counts;
    bool scanned;
    int* dev_status;

    __device__ __forceinline__ Buffer pairs_buffer(const void* base) const
    {
        return Buffer{base, 4 * pairs, dev_status};
    }
    __device__ __forceinline__ Buffer rows_buffer() const { return Buffer{row_token, 4 * rows, dev_status}; }
    __device__ __forceinline__ Buffer counts_buffer(int chunks) const
    {
        return Buffer{counts, static_cast<int64_t>(4) * (chunks + (scanned ? 1 : 0)) * E, dev_status};
    }
};

__device__ __forceinline__ int pair_expert(const PlanArgs& a, int64_t i)
{
    const int e = a.pairs_buffer(a.experts).load(a.experts + i);
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
        a.counts_buffer(gridDim.x).store(a.counts + static_cast<int64_t>(blockIdx.x) * a.E + e, count[e]);
}

// counts -> those of the chunks before, and the totals behind them: a CTA takes 32 experts (one per
// lane), its warps consecutive shares of the chunks.
__global__ void __launch_bounds__(1024) plan_scan_kernel(const PlanArgs a, int chunks)
{
    __shared__ int sums[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const int share = (chunks + 31) / 32, first = warp * share;
    const int last = first + share < chunks ? first + share : chunks;
    int32_t* column = a.counts + e;
    const Buffer counts = a.counts_buffer(chunks);
    int sum = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int c = first; c < last; ++c) sum += counts.load(column + static_cast<int64_t>(c) * a.E);
    }
    sums[warp][lane] = sum;
    __syncthreads();
    int at = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
        if (w < warp) at += sums[w][lane];
        all += sums[w][lane];
    }
    if (e < a.E) {
        for (int c = first; c < last; ++c) {
            int32_t* p = column + static_cast<int64_t>(c) * a.E;
            const int n = counts.load(p);
            counts.store(p, at);
            at += n;
        }
        if (warp == 0) counts.store(column + static_cast<int64_t>(chunks) * a.E, all);
    }
}

__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(const PlanArgs a)
{
    extern __shared__ int next[];  // [kPlanWarps][E] pairs of each warp, then its next row
    __shared__ int total[kMaxExperts], before[kMaxExperts], start[kMaxExperts + 1];
    __shared__ int warp_sums[kPlanWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunk = blockIdx.x, chunks = gridDim.x;
    const Buffer counts = a.counts_buffer(chunks), tokens = a.rows_buffer();
    int* warp_next = next + warp * a.E;
    for (int i = threadIdx.x; i < kPlanWarps * a.E; i += kPlanThreads) next[i] = 0;
    __syncthreads();
    // the warp's share of the chunk, in order
    constexpr int kPerWarp = kPlanPairs / kPlanWarps;
    const int64_t first = static_cast<int64_t>(chunk) * kPlanPairs + warp * kPerWarp;
    int mine[kPerWarp / 32];
#pragma unroll
    for (int i = 0; i < kPerWarp / 32; ++i) {
        const int64_t p = first + 32 * i + lane;
        mine[i] = p < a.pairs ? pair_expert(a, p) : -1;
        if (mine[i] >= 0) atomicAdd(&warp_next[mine[i]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads) {
        int sum = 0, prior = 0;
        if (a.scanned) {
            prior = counts.load(a.counts + static_cast<int64_t>(chunk) * a.E + e);
            sum = counts.load(a.counts + static_cast<int64_t>(chunks) * a.E + e);
        } else if (a.counts) {
#pragma unroll
            for (int c = 0; c < kPlanScan; ++c) {
                if (c >= chunks) break;
                const int n = counts.load(a.counts + static_cast<int64_t>(c) * a.E + e);
                if (c < chunk) prior += n;
                sum += n;
            }
        } else {
            for (int w = 0; w < kPlanWarps; ++w) sum += next[w * a.E + e];
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
        for (int e = threadIdx.x; e <= a.E; e += kPlanThreads)
            st_checked(a.offsets + e, start[e], a.offsets, static_cast<int64_t>(4) * (a.E + 1),
                       a.dev_status);
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads) {
        int row = start[e] + before[e];
        for (int w = 0; w < kPlanWarps; ++w) {
            const int n = next[w * a.E + e];
            next[w * a.E + e] = row;
            row += n;
        }
    }
    __syncthreads();
    // place 32 pairs at a time: equal experts in lane order
#pragma unroll
    for (int i = 0; i < kPerWarp / 32; ++i) {
        const int64_t p = first + 32 * i + lane;
        if (first + 32 * i >= a.pairs) break;  // the whole warp
        const unsigned same = __match_any_sync(kAll, mine[i]);
        int row = -1;
        if (mine[i] >= 0) row = warp_next[mine[i]] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (mine[i] >= 0 && lane == 31 - __clz(same)) warp_next[mine[i]] = row + 1;
        __syncwarp();
        if (p < a.pairs) {
            a.pairs_buffer(a.pair_row).store(a.pair_row + p, row);
            if (row >= 0 && row < a.rows) tokens.store(a.row_token + row, static_cast<int32_t>(p / a.k));
        }
    }
    // rows without a token: the ends of the regions, and everything behind the last
    for (int e = chunk * kPlanWarps + warp; e < a.E; e += chunks * kPlanWarps)
        for (int r = start[e] + total[e] + lane; r < start[e + 1]; r += 32) tokens.store(a.row_token + r, -1);
    for (int64_t r = start[a.E] + static_cast<int64_t>(chunk) * kPlanThreads + threadIdx.x; r < a.rows;
         r += static_cast<int64_t>(chunks) * kPlanThreads)
        tokens.store(a.row_token + r, -1);
}

template <typename T>
cudaError_t launch_route_t(const RouteArgs& a, cudaStream_t s)
{
    const int warps = kRouteThreads / 32;
    const unsigned grid = (static_cast<unsigned>(a.T) + warps - 1) / warps;  // T up to 2^31 - 1
    const size_t smem = a.groups > 1 ? sizeof(double) * warps * a.E : 0;  // choose_exact's
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
    const unsigned grid = (static_cast<unsigned>(a.T) + warps - 1) / warps;  // T up to 2^31 - 1
    if (a.E <= 32)       route_backward_kernel<1, T><<<grid, kRouteThreads, 0, s>>>(a);
    else if (a.E <= 64)  route_backward_kernel<2, T><<<grid, kRouteThreads, 0, s>>>(a);
    else if (a.E <= 128) route_backward_kernel<4, T><<<grid, kRouteThreads, 0, s>>>(a);
    else if (a.E <= 256) route_backward_kernel<8, T><<<grid, kRouteThreads, 0, s>>>(a);
    else                 route_backward_kernel<16, T><<<grid, kRouteThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// Rows that start on 16-byte boundaries.
bool rows_aligned(const void* p, int64_t ld, int64_t esize)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * esize % 16 == 0;
}

// Experts per lane of the kernels' variants.
int per_lane(int64_t E) { return E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : E <= 256 ? 8 : 16; }

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
    a.wide = rows_aligned(logits, ld, bf16 ? 2 : 4) && (!bias || rows_aligned(bias, 0, 4));
    const int npl = per_lane(E), size = static_cast<int>(E / groups), lanes = size / npl;
    a.group_lanes = groups == 1 ? 1 : (size % npl == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0);
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
    a.wide = rows_aligned(logits, ld, bf16 ? 2 : 4) && rows_aligned(dlogits, ldd, bf16 ? 2 : 4);
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
    a.scanned = chunks >= kPlanScan;
    if (chunks > 1) plan_count_kernel<<<chunks, kPlanThreads, 0, s>>>(a);
    if (a.scanned) plan_scan_kernel<<<(E + 31) / 32, 1024, 0, s>>>(a, chunks);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    plan_place_kernel<<<chunks, kPlanThreads, sizeof(int) * kPlanWarps * E, s>>>(a);
    return cudaGetLastError();
}

}  // namespace nvfp4
