// The rows of a mixture layer's experts back to tokens, and the gradient of that.
//   combine          : out[t] = sum_j w[t, j] y[pair_row[t, j]] (FP32 sum in slot order; w = 1 without
//                      weights, which is the backward pass of the gather into expert order)
//   combine_backward : dy[pair_row[t, j]] = w[t, j] dout[t]; dw[t, j] = sum_c dout[t, c] y[row, c]
// Pairs without a row add nothing and have zero gradient; a token without pairs gives zeros.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bounds_check.cuh"
#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kMaxK = 32;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack8(const float* f)
{
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                      pack_bf16(f[6], f[7]));
}

__device__ __forceinline__ float pair_weight(const CombineArgs& a, int64_t t, int j)
{
    return ld_checked(a.weights + t * a.map.k + j, a.weights, 4 * a.map.tokens * a.map.k, a.dev_status);
}

// Pairs whose rows are read together: eight loads in flight per thread.
constexpr int kTogether = 8;

// A CTA per token and slice of its columns; a thread takes 8 columns at a time.  Bound by HBM: B200,
// 8192 tokens x 8 rows of 4096 89 us (6.8 TB/s, the output still partly in L2); 103 us with the rows
// read one after another.
template <bool F32>
__global__ void __launch_bounds__(128) combine_kernel(const CombineArgs a)
{
    __shared__ int row[kMaxK];
    __shared__ float weight[kMaxK];
    const int64_t t = blockIdx.x;
    const int k = static_cast<int>(a.map.k);
    if (threadIdx.x < kMaxK) {
        const int r = threadIdx.x < k ? static_cast<int>(a.map.pair_target(t, threadIdx.x, a.rows)) : -1;
        row[threadIdx.x] = r;
        weight[threadIdx.x] = r >= 0 && a.weights ? pair_weight(a, t, threadIdx.x) : 1.0f;
    }
    __syncthreads();
    const int64_t ob = matrix_bytes(a.map.tokens, a.cols, a.ldo, F32 ? 4 : 2);
    const int64_t yb = bf16_matrix_bytes(a.rows, a.cols, a.ldy);
    const int64_t vecs = a.cols >> 3;
    for (int64_t v = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x; v < vecs;
         v += static_cast<int64_t>(gridDim.y) * blockDim.x) {
        float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        for (int j0 = 0; j0 < k; j0 += kTogether) {
            uint4 y[kTogether];
#pragma unroll
            for (int j = 0; j < kTogether; ++j) {
                const int r = row[j0 + j];
                y[j] = make_uint4(0, 0, 0, 0);
                if (r >= 0)
                    y[j] = ldg_checked(reinterpret_cast<const uint4*>(a.y + r * a.ldy) + v, a.y, yb,
                                       a.dev_status);
            }
#pragma unroll
            for (int j = 0; j < kTogether; ++j) {
                if (row[j0 + j] < 0) continue;  // adds nothing, whatever its weight
                float f[8];
                unpack8(y[j], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] += weight[j0 + j] * f[i];
            }
        }
        if (F32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + t * a.ldo) + 2 * v;
            st_checked(o, make_float4(sum[0], sum[1], sum[2], sum[3]), a.out, ob, a.dev_status);
            st_checked(o + 1, make_float4(sum[4], sum[5], sum[6], sum[7]), a.out, ob, a.dev_status);
        } else {
            st_checked(reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + t * a.ldo) + v,
                       pack8(sum), a.out, ob, a.dev_status);
        }
    }
}

// A CTA per token.  Its pairs are taken eight at a time: the thread's 8 columns of the gradient are
// read once for them, the pairs' columns of y together, and the eight dot products are reduced over
// the CTA in a fixed order.  The CTAs behind the tokens zero the rows without a token.  Bound by HBM:
// B200, 8192 tokens x 8 rows of 4096 201 us (5.7 TB/s), 4096 x 6 of 2048 45 us (4.8 TB/s); pair by pair
// the latter took 98 us.
template <bool F32>
__global__ void __launch_bounds__(128) combine_backward_kernel(const CombineArgs a)
{
    __shared__ float part[kMaxK][4];
    const int64_t vecs = a.cols >> 3;
    const int64_t yb = bf16_matrix_bytes(a.rows, a.cols, a.ldy);
    const int64_t db = bf16_matrix_bytes(a.rows, a.cols, a.lddy);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= a.map.tokens) {
        // a warp looks at 32 rows at once
        const int64_t used = a.map.used_rows(a.rows);
        const int64_t warps = (gridDim.x - a.map.tokens) * 4;
        for (int64_t r0 = 32 * ((blockIdx.x - a.map.tokens) * 4 + warp); r0 < used; r0 += 32 * warps) {
            const int64_t token = a.map.token_of(r0 + lane);  // used is a multiple of 128
            for (unsigned left = __ballot_sync(0xFFFFFFFFu, token < 0 || token >= a.map.tokens); left;
                 left &= left - 1) {
                uint4* d = reinterpret_cast<uint4*>(a.dy + (r0 + __ffs(left) - 1) * a.lddy);
                for (int64_t v = lane; v < vecs; v += 32)
                    st_checked(d + v, make_uint4(0, 0, 0, 0), a.dy, db, a.dev_status);
            }
        }
        return;
    }
    const int64_t t = blockIdx.x;
    const int k = static_cast<int>(a.map.k);
    __shared__ int row[kMaxK];
    __shared__ float weight[kMaxK];
    if (threadIdx.x < kMaxK) {
        const int r = threadIdx.x < k ? static_cast<int>(a.map.pair_target(t, threadIdx.x, a.rows)) : -1;
        row[threadIdx.x] = r;
        weight[threadIdx.x] = r >= 0 ? pair_weight(a, t, threadIdx.x) : 0.0f;
    }
    __syncthreads();
    const int64_t gb = matrix_bytes(a.map.tokens, a.cols, a.ldo, F32 ? 4 : 2);
    for (int j0 = 0; j0 < k; j0 += kTogether) {
        float dot[kTogether];
#pragma unroll
        for (int j = 0; j < kTogether; ++j) dot[j] = 0.0f;
        for (int64_t v = threadIdx.x; v < vecs; v += blockDim.x) {
            uint4 y[kTogether];
#pragma unroll
            for (int j = 0; j < kTogether; ++j) {
                const int r = row[j0 + j];
                if (r >= 0)
                    y[j] = ldg_checked(reinterpret_cast<const uint4*>(a.y + r * a.ldy) + v, a.y, yb,
                                       a.dev_status);
            }
            float g[8];
            if (F32) {
                const float4* p = reinterpret_cast<const float4*>(
                    static_cast<const float*>(a.dout) + t * a.ldo) + 2 * v;
                const float4 lo = ldg_checked(p, a.dout, gb, a.dev_status);
                const float4 hi = ldg_checked(p + 1, a.dout, gb, a.dev_status);
                g[0] = lo.x; g[1] = lo.y; g[2] = lo.z; g[3] = lo.w;
                g[4] = hi.x; g[5] = hi.y; g[6] = hi.z; g[7] = hi.w;
            } else {
                unpack8(ldg_checked(reinterpret_cast<const uint4*>(
                                        static_cast<const uint16_t*>(a.dout) + t * a.ldo) + v,
                                    a.dout, gb, a.dev_status), g);
            }
#pragma unroll
            for (int j = 0; j < kTogether; ++j) {
                const int r = row[j0 + j];
                if (r < 0) continue;
                float f[8], d[8];
                unpack8(y[j], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot[j] += g[i] * f[i];
                    d[i] = weight[j0 + j] * g[i];
                }
                st_checked(reinterpret_cast<uint4*>(a.dy + r * a.lddy) + v, pack8(d), a.dy, db,
                           a.dev_status);
            }
        }
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
#pragma unroll
            for (int s = 16; s; s >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], s);
            if (lane == 0) part[j0 + j][warp] = dot[j];
        }
    }
    __syncthreads();
    if (threadIdx.x < k)
        st_checked(a.dweights + t * k + threadIdx.x,
                   (part[threadIdx.x][0] + part[threadIdx.x][1]) +
                       (part[threadIdx.x][2] + part[threadIdx.x][3]),
                   a.dweights, 4 * a.map.tokens * k, a.dev_status);
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, bool f32, int sm_count, cudaStream_t s)
{
    // slices of 1024 columns when there are too few tokens to fill the SMs (B200, 16 tokens x 8 rows of
    // 4096: 2.1 us; a CTA per token 3.7)
    const int64_t slices = (a.cols / 8 + 127) / 128;
    int64_t y = (4 * sm_count + a.map.tokens - 1) / a.map.tokens;
    if (y > slices) y = slices;
    if (y < 1) y = 1;
    const dim3 grid(static_cast<unsigned>(a.map.tokens), static_cast<unsigned>(y));
    if (f32) combine_kernel<true><<<grid, 128, 0, s>>>(a);
    else     combine_kernel<false><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_combine_backward(const CombineArgs& a, bool f32, int sm_count, cudaStream_t s)
{
    const int64_t grid = a.map.tokens + (a.rows < sm_count ? a.rows : sm_count);
    if (f32) combine_backward_kernel<true><<<static_cast<unsigned>(grid), 128, 0, s>>>(a);
    else     combine_backward_kernel<false><<<static_cast<unsigned>(grid), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace nvfp4
