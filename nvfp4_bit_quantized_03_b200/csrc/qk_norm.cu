// Norms of queries and keys for each head, with the position rotation in the same pass, and the
// gradient of both.  Per head of D values x, weight w, angles of the token's position p:
//   r = 1 / sqrt(mean x^2 + eps),  n = r x,  y = w n,  z = y with its first `rotary` values turned in pairs
//   backward: dy = dz turned back,  dw = sum dy n,  dn = w dy,  dx = r (dn - n mean(dn n))
// All in FP32; the only rounding to fewer bits is the one of the outputs to their type.
//
// A lane holds a unit of 16 values of a head, two chunks of 8: both halves of 8 rotated pairs
// (chunks 8 u and rotary / 2 + 8 u, or the 16 neighbours 16 u .. when the pairs are neighbours), or 16
// neighbours behind the rotated part.  So a pair never leaves its lane, a lane stores only where it
// has loaded (outputs may be the inputs), and the mean is one reduction over the head's lanes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "bounds_check.cuh"
#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kWarps = 4;  // warps per CTA
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kDevIndex = 8;  // NVFP4_DEVSTAT_INDEX

template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t at, int64_t bytes, int* status, float* f)
{
    if (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        const float4 a = ld_checked(p, base, bytes, status), b = ld_checked(p + 1, base, bytes, status);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        unpack8(ld_checked(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at), base,
                           bytes, status), f);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t at, int64_t bytes, int* status, const float* f)
{
    if (F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
        st_checked(p, make_float4(f[0], f[1], f[2], f[3]), base, bytes, status);
        st_checked(p + 1, make_float4(f[4], f[5], f[6], f[7]), base, bytes, status);
    } else {
        st_checked(reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at),
                   make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])),
                   base, bytes, status);
    }
}

// 16 values of an array of one FP32 per value of a head (a weight; 1 without one).
__device__ __forceinline__ void load_weight(const float* w, int c0, int c1, int D, int* status, float* f)
{
    if (!w) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = 1.0f;
        return;
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float4 v = ldg_checked(reinterpret_cast<const float4*>(w + (h < 2 ? c0 : c1) + 4 * (h & 1)), w,
                                     4 * D, status);
        f[4 * h] = v.x; f[4 * h + 1] = v.y; f[4 * h + 2] = v.z; f[4 * h + 3] = v.w;
    }
}

// The place of a lane: its head among those a warp takes together, its unit of that head.
struct Place {
    int slot, c0, c1;  // c0, c1: first values of the unit's two chunks
    bool in, turned;   // the head has this unit; its values are rotated
};
__device__ __forceinline__ Place place(const HeadsArgs& a, bool interleaved, int lane)
{
    const int u = lane & (a.lanes - 1);
    Place p;
    p.slot = lane / a.lanes;
    p.in = 16 * u < a.D;
    p.turned = 16 * u < a.rotary;
    p.c0 = interleaved || !p.turned ? 16 * u : 8 * u;
    p.c1 = interleaved || !p.turned ? 16 * u + 8 : a.rotary / 2 + 8 * u;
    return p;
}

// Cosines and sines of the unit's 8 pairs at the token's position; false for a token without one.
__device__ __forceinline__ bool load_angles(const HeadsArgs& a, int64_t t, const Place& p, int lane, float* c,
                                            float* s)
{
    int64_t at = t;
    if (a.positions) at = ld_checked(a.positions + t, a.positions, 4 * a.tokens, a.dev_status);
    if (at < 0) return false;
    if (a.rotary && at >= a.table_rows) {
        if (lane == 0 && a.dev_status) atomicOr(a.dev_status, kDevIndex);
        return false;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.0f;
        s[i] = 0.0f;
    }
    if (p.turned) {
        const int u8 = 8 * (lane & (a.lanes - 1));
        const float* row = a.table + at * a.rotary;
        const int64_t bytes = 4 * a.table_rows * a.rotary;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 vc = ldg_checked(reinterpret_cast<const float4*>(row + u8) + h, a.table, bytes,
                                          a.dev_status);
            const float4 vs = ldg_checked(reinterpret_cast<const float4*>(row + a.rotary / 2 + u8) + h, a.table,
                                          bytes, a.dev_status);
            c[4 * h] = vc.x; c[4 * h + 1] = vc.y; c[4 * h + 2] = vc.z; c[4 * h + 3] = vc.w;
            s[4 * h] = vs.x; s[4 * h + 1] = vs.y; s[4 * h + 2] = vs.z; s[4 * h + 3] = vs.w;
        }
    }
    return true;
}

// f[0..15]: the unit's values, turned by the angles (SIGN +1) or back (-1).
template <bool INTERLEAVED, int SIGN>
__device__ __forceinline__ void turn(float* f, const float* c, const float* s)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int ia = INTERLEAVED ? 2 * i : i, ib = INTERLEAVED ? 2 * i + 1 : i + 8;
        const float x = f[ia], y = f[ib], sn = SIGN > 0 ? s[i] : -s[i];
        f[ia] = x * c[i] - y * sn;
        f[ib] = y * c[i] + x * sn;
    }
}

__device__ __forceinline__ float head_sum(float v, int lanes)
{
    for (int w = lanes >> 1; w; w >>= 1) v += __shfl_xor_sync(kAll, v, w);
    return v;
}

// 1 / sqrt(mean x^2 + eps) of the head.  Where the squares leave FP32 the values are taken times
// `scale` = 2^-70 (1 otherwise), in place; then the root is that of the scaled ones, so that scale r x is
// the normalised value either way.
__device__ __forceinline__ float head_norm(float* x, const HeadsArgs& a, float& scale)
{
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss += x[i] * x[i];
    ss = head_sum(ss, a.lanes);
    scale = 1.0f;
    float eps = a.eps;
    const bool large = !(ss < INFINITY);
    if (__any_sync(kAll, large)) {
        float sl = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float v = x[i] * 0x1p-70f;
            sl += v * v;
            if (large) x[i] = v;
        }
        sl = head_sum(sl, a.lanes);
        if (large) {
            ss = sl;
            scale = 0x1p-70f;
            eps *= 0x1p-70f * 0x1p-70f;
        }
    }
    return rsqrtf(ss * a.inv_D + eps);
}

__device__ __forceinline__ int64_t extent(const HeadsView& v, const HeadsArgs& a, int64_t esize)
{
    return esize * ((a.tokens - 1) * v.token_stride + (v.heads - 1) * v.head_stride + a.D);
}

template <bool IN_F32, bool OUT_F32, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_kernel(const HeadsArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t t = item / a.slices;
    if (t >= a.tokens) return;
    const Place p = place(a, INTERLEAVED, lane);
    float c[8], s[8];
    const bool there = load_angles(a, t, p, lane, c, s);
    const int together = 32 / a.lanes;
    const int q_steps = (a.x[0].heads + together - 1) / together;
    const int steps = q_steps + (a.x[1].heads + together - 1) / together;
    for (int j = static_cast<int>(item % a.slices); j < steps; j += a.slices) {
        const int kind = j >= q_steps;
        const HeadsView& x = a.x[kind];
        const HeadsView& z = a.z[kind];
        const int h = (kind ? j - q_steps : j) * together + p.slot;
        const bool on = p.in && h < x.heads;
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = 0.0f;
        if (there) {
            float w[16];
            if (on) {
                const int64_t at = t * x.token_stride + h * x.head_stride;
                const int64_t bytes = extent(x, a, IN_F32 ? 4 : 2);
                load8<IN_F32>(x.data, at + p.c0, bytes, a.dev_status, f);
                load8<IN_F32>(x.data, at + p.c1, bytes, a.dev_status, f + 8);
                load_weight(a.weight[kind], p.c0, p.c1, a.D, a.dev_status, w);
            }
            float scale;
            const float r = head_norm(f, a, scale);
            if (on) {
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = f[i] * r * w[i];
                if (p.turned) turn<INTERLEAVED, 1>(f, c, s);
            }
        }
        if (on) {
            const int64_t at = t * z.token_stride + h * z.head_stride;
            const int64_t bytes = extent(z, a, OUT_F32 ? 4 : 2);
            store8<OUT_F32>(z.data, at + p.c0, bytes, a.dev_status, f);
            store8<OUT_F32>(z.data, at + p.c1, bytes, a.dev_status, f + 8);
        }
    }
}

// The first q_ctas CTAs take the queries, the others the keys: a warp keeps one weight and the partial
// sums of its gradient in registers over all its tokens.  The CTA's sums go to a row of the workspace.
template <bool X_F32, bool Z_F32, bool DX_F32, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_backward_kernel(const HeadsArgs a)
{
    __shared__ float part[kWarps][kMaxHeadDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kind = static_cast<int>(blockIdx.x) >= a.q_ctas;
    const int64_t cta = kind ? blockIdx.x - a.q_ctas : blockIdx.x;
    const int64_t ctas = kind ? gridDim.x - a.q_ctas : a.q_ctas;
    const HeadsView& xv = a.x[kind];
    const HeadsView& zv = a.z[kind];
    const HeadsView& dv = a.dx[kind];
    const Place p = place(a, INTERLEAVED, lane);
    const int together = 32 / a.lanes;
    const int64_t steps = (xv.heads + together - 1) / together;
    float w[16], dw[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = dw[i] = 0.0f;
    if (p.in) load_weight(a.weight[kind], p.c0, p.c1, a.D, a.dev_status, w);
    // a warp's items in order: all steps of a token before the next one
    for (int64_t item = cta * kWarps + warp; item < a.tokens * a.slices; item += ctas * kWarps) {
        const int64_t t = item / a.slices;
        float c[8], s[8];
        const bool there = load_angles(a, t, p, lane, c, s);
        for (int64_t j = item % a.slices; j < steps; j += a.slices) {
            const int64_t h = j * together + p.slot;
            const bool on = p.in && h < xv.heads;
            float f[16], g[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = g[i] = 0.0f;
            if (there) {
                if (on) {
                    const int64_t at = t * xv.token_stride + h * xv.head_stride;
                    const int64_t bytes = extent(xv, a, X_F32 ? 4 : 2);
                    load8<X_F32>(xv.data, at + p.c0, bytes, a.dev_status, f);
                    load8<X_F32>(xv.data, at + p.c1, bytes, a.dev_status, f + 8);
                    const int64_t gat = t * zv.token_stride + h * zv.head_stride;
                    const int64_t gbytes = extent(zv, a, Z_F32 ? 4 : 2);
                    load8<Z_F32>(zv.data, gat + p.c0, gbytes, a.dev_status, g);
                    load8<Z_F32>(zv.data, gat + p.c1, gbytes, a.dev_status, g + 8);
                    if (p.turned) turn<INTERLEAVED, -1>(g, c, s);
                }
                float scale;
                const float r = head_norm(f, a, scale);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    f[i] *= r;
                    dw[i] += g[i] * f[i];
                    g[i] *= w[i];
                    dot += g[i] * f[i];
                }
                dot = head_sum(dot, a.lanes) * a.inv_D;
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = r * (g[i] - f[i] * dot) * scale;
            }
            if (on) {
                const int64_t at = t * dv.token_stride + h * dv.head_stride;
                const int64_t bytes = extent(dv, a, DX_F32 ? 4 : 2);
                store8<DX_F32>(dv.data, at + p.c0, bytes, a.dev_status, f);
                store8<DX_F32>(dv.data, at + p.c1, bytes, a.dev_status, f + 8);
            }
        }
    }
    // over the heads of a warp, then over the warps, in a fixed order
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        for (int m = a.lanes; m < 32; m <<= 1) dw[i] += __shfl_xor_sync(kAll, dw[i], m);
        if (p.slot == 0 && p.in) part[warp][(i < 8 ? p.c0 : p.c1) + (i & 7)] = dw[i];
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int d = threadIdx.x; d < a.D; d += 32 * kWarps) {
        float sum = part[0][d];
#pragma unroll
        for (int v = 1; v < kWarps; ++v) sum += part[v][d];
        st_checked(a.partials + static_cast<int64_t>(blockIdx.x) * a.D + d, sum, a.partials,
                   4 * static_cast<int64_t>(gridDim.x) * a.D, a.dev_status);
    }
}

// Sums of the CTAs' rows: 32 values of the head per CTA and kind, a warp per 32nd of the rows.
__global__ void __launch_bounds__(1024) weight_gradient_kernel(const HeadsArgs a, int ctas)
{
    __shared__ float part[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kind = blockIdx.y;
    const int d = blockIdx.x * 32 + lane;
    const int first = kind ? a.q_ctas : 0, last = kind ? ctas : a.q_ctas;
    float sum = 0.0f;
    if (d < a.D)
        for (int r = first + warp; r < last; r += 32)
            sum += ld_checked(a.partials + static_cast<int64_t>(r) * a.D + d, a.partials,
                              4 * static_cast<int64_t>(ctas) * a.D, a.dev_status);
    part[warp][lane] = sum;
    __syncthreads();
    float v = part[lane][warp];
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(kAll, v, m);
    const int out = blockIdx.x * 32 + warp;
    if (lane == 0 && out < a.D && a.dweight[kind])
        st_checked(a.dweight[kind] + out, v, a.dweight[kind], 4 * a.D, a.dev_status);
}

void set_lanes(HeadsArgs& a)
{
    a.lanes = 1;
    while (16 * a.lanes < a.D) a.lanes *= 2;
    a.inv_D = 1.0f / static_cast<float>(a.D);
}

}  // namespace

cudaError_t launch_qk_norm_rope(HeadsArgs a, bool in_f32, bool out_f32, bool interleaved, int sm_count,
                                cudaStream_t s)
{
    set_lanes(a);
    const int64_t together = 32 / a.lanes;
    const int64_t steps = (a.x[0].heads + together - 1) / together + (a.x[1].heads + together - 1) / together;
    // a warp takes a whole token, or a slice of its heads where the tokens are too few to fill the SMs
    int64_t slices = (32LL * sm_count + a.tokens - 1) / a.tokens;
    if (slices > steps) slices = steps;
    a.slices = static_cast<int>(slices < 1 ? 1 : slices);
    const int64_t ctas = (a.tokens * a.slices + kWarps - 1) / kWarps;
    const dim3 grid(static_cast<unsigned>(ctas));
#define QK_FORWARD(I, O)                                                                            \
    (interleaved ? qk_norm_rope_kernel<I, O, true><<<grid, 32 * kWarps, 0, s>>>(a)                  \
                 : qk_norm_rope_kernel<I, O, false><<<grid, 32 * kWarps, 0, s>>>(a))
    if (in_f32 && out_f32) QK_FORWARD(true, true);
    else if (in_f32) QK_FORWARD(true, false);
    else if (out_f32) QK_FORWARD(false, true);
    else QK_FORWARD(false, false);
#undef QK_FORWARD
    return cudaGetLastError();
}

int qk_backward_ctas(int64_t tokens, int64_t heads_q, int64_t heads_k, int64_t D)
{
    int64_t lanes = 1;
    while (16 * lanes < D) lanes *= 2;
    const int64_t together = 32 / lanes;
    const int64_t steps = (heads_q + together - 1) / together + (heads_k + together - 1) / together;
    const int64_t ctas = (tokens * steps + kWarps - 1) / kWarps;
    return static_cast<int>(ctas < 2 ? 2 : (ctas < kMaxHeadCtas ? ctas : kMaxHeadCtas));
}

cudaError_t launch_qk_norm_rope_backward(HeadsArgs a, bool x_f32, bool z_f32, bool dx_f32, bool interleaved,
                                         cudaStream_t s)
{
    set_lanes(a);
    const int ctas = qk_backward_ctas(a.tokens, a.x[0].heads, a.x[1].heads, a.D);
    const int64_t hq = a.x[0].heads, hk = a.x[1].heads;
    int64_t q = (ctas * hq + (hq + hk) / 2) / (hq + hk);
    if (q < (hq ? 1 : 0)) q = 1;
    if (q > ctas - (hk ? 1 : 0)) q = ctas - (hk ? 1 : 0);
    a.q_ctas = static_cast<int>(q);
    const int64_t together = 32 / a.lanes;
    const int64_t most = hq > hk ? hq : hk;
    const int64_t steps = (most + together - 1) / together;
    int64_t slices = (kMaxHeadCtas * kWarps + a.tokens - 1) / a.tokens;
    if (slices > steps) slices = steps;
    a.slices = static_cast<int>(slices < 1 ? 1 : slices);
    const dim3 grid(static_cast<unsigned>(ctas));
#define QK_BACKWARD(X, Z, D)                                                                            \
    (interleaved ? qk_norm_rope_backward_kernel<X, Z, D, true><<<grid, 32 * kWarps, 0, s>>>(a)          \
                 : qk_norm_rope_backward_kernel<X, Z, D, false><<<grid, 32 * kWarps, 0, s>>>(a))
    switch ((x_f32 ? 4 : 0) + (z_f32 ? 2 : 0) + (dx_f32 ? 1 : 0)) {
        case 0: QK_BACKWARD(false, false, false); break;
        case 1: QK_BACKWARD(false, false, true); break;
        case 2: QK_BACKWARD(false, true, false); break;
        case 3: QK_BACKWARD(false, true, true); break;
        case 4: QK_BACKWARD(true, false, false); break;
        case 5: QK_BACKWARD(true, false, true); break;
        case 6: QK_BACKWARD(true, true, false); break;
        default: QK_BACKWARD(true, true, true); break;
    }
#undef QK_BACKWARD
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.D + 31) / 32), 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weight_gradient_kernel, static_cast<const HeadsArgs>(a), ctas);
}

}  // namespace nvfp4
