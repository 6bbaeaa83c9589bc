// Norms of queries and keys for each head, with the position rotation in the same pass, and the
// gradient of both.  Per head of D values x, weight w, angles of the token's position p:
//   r = 1 / sqrt(mean x^2 + eps),  n = r x,  y = w n,  z = y with its first `rotary` values turned in pairs
//   backward: dy = dz turned back,  dw = sum dy n,  dn = w dy,  dx = r (dn - n mean(dn n))
// All in FP32; the only rounding to fewer bits is the one of the outputs to their type.
//
// A lane holds a unit of 16 values of a head, the first and the second ones of 8 rotated pairs (or 16
// neighbours behind the rotated part).  So a pair never leaves its lane, a lane stores only where it
// has loaded (outputs may be the inputs), and the mean is one reduction over the head's lanes.  The arithmetic
// goes two values at a time (.f32x2): by single values the passes were bound by instruction issue.
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

typedef uint64_t Two;  // two FP32 values

__device__ __forceinline__ Two fma2(Two a, Two b, Two c)
{
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ Two both(float v) { return f2pack(v, v); }

// 8 values as they lie in memory: a chunk.
template <bool F32>
struct Chunk {
    uint4 v[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ void load8(const char* at, const void* base, int64_t bytes, int* status, Chunk<F32>& r)
{
    const uint4* p = reinterpret_cast<const uint4*>(at);
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) r.v[i] = ld_checked(p + i, base, bytes, status);
}
template <bool F32>
__device__ __forceinline__ void store8(char* at, void* base, int64_t bytes, int* status, const Chunk<F32>& r)
{
    uint4* p = reinterpret_cast<uint4*>(at);
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) st_checked(p + i, r.v[i], base, bytes, status);
}
__device__ __forceinline__ float raw(uint32_t v) { return __uint_as_float(v); }

// The unit of two chunks: v[0..3] the first values of the 8 pairs, v[4..7] the second ones.  Pairs are
// value i of both chunks, or neighbours.
template <bool F32, bool INTERLEAVED>
__device__ __forceinline__ void to_unit(const Chunk<F32>& x, const Chunk<F32>& y, Two* v)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const Chunk<F32>& c = h ? y : x;
        float f[8];
        if (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4& w = c.v[F32 ? i : 0];
                f[4 * i] = raw(w.x); f[4 * i + 1] = raw(w.y); f[4 * i + 2] = raw(w.z); f[4 * i + 3] = raw(w.w);
            }
        } else {
            unpack8(c.v[0], f);
        }
        if (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[2 * h + i] = f2pack(f[4 * i], f[4 * i + 2]);
                v[4 + 2 * h + i] = f2pack(f[4 * i + 1], f[4 * i + 3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * h + i] = f2pack(f[2 * i], f[2 * i + 1]);
        }
    }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool F32, bool INTERLEAVED>
__device__ __forceinline__ void from_unit(const Two* v, Chunk<F32>& x, Chunk<F32>& y)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        Chunk<F32>& c = h ? y : x;
        float f[8];
        if (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[4 * i] = f2lo(v[2 * h + i]);
                f[4 * i + 1] = f2lo(v[4 + 2 * h + i]);
                f[4 * i + 2] = f2hi(v[2 * h + i]);
                f[4 * i + 3] = f2hi(v[4 + 2 * h + i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = f2lo(v[4 * h + i]);
                f[2 * i + 1] = f2hi(v[4 * h + i]);
            }
        }
        if (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                c.v[F32 ? i : 0] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                              __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
        } else {
            c.v[0] = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
        }
    }
}

// The place of a lane: its head among those a warp takes together, its unit of that head.
struct Place {
    int slot, unit;
    int c0, c1;        // first values of the unit's two chunks
    bool in, turned;   // the head has this unit; its values are rotated
};
template <bool INTERLEAVED>
__device__ __forceinline__ Place place(const HeadsArgs& a, int lane)
{
    Place p;
    p.unit = lane & (a.lanes - 1);
    p.slot = lane / a.lanes;
    p.in = 16 * p.unit < a.D;
    p.turned = 16 * p.unit < a.rotary;
    p.c0 = INTERLEAVED || !p.turned ? 16 * p.unit : 8 * p.unit;
    p.c1 = INTERLEAVED || !p.turned ? 16 * p.unit + 8 : a.rotary / 2 + 8 * p.unit;
    return p;
}
// Place i (0 .. 15) of a unit's values: which value of the head it is.
template <bool INTERLEAVED>
__device__ __forceinline__ int value_at(const Place& p, int i)
{
    if (INTERLEAVED) return 16 * p.unit + 2 * (i & 7) + (i >> 3);
    return (i < 8 ? p.c0 : p.c1) + (i & 7);
}

// Cosines and sines of the unit's 8 pairs at the token's position; false for a token without one.
__device__ __forceinline__ bool load_angles(const HeadsArgs& a, int64_t t, const Place& p, int lane, Two* c, Two* s)
{
    int64_t at = t;
    if (a.positions) at = ld_checked(a.positions + t, a.positions, 4 * a.tokens, a.dev_status);
    if (at < 0) return false;
    if (a.rotary && at >= a.table_rows) {
        if (lane == 0 && a.dev_status) atomicOr(a.dev_status, kDevIndex);
        return false;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i] = both(1.0f);
        s[i] = both(0.0f);
    }
    if (p.turned) {
        const float* row = a.table + at * a.rotary + 8 * p.unit;
        const int64_t bytes = 4 * a.table_rows * a.rotary;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 vc = ldg_checked(reinterpret_cast<const float4*>(row) + h, a.table, bytes, a.dev_status);
            const float4 vs = ldg_checked(reinterpret_cast<const float4*>(row + a.rotary / 2) + h, a.table, bytes,
                                          a.dev_status);
            c[2 * h] = f2pack(vc.x, vc.y);
            c[2 * h + 1] = f2pack(vc.z, vc.w);
            s[2 * h] = f2pack(vs.x, vs.y);
            s[2 * h + 1] = f2pack(vs.z, vs.w);
        }
    }
    return true;
}

// The unit's pairs turned by the angles (SIGN +1) or back (-1).
template <int SIGN>
__device__ __forceinline__ void turn(Two* v, const Two* c, const Two* s)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Two x = v[i], y = v[4 + i];
        if (SIGN > 0) {
            v[i] = sub2_rn(mul2_rn(x, c[i]), mul2_rn(y, s[i]));
            v[4 + i] = fma2(x, s[i], mul2_rn(y, c[i]));
        } else {
            v[i] = fma2(y, s[i], mul2_rn(x, c[i]));
            v[4 + i] = sub2_rn(mul2_rn(y, c[i]), mul2_rn(x, s[i]));
        }
    }
}

__device__ __forceinline__ float head_sum(float v, int lanes)
{
#pragma unroll
    for (int w = 16; w; w >>= 1)
        if (lanes > w) v += __shfl_xor_sync(kAll, v, w);
    return v;
}

// 1 / sqrt(mean x^2 + eps) of the head.  Where the squares leave FP32 the values are taken times
// `scale` = 2^-70 (1 otherwise), in place; then the root is that of the scaled ones, so that scale r x is
// the normalised value either way.
__device__ __forceinline__ float head_norm(Two* x, const HeadsArgs& a, float& scale)
{
    Two sum = mul2_rn(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) sum = fma2(x[i], x[i], sum);
    float ss = head_sum(f2lo(sum) + f2hi(sum), a.lanes);
    scale = 1.0f;
    float eps = a.eps;
    const bool large = !(ss < INFINITY);
    if (__any_sync(kAll, large)) {
        float sl = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Two v = mul2_rn(x[i], both(0x1p-70f));
            sl += f2lo(v) * f2lo(v) + f2hi(v) * f2hi(v);
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

// The weights (ones without them) of queries and keys in shared memory, four by four of a unit's places and
// then by unit: lanes read neighbouring 16 bytes.
constexpr int kMaxUnits = kMaxHeadDim / 16;
typedef float4 Weights[2][4][kMaxUnits];
template <bool INTERLEAVED>
__device__ __forceinline__ void share_weights(Weights shared, const HeadsArgs& a)
{
    for (int i = threadIdx.x; i < 32 * a.lanes; i += 32 * kWarps) {
        const int kind = i >= 16 * a.lanes, v = i - kind * 16 * a.lanes;
        const Place p = place<INTERLEAVED>(a, v / 16);  // a.lanes is at least the number of units
        const int d = value_at<INTERLEAVED>(p, v & 15);
        const float* w = a.weight[kind];
        reinterpret_cast<float*>(&shared[kind][(v & 15) / 4][v / 16])[v & 3] =
            !p.in ? 0.0f : (w ? ldg_checked(w + d, w, 4 * a.D, a.dev_status) : 1.0f);
    }
    __syncthreads();
}
__device__ __forceinline__ void unit_weights(const float4 (*shared)[kMaxUnits], const Place& p, Two* w)
{
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float4 v = shared[h][p.unit];
        w[2 * h] = f2pack(v.x, v.y);
        w[2 * h + 1] = f2pack(v.z, v.w);
    }
}

// The two chunks of a lane's unit of a head.
template <bool F32>
struct Unit {
    Chunk<F32> a, b;
};
// A lane's way through the heads of a token: head slot, slot + step, ...
template <bool F32>
struct Walk {
    char* at;
    int64_t step, second;  // bytes to the next head, to the unit's second chunk
    void* base;            // for the debug build's checks
    int64_t bytes;
    int* status;
    __device__ __forceinline__ Walk(const HeadsView& v, const HeadsArgs& a, int64_t t, int64_t head, int64_t heads_on,
                                    const Place& p)
    {
        constexpr int64_t size = F32 ? 4 : 2;
        at = static_cast<char*>(v.data) + size * (t * v.token_stride + head * v.head_stride + p.c0);
        step = size * heads_on * v.head_stride;
        second = size * (p.c1 - p.c0);
        base = v.data;
        bytes = size * ((a.tokens - 1) * v.token_stride + (v.heads - 1) * v.head_stride + a.D);
        status = a.dev_status;
    }
    __device__ __forceinline__ void load(Unit<F32>& u)
    {
        load8<F32>(at, base, bytes, status, u.a);
        load8<F32>(at + second, base, bytes, status, u.b);
    }
    __device__ __forceinline__ void store(const Unit<F32>& u)
    {
        store8<F32>(at, base, bytes, status, u.a);
        store8<F32>(at + second, base, bytes, status, u.b);
    }
};
// Zeros for the heads of a token without a position.
template <bool F32>
__device__ __forceinline__ void zero_heads(Walk<F32> z, int64_t h, int64_t heads_on, int64_t heads)
{
    const Unit<F32> zero = {};
    for (; h < heads; h += heads_on, z.at += z.step) z.store(zero);
}

// A warp takes a token, or a slice of its heads; the values of its next heads are on their way while it works on
// those before.  (The first ones are read for padding too, and not used.)  Bound by HBM: B200, 16384 tokens, 32 + 8
// heads of 128, bf16 64 us (5.4 TB/s, issue slots 58 % busy), FP32 109 (6.2 TB/s); without the next heads under way 72,
// with the weights read from memory for every head instead of from shared memory 70.  The bounds of 7 and 6 CTAs
// (72 and 80 registers) make three of the eight variants spill, bf16 and FP32 to bf16 with halves paired 20 bytes each.
template <bool IN_F32, bool OUT_F32, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps, IN_F32 ? 6 : 7) qk_norm_rope_kernel(const HeadsArgs a)
{
    __shared__ Weights weights;
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t t = item / a.slices;
    const Place p = place<INTERLEAVED>(a, lane);
    const int together = 32 / a.lanes;
    const int q_steps = static_cast<int>((a.x[0].heads + together - 1) / together);
    const int heads_on = together * a.slices;
    // the slice's first heads of the queries, and, where those end, of the keys
    const int slice = static_cast<int>(item - t * a.slices);
    const int k_first = slice >= q_steps ? slice - q_steps : (a.slices - (q_steps - slice) % a.slices) % a.slices;
    Unit<IN_F32> next = {};
    Two c[4], s[4];
    bool there = false;
    if (t < a.tokens) {
        if (p.in && slice * together + p.slot < a.x[0].heads)
            Walk<IN_F32>(a.x[0], a, t, slice * together + p.slot, heads_on, p).load(next);
        there = load_angles(a, t, p, lane, c, s);
    }
    share_weights<INTERLEAVED>(weights, a);
    if (t >= a.tokens) return;
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        const int all = static_cast<int>(a.x[kind].heads), heads = p.in ? all : 0;
        const int first = (kind ? k_first : slice) * together + p.slot;
        Walk<OUT_F32> z(a.z[kind], a, t, first, heads_on, p);
        if (!there) {
            zero_heads(z, first, heads_on, heads);
            continue;
        }
        Walk<IN_F32> x(a.x[kind], a, t, first, heads_on, p);
        if (kind && first < heads) x.load(next);
        // the whole warp goes on while a head of it is left (the lanes of a head reduce together)
        int left = all - (first - p.slot);
        for (int h = first; left > 0; left -= heads_on, h += heads_on) {
            Two v[8];
            to_unit<IN_F32, INTERLEAVED>(next.a, next.b, v);
            if (h + heads_on < heads) {
                x.at += x.step;
                x.load(next);
            }
            float scale;
            const Two r = both(head_norm(v, a, scale));
            Two w[8];
            unit_weights(weights[kind], p, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = mul2_rn(mul2_rn(v[i], r), w[i]);
            if (p.turned) turn<1>(v, c, s);
            if (h < heads) {
                Unit<OUT_F32> u;
                from_unit<OUT_F32, INTERLEAVED>(v, u.a, u.b);
                z.store(u);
                z.at += z.step;
            }
        }
    }
}

// The first q_ctas CTAs take the queries, the others the keys: a warp keeps the partial sums of one weight's
// gradient in registers over all its tokens.  The CTA's sums go to a row of the workspace.  B200, 16384 tokens, 32 +
// 8 heads of 128, bf16 111 us with the second kernel (4.6 TB/s), FP32 173 (5.8 TB/s): 16 warps of 125 to 128 registers
// per SM leave the issue slots 44 % busy and wait for the chain norm, dot, result.  The bf16 variants spill nothing, those
// with FP32 on one side up to 16 bytes; 20 warps spill more (141 us).  One value at a time 130 us; a ring of copies in
// shared memory ahead of the warp changes nothing (110, and 54 against 42 us for 4096 tokens, 16 + 4 heads of 256,
// FP32); the next token's first heads and angles under way 137.
template <bool X_F32, bool Z_F32, bool DX_F32, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps, 4) qk_norm_rope_backward_kernel(const HeadsArgs a)
{
    // Lanes behind the last head hold zeros or, again, a head of this token before, which must not reach dw (a
    // select of r = 0 would make NaN of its infinite gradients).  Their gradient is cleared, or dw's sums are skipped: 16384
    // tokens, 32 + 8 heads of 128, FP32 throughout 174 and 189 us, FP32 x and dz alone 150 and 165; bf16 115 and 111, FP32
    // x alone 133 and 131 (registers).
    constexpr bool CLEAR = X_F32 && Z_F32;
    __shared__ Weights weights;
    __shared__ float part[kWarps][kMaxHeadDim];
    share_weights<INTERLEAVED>(weights, a);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kind = static_cast<int>(blockIdx.x) >= a.q_ctas;
    const int64_t cta = kind ? blockIdx.x - a.q_ctas : blockIdx.x;
    const int64_t warps = (kind ? gridDim.x - a.q_ctas : a.q_ctas) * kWarps;
    const Place p = place<INTERLEAVED>(a, lane);
    const int together = 32 / a.lanes;
    const int heads_on = together * a.slices;
    const int all = static_cast<int>(a.x[kind].heads), heads = p.in ? all : 0;
    Two dw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = 0;
    // a warp's items in order: all heads of a token (or of its slice) before the next one
    for (int64_t item = cta * kWarps + warp; item < a.tokens * a.slices; item += warps) {
        const int64_t t = item / a.slices;
        const int base = static_cast<int>(item - t * a.slices) * together;
        int h = base + p.slot;
        Walk<X_F32> x(a.x[kind], a, t, h, heads_on, p);
        Walk<Z_F32> z(a.z[kind], a, t, h, heads_on, p);
        Walk<DX_F32> dx(a.dx[kind], a, t, h, heads_on, p);
        Unit<X_F32> next_x = {};
        Unit<Z_F32> next_z = {};
        if (h < heads) {
            x.load(next_x);
            z.load(next_z);
        }
        Two c[4], s[4];
        if (!load_angles(a, t, p, lane, c, s)) {
            zero_heads(dx, h, heads_on, heads);
            continue;
        }
        // the whole warp goes on while a head of it is left (the lanes of a head reduce together)
        for (int left = all - base; left > 0; left -= heads_on, h += heads_on) {
            Two f[8], g[8];
            to_unit<X_F32, INTERLEAVED>(next_x.a, next_x.b, f);
            to_unit<Z_F32, INTERLEAVED>(next_z.a, next_z.b, g);
            if (h + heads_on < heads) {
                x.at += x.step;
                z.at += z.step;
                x.load(next_x);
                z.load(next_z);
            } else if (CLEAR) {
                next_z = {};
            }
            if (p.turned) turn<-1>(g, c, s);
            float scale;
            const float r = head_norm(f, a, scale);
            Two w[8];
            unit_weights(weights[kind], p, w);
            // with e = r dy: dw += e x, dx = w e - (r x) (r mean(w e x)); r^2 by itself may leave FP32
            Two sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = mul2_rn(g[i], both(r));
            if (CLEAR || h < heads) {
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[i] = fma2(g[i], f[i], dw[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                g[i] = mul2_rn(g[i], w[i]);
                sum = fma2(g[i], f[i], sum);
            }
            const float dot = head_sum(f2lo(sum) + f2hi(sum), a.lanes) * a.inv_D;
            const Two back = both(-dot * r);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = fma2(mul2_rn(f[i], both(r)), back, g[i]);
            if (scale != 1.0f) {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = mul2_rn(f[i], both(scale));
            }
            if (h < heads) {
                Unit<DX_F32> u;
                from_unit<DX_F32, INTERLEAVED>(f, u.a, u.b);
                dx.store(u);
                dx.at += dx.step;
            }
        }
    }
    // over the heads of a warp, then over the warps, in a fixed order
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const Two two = dw[(i & 7) / 2 + 4 * (i >> 3)];
        float v = i & 1 ? f2hi(two) : f2lo(two);
        for (int m = a.lanes; m < 32; m <<= 1) v += __shfl_xor_sync(kAll, v, m);
        if (p.slot == 0 && p.in) part[warp][value_at<INTERLEAVED>(p, i)] = v;
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
