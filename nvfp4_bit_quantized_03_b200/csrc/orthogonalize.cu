// Newton-Schulz orthogonalisation of weight gradients (the update of the Muon optimiser):
//   X = G / (|G|_F + eps);  per step  A = X X^T,  B = b A + c A^2,  X <- a X + B X
// for every matrix of a batch, on the side where X has no more rows than columns (X = G^T otherwise).
// In exact arithmetic a step maps every singular value s of X to a s + b s^3 + c s^5 and keeps the singular
// vectors.
//
// Precision.  Every product takes FP16 operands (11 significant bits) with FP32 accumulation; X itself stays
// in FP32 between steps, and only its copy for the products is rounded.  A, B and the copy are held times
// powers of two that keep their values inside FP16's normal range: X times S ~ sqrt(columns), A times
// 2^12, B times 2^10.  The error of the result is then about that of its own rounding to bf16 (emulated in
// FP64, rms of error over rms of result: 1.2e-3 .. 1.9e-3 against 1.7e-3 for the rounding).  With X
// itself in FP16 a gradient of low rank is lost (1.5e-1: rounding noise of the directions that are not there
// is raised like everything else), with bf16 operands the error is 1e-2 and more.
//
// Kernels: the sum of squares (FP64), the scaled copies of X, then three products per step, one
// kernel each, chained by programmatic launches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "gemm_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

using gemm::bulk_wait_all;
using gemm::bulk_wait_read;
using gemm::cluster_rank;
using gemm::cluster_sync;
using gemm::desc_sw128;
using gemm::fence_async_smem;
using gemm::mbar_arrive_cluster;
using gemm::mbar_expect_tx;
using gemm::mbar_init;
using gemm::mma_commit_pair;
using gemm::named_sync;
using gemm::smem_u32;
using gemm::tc_fence_after;
using gemm::tc_fence_before;
using gemm::tmem_ld32;
using gemm::tmem_wait_ld;
using gemm::wait_bounded;

constexpr float kScaleA = 4096.0f;  // A is held times this,
constexpr float kScaleB = 1024.0f;  // B times this

// ---- the product kernels -----------------------------------------------------------------

enum Product { kGram = 0, kSquare = 1, kUpdate = 2, kLast = 3 };

constexpr int kBlock = 128;                    // rows a CTA loads of either operand; its tensor-memory lanes
constexpr int kDepth = 64;                     // K per pipeline stage (128 bytes of FP16)
constexpr int kOperandBytes = kBlock * 128;    // 16 KB
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;                   // two per lane quarter, half of the columns each
constexpr int kFirstEpi = 2;
constexpr int kGateWarp = kFirstEpi + kEpiWarps;
constexpr int kThreads = 32 * (kGateWarp + 1);
constexpr int kGateBar = 1;                    // named barriers 1 .. 6: issuer and gate, one per stage
constexpr int kStaging = 4096;                 // per epilogue warp: 32 rows of 64 FP16
constexpr int kBarBytes = 256;
constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kStaging + kBarBytes + 1024;
constexpr int kStateBlock = kBlock * kBlock;   // FP32 values of X per block of the state
static_assert(kSmem <= 232448, "shared memory per CTA");

// barriers (the same offsets in both CTAs of a pair)
constexpr int kBarFull = 0;                       // [stages] leader: the stage's bytes of both CTAs landed
constexpr int kBarEmpty = kBarFull + kStages;     // [stages] the stage's MMAs completed
constexpr int kBarAccFull = kBarEmpty + kStages;  // [2] the accumulator is complete
constexpr int kBarAccEmpty = kBarAccFull + 2;     // [2] leader: the epilogues have drained it
constexpr int kBarDrain = kBarAccEmpty + 2;
constexpr int kBars = kBarDrain + 1;
static_assert(kBars * 8 + 16 <= kBarBytes, "barrier area");

struct ProductArgs {
    int m, n, k;           // rows and columns of the result, length of the products
    int batch;
    float alpha, beta;     // result = alpha * (A or X) + beta * accumulator
    const __half* addend;  // square: A [batch][m][pitch]
    int64_t pitch;
    float* state;          // update: X in FP32, blocks of 128 x 128 in the order of the epilogue's lanes
    int state_rows, state_cols;  // blocks of a matrix
    uint16_t* out;         // last: the result, bf16
    int64_t ldo, out_stride;
    int transposed;        // last: out is X^T
    int by_tma;            // last: out's addresses suit tensor stores
    int* dev_status;
};

template <int CG>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar)
{
    if (CG == 2)  // signals a barrier of the pair's leader, from either CTA
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
            "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        gemm::tma_load_3d(dst, map, x, y, z, bar);
}

__device__ __forceinline__ void store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(x), "r"(y), "r"(z), "r"(src)
        : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ uint32_t leader_address(uint32_t a)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
    return r;
}

// Operand whose rows run along K in shared memory (64 rows of K x 128 bytes, 128-byte swizzle): 64 values of
// the other axis per row, the next 64 of them 8 KB on (leading offset), groups of 8 rows 1 KB apart.
__device__ __forceinline__ uint64_t desc_across(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(8192 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

// D += A . B over K = 16; FP16 operands, FP32 accumulator.
template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(accumulate)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    if (CG == 2)
        mma_commit_pair(bar);
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
}
template <int CG>
__device__ __forceinline__ void arrive_leader(uint32_t bar)
{
    if (CG == 2)
        mbar_arrive_cluster(bar, 0);
    else
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

struct Tile {
    int e, i, j;  // matrix, row and column of tiles
};
// The symmetric products (gram, square) have tiles on and below the diagonal only, row by row; the others go
// down the columns, so that the left operand (m x m) stays in L2 and X is read once.
template <int OP>
__device__ __forceinline__ Tile tile_at(int64_t t, int rows, int cols)
{
    Tile r;
    if (OP == kGram || OP == kSquare) {
        const int per = rows * (rows + 1) / 2;
        r.e = static_cast<int>(t / per);
        const int l = static_cast<int>(t - static_cast<int64_t>(r.e) * per);
        int i = static_cast<int>((sqrtf(8.0f * l + 1.0f) - 1.0f) * 0.5f);
        while (i * (i + 1) / 2 > l) --i;
        while ((i + 1) * (i + 2) / 2 <= l) ++i;
        r.i = i;
        r.j = l - i * (i + 1) / 2;
    } else {
        const int per = rows * cols;
        r.e = static_cast<int>(t / per);
        const int l = static_cast<int>(t - static_cast<int64_t>(r.e) * per);
        r.i = l % rows;
        r.j = l / rows;
    }
    return r;
}

// One tile of 128 CG x 128 CG per CTA (CG 1) or pair of CTAs (CG 2: cta_group::2, each CTA holds half of
// either operand's rows and the accumulator of its 128 rows).  Warp 0 loads, warp 1 issues the MMAs, warps
// 2..9 turn accumulators into results; two accumulators, so that a tile's results are written while the next
// one is multiplied.
template <int CG, int OP>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_d, const __grid_constant__ CUtensorMap map_t,
                   const ProductArgs p)
{
    constexpr int TILE = kBlock * CG;
    constexpr int ACC_COLS = TILE;           // tensor-memory columns of an accumulator
    constexpr bool SYMMETRIC = OP == kGram || OP == kSquare;
    constexpr bool ACROSS = OP == kUpdate || OP == kLast;  // the right operand's rows run along K
    constexpr uint32_t IDESC = (1u << 4) | (ACROSS ? 1u << 16 : 0u) | (static_cast<uint32_t>(TILE >> 3) << 17) |
                               (static_cast<uint32_t>(TILE >> 4) << 24);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* staging = smem + kStages * kStageBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kEpiWarps * kStaging);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0;
    const int64_t worker = blockIdx.x / CG, workers = gridDim.x / CG;
    const int rows = (p.m + TILE - 1) / TILE, cols = (p.n + TILE - 1) / TILE;
    const int64_t total = static_cast<int64_t>(p.batch) * (SYMMETRIC ? rows * (rows + 1) / 2 : rows * cols);
    const int depth = (p.k + kDepth - 1) / kDepth;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(kBarFull + s), 1);
            mbar_init(bar(kBarEmpty + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(kBarAccFull + b), 1);
            mbar_init(bar(kBarAccEmpty + b), CG * kEpiWarps);
        }
        mbar_init(bar(kBarDrain), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_b)) : "memory");
    }
    if (warp == 1) {
        if (CG == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(2 * ACC_COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(2 * ACC_COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // everything this kernel reads is the work of the kernels ahead
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 0 && lane == 0) {
        // ---------------- loads ----------------
        asm volatile("fence.proxy.async;" ::: "memory");  // copies written by ordinary stores
        int stage = 0;
        uint32_t phase = 0, fills = 0;
        bool ok = true;
        for (int64_t t = worker; t < total && ok; t += workers) {
            const Tile c = tile_at<OP>(t, rows, cols);
            const int ya = c.i * TILE + rank * kBlock, yb = c.j * TILE + rank * kBlock;
            for (int d = 0; d < depth; ++d) {
                if (!wait_bounded(bar(kBarEmpty + stage), phase ^ 1, abort_flag, p.dev_status)) {
                    ok = false;
                    break;
                }
                if (kBoundsCheck && !(gemm::tma_box_start_ok(d * kDepth, ya, 2, p.dev_status) &&
                                      gemm::tma_box_start_ok(yb, d * kDepth, 2, p.dev_status) &&
                                      c.e < p.batch)) {
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                const uint32_t full = CG == 2 ? leader_address(bar(kBarFull + stage)) : bar(kBarFull + stage);
                const uint32_t at = smem_u32(smem + stage * kStageBytes);
                if (rank == 0) mbar_expect_tx(bar(kBarFull + stage), CG * kStageBytes);
                load_3d<CG>(at, &map_a, d * kDepth, ya, c.e, full);
                if (ACROSS) {
                    load_3d<CG>(at + kOperandBytes, &map_b, yb, d * kDepth, c.e, full);
                    load_3d<CG>(at + kOperandBytes + kOperandBytes / 2, &map_b, yb + 64, d * kDepth, c.e, full);
                } else {
                    load_3d<CG>(at + kOperandBytes, &map_b, d * kDepth, yb, c.e, full);
                }
                ++fills;
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) {
            // Every copy already issued lands before the CTA can exit: the leader waits for the fills it
            // announced, a peer (whose copies signal the leader) the time in which copies land.
            if (rank == 0) {
                for (uint32_t s = 0; s < kStages; ++s) {
                    const uint32_t n = fills > s ? (fills - s + kStages - 1) / kStages : 0u;
                    if (n) wait_bounded(bar(kBarFull + s), (n - 1) & 1, abort_flag, nullptr, true, 100000000ull);
                }
            }
            const uint64_t t0 = gemm::globaltimer();
            while (gemm::globaltimer() - t0 < 5000000ull) __nanosleep(1000);
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer ----------------
        // It polls no barrier: the gate has seen the stage's bytes land (and, at a tile's first stage, the
        // accumulator drained) when both meet at the stage's named barrier.  After an abort the gate keeps
        // meeting the issuer, which runs its schedule on stale operands (in bounds, results discarded).
        const uint32_t s0 = smem_u32(smem);
        int stage = 0, it = 0;
        for (int64_t t = worker; t < total; t += workers, ++it) {
            const uint32_t acc = tmem + (it & 1) * ACC_COLS;
            for (int d = 0; d < depth; ++d) {
                named_sync(kGateBar + stage, 64);
                if (lane == 0) {
                    tc_fence_after();
                    const uint64_t da = desc_sw128(s0 + stage * kStageBytes);
                    const uint64_t db = ACROSS ? desc_across(s0 + stage * kStageBytes + kOperandBytes)
                                               : desc_sw128(s0 + stage * kStageBytes + kOperandBytes);
#pragma unroll
                    for (int k = 0; k < kDepth / 16; ++k)  // 32 bytes of a row, or 16 rows, further on
                        mma_f16<CG>(acc, da + 2 * k, db + (ACROSS ? 128 : 2) * k, IDESC, (d | k) != 0 ? 1u : 0u);
                    mma_commit<CG>(bar(kBarEmpty + stage));
                    if (d + 1 == depth) mma_commit<CG>(bar(kBarAccFull + (it & 1)));
                }
                __syncwarp();
                if (++stage == kStages) stage = 0;
            }
        }
        // every MMA completes before the tensor memory can be freed
        if (lane == 0 && it > 0) {
            mma_commit<CG>(bar(kBarDrain));
            wait_bounded(bar(kBarDrain), 0, abort_flag, nullptr, true);
        }
    } else if (warp == kGateWarp && rank == 0) {
        // ---------------- the issuer's gate ----------------
        int stage = 0, it = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t t = worker; t < total; t += workers, ++it) {
            for (int d = 0; d < depth; ++d) {
                if (lane == 0 && ok) {
                    if (d == 0)
                        ok = wait_bounded(bar(kBarAccEmpty + (it & 1)), ((it >> 1) & 1) ^ 1, abort_flag,
                                          p.dev_status);
                    if (ok) ok = wait_bounded(bar(kBarFull + stage), phase, abort_flag, p.dev_status);
                }
                __syncwarp();
                named_sync(kGateBar + stage, 64);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp >= kFirstEpi && warp < kFirstEpi + kEpiWarps) {
        // ---------------- epilogue ----------------
        constexpr int SLICE = 64 * CG;  // columns of a warp
        const int q = warp & 3, half = (warp - kFirstEpi) >> 2;
        const uint32_t stage_buf = smem_u32(staging + (warp - kFirstEpi) * kStaging);
        int it = 0;
        for (int64_t t = worker; t < total; t += workers, ++it) {
            const Tile c = tile_at<OP>(t, rows, cols);
            const int buf = it & 1;
            const int r0 = c.i * TILE + rank * kBlock + 32 * q;  // the warp's rows (one per lane)
            const int c0 = c.j * TILE + half * SLICE;            // its columns
            bool ready = lane == 0 ? wait_bounded(bar(kBarAccFull + buf), (it >> 1) & 1, abort_flag, p.dev_status)
                                   : false;
            ready = __shfl_sync(0xFFFFFFFFu, ready ? 1 : 0, 0) != 0;
            if (!ready) break;
            tc_fence_after();
#pragma unroll 1
            for (int w = 0; w < CG; ++w) {  // 64 columns at a time
                const int col = c0 + 64 * w;
                uint32_t packed[32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float f[32];
                    const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q) << 16) + buf * ACC_COLS +
                                           half * SLICE + 64 * w + 32 * h;
                    uint32_t v[32];
                    tmem_ld32(taddr, v);
                    if (OP == kGram) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) f[i] = 0.0f;
                    } else if (OP == kSquare) {
                        const int row = r0 + lane;
                        const __half* src = p.addend + (static_cast<int64_t>(c.e) * p.m + row) * p.pitch + col + 32 * h;
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            uint4 x = make_uint4(0, 0, 0, 0);
                            if (row < p.m && col + 32 * h + 8 * g < p.pitch)
                                x = ld_checked(reinterpret_cast<const uint4*>(src) + g, p.addend,
                                               2 * static_cast<int64_t>(p.batch) * p.m * p.pitch, p.dev_status);
                            const __half2* hx = reinterpret_cast<const __half2*>(&x);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 two = __half22float2(hx[i]);
                                f[8 * g + 2 * i] = two.x;
                                f[8 * g + 2 * i + 1] = two.y;
                            }
                        }
                    } else {
                        const int cc = col + 32 * h;
                        const int64_t block = (static_cast<int64_t>(c.e) * p.state_rows + r0 / kBlock) * p.state_cols +
                                              cc / kBlock;
                        if (r0 / kBlock < p.state_rows && cc / kBlock < p.state_cols) {
                            float4* src = reinterpret_cast<float4*>(p.state + block * kStateBlock) +
                                          (q * 32 + (cc % kBlock) / 4) * 32 + lane;
                            const int64_t bytes = 4LL * kStateBlock * p.batch * p.state_rows * p.state_cols;
#pragma unroll
                            for (int g = 0; g < 8; ++g) {
                                const float4 x = ld_checked(src + 32 * g, p.state, bytes, p.dev_status);
                                f[4 * g] = x.x; f[4 * g + 1] = x.y; f[4 * g + 2] = x.z; f[4 * g + 3] = x.w;
                            }
                        }
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        f[i] = OP == kGram ? p.beta * __uint_as_float(v[i])
                                           : p.alpha * f[i] + p.beta * __uint_as_float(v[i]);
                    if (OP == kUpdate) {
                        const int cc = col + 32 * h;
                        const int64_t block = (static_cast<int64_t>(c.e) * p.state_rows + r0 / kBlock) * p.state_cols +
                                              cc / kBlock;
                        if (r0 / kBlock < p.state_rows && cc / kBlock < p.state_cols) {
                            float4* dst = reinterpret_cast<float4*>(p.state + block * kStateBlock) +
                                          (q * 32 + (cc % kBlock) / 4) * 32 + lane;
                            const int64_t bytes = 4LL * kStateBlock * p.batch * p.state_rows * p.state_cols;
#pragma unroll
                            for (int g = 0; g < 8; ++g)
                                st_checked(dst + 32 * g, make_float4(f[4 * g], f[4 * g + 1], f[4 * g + 2], f[4 * g + 3]),
                                           p.state, bytes, p.dev_status);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        packed[16 * h + i] = OP == kLast ? pack_bf16(f[2 * i], f[2 * i + 1])
                                                         : pack_half(f[2 * i], f[2 * i + 1]);
                }
                if (w == CG - 1) {  // the last of the warp's slice is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_leader<CG>(bar(kBarAccEmpty + buf));
                }
                const bool inside = r0 < p.m && col < p.n;
                const bool direct = OP != kLast || !p.transposed;
                const bool turned = SYMMETRIC ? c.i != c.j : (OP == kLast && p.transposed);
                if (direct) {
                    // row `lane`: 128 bytes, its 16-byte chunks permuted by the 128-byte swizzle
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage_buf + 128 * lane +
                                                                                       16 * (g ^ (lane & 7))),
                                     "r"(packed[4 * g]), "r"(packed[4 * g + 1]), "r"(packed[4 * g + 2]),
                                     "r"(packed[4 * g + 3])
                                     : "memory");
                    if (OP != kLast || p.by_tma) {
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0 && inside &&
                            (!kBoundsCheck || gemm::tma_box_start_ok(col, r0, 2, p.dev_status)))
                            store_3d(&map_d, stage_buf, col, r0, c.e);
                    } else {
                        __syncwarp();
                        const int64_t bytes = 2 * ((p.batch - 1) * p.out_stride + (p.m - 1) * p.ldo + p.n);
                        for (int r = 0; r < 32 && r0 + r < p.m; ++r)
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                const int x = 2 * (lane + 32 * g);
                                uint16_t v;
                                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(stage_buf + 128 * r +
                                                                                   (((x >> 4) ^ (r & 7)) << 4) + (x & 15)));
                                if (col + x / 2 < p.n)
                                    st_checked(p.out + c.e * p.out_stride + (r0 + r) * p.ldo + col + x / 2, v, p.out,
                                               bytes, p.dev_status);
                            }
                        __syncwarp();
                    }
                }
                if (turned) {
                    // row j of the turned box: the warp's 32 rows of column j
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(stage_buf + 128 * i + 2 * lane),
                                     "h"(static_cast<uint16_t>(packed[i]))
                                     : "memory");
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(stage_buf + 128 * i + 64 + 2 * lane),
                                     "h"(static_cast<uint16_t>(packed[i] >> 16))
                                     : "memory");
                    }
                    if (OP != kLast || p.by_tma) {
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0 && inside &&
                            (!kBoundsCheck || gemm::tma_box_start_ok(r0, col, 2, p.dev_status)))
                            store_3d(&map_t, stage_buf, r0, col, c.e);
                    } else {
                        __syncwarp();
                        const int64_t bytes = 2 * ((p.batch - 1) * p.out_stride + (p.n - 1) * p.ldo + p.m);
                        if (r0 + lane < p.m)
                            for (int j = 0; j < 64 && col + j < p.n; ++j) {
                                uint16_t v;
                                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(stage_buf + 64 * j + 2 * lane));
                                st_checked(p.out + c.e * p.out_stride + (col + j) * p.ldo + r0 + lane, v, p.out, bytes,
                                           p.dev_status);
                            }
                        __syncwarp();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
    }

    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if (CG == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * ACC_COLS)
                         : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * ACC_COLS)
                         : "memory");
    }
}

// ---- the norm and the scaled copies --------------------------------------------------------

constexpr int kNormThreads = 256;

struct PrepareArgs {
    const void* g;
    int64_t rows, cols, ldg, g_stride;  // of G
    int64_t m, n, pitch;                // of X (G or G^T) and of its FP16 copy
    int batch, transposed;
    int parts;                          // partial sums per matrix
    double* partials;                   // [batch][parts]
    float* state;
    int state_rows, state_cols;
    __half* x;
    double scale, eps;
    int* dev_status;
};

template <bool F32>
__device__ __forceinline__ float element(const PrepareArgs& a, int64_t at, int64_t bytes)
{
    if (F32) return ldg_checked(static_cast<const float*>(a.g) + at, a.g, bytes, a.dev_status);
    const uint16_t v = ldg_checked(static_cast<const uint16_t*>(a.g) + at, a.g, bytes, a.dev_status);
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

__device__ __forceinline__ double block_sum(double v, double* shared)
{
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, s);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < kNormThreads / 32; ++w) sum += shared[w];
    __syncthreads();
    return sum;
}

// Partial sums of the squares, in FP64: no value of FP32 or bf16 leaves its range when squared.
template <bool F32>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const PrepareArgs a)
{
    __shared__ double shared[kNormThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t e = blockIdx.y;
    const int64_t bytes = (F32 ? 4 : 2) * ((a.batch - 1) * a.g_stride + (a.rows - 1) * a.ldg + a.cols);
    double sum = 0.0;
    // a warp takes rows (or pieces of 1024 values of them) in turn
    const int64_t pieces = (a.cols + 1023) / 1024;
    const int warps = kNormThreads / 32;
    for (int64_t i = blockIdx.x * warps + (threadIdx.x >> 5); i < a.rows * pieces;
         i += static_cast<int64_t>(gridDim.x) * warps) {
        const int64_t r = i / pieces, c0 = (i - r * pieces) * 1024;
        const int64_t end = c0 + 1024 < a.cols ? c0 + 1024 : a.cols;
        const int64_t base = e * a.g_stride + r * a.ldg;
#pragma unroll 8
        for (int64_t c = c0 + (threadIdx.x & 31); c < end; c += 32) {
            const double v = element<F32>(a, base + c, bytes);
            sum += v * v;
        }
    }
    sum = block_sum(sum, shared);
    if (threadIdx.x == 0)
        st_checked(a.partials + e * a.parts + blockIdx.x, sum, a.partials,
                   8 * static_cast<int64_t>(a.batch) * a.parts, a.dev_status);
}

// X times the scale over the norm: in FP32 in the order of the products' epilogue, and in FP16 row by row.
// A CTA takes pieces of 32 rows x 128 columns of X through shared memory (G^T: both sides stay coalesced).
template <bool F32>
__global__ void __launch_bounds__(kNormThreads) prepare_kernel(const PrepareArgs a)
{
    __shared__ double shared[kNormThreads / 32];
    __shared__ __align__(16) float tile[32][132];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t bytes = (F32 ? 4 : 2) * ((a.batch - 1) * a.g_stride + (a.rows - 1) * a.ldg + a.cols);
    const int64_t row_pieces = (a.m + 31) / 32, col_pieces = (a.n + 127) / 128;
    const int64_t per = row_pieces * col_pieces;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t have = -1;
    double scale = 0.0;
    bool finite = true;
    for (int64_t i = blockIdx.x; i < per * a.batch; i += gridDim.x) {
        const int64_t e = i / per, l = i - e * per;
        const int64_t r0 = l / col_pieces * 32, c0 = l % col_pieces * 128;
        if (e != have) {
            double sum = 0.0;
            for (int j = threadIdx.x; j < a.parts; j += kNormThreads)
                sum += ld_checked(a.partials + e * a.parts + j, a.partials,
                                  8 * static_cast<int64_t>(a.batch) * a.parts, a.dev_status);
            sum = block_sum(sum, shared);
            finite = sum < INFINITY;
            const double norm = sqrt(sum) + a.eps;
            scale = norm > 0.0 ? a.scale / norm : 0.0;
            have = e;
            if (!finite && l == 0 && threadIdx.x == 0 && a.dev_status) atomicOr(a.dev_status, 1);  // NONFINITE
        }
        __syncthreads();  // the piece before has left the tile
        if (a.transposed) {
            for (int c = warp; c < 128; c += kNormThreads / 32) {
                const int64_t r = r0 + lane, cc = c0 + c;
                float v = 0.0f;
                if (r < a.m && cc < a.n && finite) {
                    const double d = element<F32>(a, e * a.g_stride + cc * a.ldg + r, bytes);
                    v = static_cast<float>(d * scale);
                }
                tile[lane][c] = v;
            }
        } else {
            for (int r = warp; r < 32; r += kNormThreads / 32)
#pragma unroll
                for (int c = lane; c < 128; c += 32) {
                    float v = 0.0f;
                    if (r0 + r < a.m && c0 + c < a.n && finite) {
                        const double d = element<F32>(a, e * a.g_stride + (r0 + r) * a.ldg + c0 + c, bytes);
                        v = static_cast<float>(d * scale);
                    }
                    tile[r][c] = v;
                }
        }
        __syncthreads();
        const int64_t block = (e * a.state_rows + r0 / kBlock) * a.state_cols + c0 / kBlock;
        float4* dst = reinterpret_cast<float4*>(a.state + block * kStateBlock) + (r0 % kBlock) / 32 * 32 * 32;
        const int64_t state_bytes = 4LL * kStateBlock * a.batch * a.state_rows * a.state_cols;
        for (int c4 = warp; c4 < 32; c4 += kNormThreads / 32)
            st_checked(dst + c4 * 32 + lane, *reinterpret_cast<const float4*>(&tile[lane][4 * c4]), a.state,
                       state_bytes, a.dev_status);
        for (int r = warp; r < 32; r += kNormThreads / 32) {
            if (r0 + r >= a.m || c0 + 4 * lane >= a.pitch) continue;
            const float4 v = *reinterpret_cast<const float4*>(&tile[r][4 * lane]);
            st_checked(reinterpret_cast<uint2*>(a.x + (e * a.m + r0 + r) * a.pitch + c0) + lane,
                       make_uint2(pack_half(v.x, v.y), pack_half(v.z, v.w)), a.x, 2 * a.batch * a.m * a.pitch,
                       a.dev_status);
        }
    }
}

// ---- host ------------------------------------------------------------------------------

size_t round256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Boxes of box_x x box_y of a batch of matrices (rows x cols values of 2 bytes, `pitch` apart).
bool make_map(CUtensorMap* map, void* data, int64_t cols, int64_t rows, int64_t batch, int64_t pitch, int64_t stride,
              int box_x, int box_y, bool swizzle, bool bf16 = false)
{
    auto enc = gemm::tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * pitch), static_cast<cuuint64_t>(2 * stride)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_x), static_cast<cuuint32_t>(box_y), 1};
    const cuuint32_t one[3] = {1, 1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, data, dims, strides,
               box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using ProductKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap,
                               const ProductArgs);

template <int CG>
ProductKernel product_of(int op)
{
    switch (op) {
        case kGram: return product_kernel<CG, kGram>;
        case kSquare: return product_kernel<CG, kSquare>;
        case kUpdate: return product_kernel<CG, kUpdate>;
        default: return product_kernel<CG, kLast>;
    }
}

cudaError_t configure_once(int* device)
{
    constexpr int kDevices = 64;
    static bool done[kDevices] = {};
    static std::mutex mutex;
    if (cudaGetDevice(device) != cudaSuccess || *device < 0 || *device >= kDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mutex);
    if (done[*device]) return cudaSuccess;
    for (int op = 0; op < 4; ++op)
        for (int cg = 1; cg <= 2; ++cg) {
            const void* f = reinterpret_cast<const void*>(cg == 1 ? product_of<1>(op) : product_of<2>(op));
            const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            if (e != cudaSuccess) return e;
        }
    done[*device] = true;
    return cudaSuccess;
}

// A kernel behind another one of the same call; it waits for that itself.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s,
                           A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct Sizes {
    int64_t m, n, x_pitch, a_pitch, state_rows, state_cols;
    int parts;
    size_t partials, state, x, a;  // bytes
};

Sizes sizes_of(int64_t batch, int64_t rows, int64_t cols)
{
    Sizes s;
    s.m = rows < cols ? rows : cols;
    s.n = rows < cols ? cols : rows;
    s.x_pitch = (s.n + 63) / 64 * 64;  // rows of whole 128-byte lines
    s.a_pitch = (s.m + 63) / 64 * 64;
    s.state_rows = (s.m + kBlock - 1) / kBlock;
    s.state_cols = (s.n + kBlock - 1) / kBlock;
    // partial sums: 16 K values each, no more than fill the SMs several times
    int64_t parts = (rows * cols + 16383) / 16384;
    const int64_t most = batch < 592 ? 592 / batch : 1;
    s.parts = static_cast<int>(parts < most ? parts : most);
    s.partials = round256(8 * static_cast<size_t>(batch) * s.parts);
    s.state = round256(4 * static_cast<size_t>(kStateBlock) * batch * s.state_rows * s.state_cols);
    s.x = round256(2 * static_cast<size_t>(batch) * s.m * s.x_pitch);
    s.a = round256(2 * static_cast<size_t>(batch) * s.m * s.a_pitch);
    return s;
}

}  // namespace

size_t orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols)
{
    const Sizes s = sizes_of(batch, rows, cols);
    return s.partials + s.state + 2 * s.x + 2 * s.a;
}

cudaError_t launch_orthogonalize(const OrthogonalizeArgs& g, int sm_count, cudaStream_t s)
{
    int device = 0;
    cudaError_t e = configure_once(&device);
    if (e != cudaSuccess) return e;
    const Sizes z = sizes_of(g.batch, g.rows, g.cols);
    const bool transposed = g.rows > g.cols;
    uint8_t* at = static_cast<uint8_t*>(g.workspace);
    double* partials = reinterpret_cast<double*>(at);
    float* state = reinterpret_cast<float*>(at += z.partials);
    __half* x[2];
    x[0] = reinterpret_cast<__half*>(at += z.state);
    x[1] = reinterpret_cast<__half*>(at += z.x);
    __half* a = reinterpret_cast<__half*>(at += z.x);
    __half* b = reinterpret_cast<__half*>(at += z.a);

    // X times S: values of about 1 where the rows of X are orthonormal
    const double S = std::ldexp(1.0, static_cast<int>(std::lround(0.5 * std::log2(static_cast<double>(z.n)))));
    PrepareArgs pa = {};
    pa.g = g.g;
    pa.rows = g.rows;
    pa.cols = g.cols;
    pa.ldg = g.ldg;
    pa.g_stride = g.g_stride;
    pa.m = z.m;
    pa.n = z.n;
    pa.pitch = z.x_pitch;
    pa.batch = static_cast<int>(g.batch);
    pa.transposed = transposed;
    pa.parts = z.parts;
    pa.partials = partials;
    pa.state = state;
    pa.state_rows = static_cast<int>(z.state_rows);
    pa.state_cols = static_cast<int>(z.state_cols);
    pa.x = x[0];
    pa.scale = S;
    pa.eps = g.eps;
    pa.dev_status = g.dev_status;

    CUtensorMap x_rows[2], x_across[2], x_store[2], a_rows, b_rows, a_store, b_store, a_turn, b_turn, out_store;
    bool ok = true;
    const int64_t xs = z.m * z.x_pitch, as = z.m * z.a_pitch;
    for (int i = 0; i < 2; ++i)
        ok = ok && make_map(&x_rows[i], x[i], z.n, z.m, g.batch, z.x_pitch, xs, kDepth, kBlock, true) &&
             make_map(&x_across[i], x[i], z.n, z.m, g.batch, z.x_pitch, xs, 64, kDepth, true) &&
             make_map(&x_store[i], x[i], z.n, z.m, g.batch, z.x_pitch, xs, 64, 32, true);
    ok = ok && make_map(&a_rows, a, z.m, z.m, g.batch, z.a_pitch, as, kDepth, kBlock, true) &&
         make_map(&b_rows, b, z.m, z.m, g.batch, z.a_pitch, as, kDepth, kBlock, true) &&
         make_map(&a_store, a, z.m, z.m, g.batch, z.a_pitch, as, 64, 32, true) &&
         make_map(&b_store, b, z.m, z.m, g.batch, z.a_pitch, as, 64, 32, true) &&
         make_map(&a_turn, a, z.m, z.m, g.batch, z.a_pitch, as, 32, 64, false) &&
         make_map(&b_turn, b, z.m, z.m, g.batch, z.a_pitch, as, 32, 64, false);
    // tensor stores want 16-byte aligned rows, and end on 16 bytes: on B200 one that was clipped at 131 columns
    // wrote past them
    const bool by_tma = (reinterpret_cast<uintptr_t>(g.out) & 15) == 0 && g.ldo % 8 == 0 &&
                        g.out_stride % 8 == 0 && g.cols % 8 == 0;
    if (by_tma)
        ok = ok && make_map(&out_store, g.out, g.cols, g.rows, g.batch, g.ldo, g.out_stride, transposed ? 32 : 64,
                            transposed ? 64 : 32, !transposed, true);
    else
        out_store = x_store[0];  // not used
    if (!ok) return cudaErrorInvalidValue;

    const dim3 norm_grid(static_cast<unsigned>(z.parts), static_cast<unsigned>(g.batch));
    if (g.f32) norm_kernel<true><<<norm_grid, kNormThreads, 0, s>>>(pa);
    else       norm_kernel<false><<<norm_grid, kNormThreads, 0, s>>>(pa);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int64_t pieces = g.batch * ((z.m + 31) / 32) * z.state_cols;
    const dim3 prepare_grid(static_cast<unsigned>(pieces < 8 * sm_count ? pieces : 8 * sm_count));
    e = launch_chained(g.f32 ? prepare_kernel<true> : prepare_kernel<false>, prepare_grid, kNormThreads, 0, 1, s, pa);
    if (e != cudaSuccess) return e;

    ProductArgs p = {};
    p.batch = static_cast<int>(g.batch);
    p.addend = a;
    p.pitch = z.a_pitch;
    p.state = state;
    p.state_rows = pa.state_rows;
    p.state_cols = pa.state_cols;
    p.out = static_cast<uint16_t*>(g.out);
    p.ldo = g.ldo;
    p.out_stride = g.out_stride;
    p.transposed = transposed;
    p.by_tma = by_tma;
    p.dev_status = g.dev_status;
    auto product = [&](int op, int64_t m, int64_t n, int64_t k, const CUtensorMap& ma, const CUtensorMap& mb,
                       const CUtensorMap& md, const CUtensorMap& mt, double alpha, double beta) {
        p.m = static_cast<int>(m);
        p.n = static_cast<int>(n);
        p.k = static_cast<int>(k);
        p.alpha = static_cast<float>(alpha);
        p.beta = static_cast<float>(beta);
        auto tiles = [&](int64_t side) {
            const int64_t r = (m + side - 1) / side, c = (n + side - 1) / side;
            return g.batch * (op == kGram || op == kSquare ? r * (r + 1) / 2 : r * c);
        };
        // pairs of CTAs from half a wave of their tiles on
        const int pairs = sm_count / 2;
        const int cg = tiles(2 * kBlock) * 2 >= pairs ? 2 : 1;
        const int64_t t = tiles(cg * kBlock), most = cg == 2 ? pairs : sm_count;
        const dim3 grid(static_cast<unsigned>(cg * (t < most ? t : most)));
        return launch_chained(cg == 1 ? product_of<1>(op) : product_of<2>(op), grid, kThreads, kSmem, cg, s, ma, mb, md,
                              mt, p);
    };
    int now = 0;
    for (int i = 0; i < g.steps; ++i) {
        const double ca = g.coefficients[3 * i], cb = g.coefficients[3 * i + 1], cc = g.coefficients[3 * i + 2];
        const bool last = i + 1 == g.steps;
        e = product(kGram, z.m, z.m, z.n, x_rows[now], x_rows[now], a_store, a_turn, 0.0, kScaleA / (S * S));
        if (e != cudaSuccess) return e;
        e = product(kSquare, z.m, z.m, z.m, a_rows, a_rows, b_store, b_turn, cb * kScaleB / kScaleA,
                    cc * kScaleB / kScaleA / kScaleA);
        if (e != cudaSuccess) return e;
        const double unit = last ? 1.0 / S : 1.0;
        e = product(last ? kLast : kUpdate, z.m, z.n, z.m, b_rows, x_across[now], last ? out_store : x_store[now ^ 1],
                    last ? out_store : a_turn, ca * unit, unit / kScaleB);
        if (e != cudaSuccess) return e;
        now ^= 1;
    }
    return cudaSuccess;
}

}  // namespace nvfp4
