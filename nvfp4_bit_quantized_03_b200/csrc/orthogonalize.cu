// Newton-Schulz orthogonalisation of weight gradients (the update of the Muon optimiser):
//   X = G / (|G|_F + eps);  per step  A = X X^T,  B = b A + c A^2,  X <- a X + B X
// for every matrix of a batch, on the side where X has no more rows than columns (X = G^T otherwise).
// In exact arithmetic a step maps every singular value s of X to a s + b s^3 + c s^5 and keeps the singular
// vectors.
//
// Precision.  Every product takes FP16 operands (11 significant bits) with FP32 accumulation; X itself stays
// in 32 bits between steps, as an FP16 value, which is the products' operand, and the rest to it in FP16 times
// 2^11: 22 bits and more.  A, B and X are held times powers of two that keep their values inside FP16's
// normal range: X times S ~ sqrt(columns), A times 2^12, B times 2^10.  The diagonals of A and B, which become much
// larger than the rest of them, stay in FP32 and out of the products: with A = H + D and B = E + F (D, F diagonal)
//   A^2 = H^2 + H D + D H + D^2,   X <- (a + F) X + E X
// take one product each of the rest, and elements of A and X by the diagonals in the epilogue.  The error of the
// result is then below that of its own rounding to bf16 (emulated in FP64, rms of error over rms of result: 1e-4
// .. 1.0e-3 against 1.7e-3 for the rounding; with the diagonals in FP16 1.2e-3 .. 2.3e-3).  With X itself in FP16 a
// gradient of low rank is lost (1.5e-1: rounding noise of the directions that are not there is raised like
// everything else), with bf16 operands the error is 1e-2 and more.
//
// Where |G|_F is below eps, X = t G / |G|_F with a t that the steps raise by a factor of about a each.  What is then
// held is X 2^-l, with an l of the matrix's own before every step, from the bound t prod (|a| + |b| s^2 + |c| s^4) of
// the singular values, that keeps it at 1 / 4 .. 1 until they get there; and B over a power of two that keeps the larger
// of b 4^l and c 16^l at 1 / 2 .. 1.  So X keeps its 22 bits however small t is, and a step without a its
// product's.  (Held as it is, X was off by 1 % at |G|_F = 1e-8 eps and lost from 1e-10 eps on.)
//
// Kernels: the sum of squares (FP64), the scaled copies of X, then three products per step, one
// kernel each, chained by programmatic launches.  (One kernel that stays on the SMs for all steps, its products
// behind a counter in memory, took 145 against 114 us for 512 x 512 and 1.27 against 1.16 ms for 4096 x 4096: the
// fences around the counter cost more than a launch.)
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

// ---- the steps ---------------------------------------------------------------------------

enum Product { kGram = 0, kSquare = 1, kUpdate = 2, kLast = 3, kFirst = 4 };  // kFirst: the first step's gram

constexpr int kBlock = 128;                    // rows of a CTA's left operand; its tensor-memory lanes
constexpr int kDepth = 64;                     // K per pipeline stage (128 bytes of FP16)
constexpr int kLeftBytes = kBlock * 128;       // 16 KB
constexpr int kBoxBytes = 64 * 128;            // a box of the right operand
constexpr int kEpiWarps = 8;                   // two per lane quarter, half of the columns each
constexpr int kFirstEpi = 2;
constexpr int kGateWarp = kFirstEpi + kEpiWarps;
constexpr int kThreads = 32 * (kGateWarp + 1);
constexpr int kGateBar = 1;                    // named barriers from 1: issuer and gate, one per stage
constexpr int kStaging = 4096;                 // per epilogue warp: 32 rows of 64 values of 2 bytes
constexpr int kBarBytes = 256;
constexpr int kRestBlock = kBlock * kBlock;    // values per block of X's rest
constexpr float kRestUnit = 1.0f / 2048.0f;

// A CTA takes tiles of 128 x 128, a pair of CTAs (CG 2) of 256 x 256; the right operand's rows are split
// between them as the left one's are.
constexpr int kStageBytes = 2 * kLeftBytes;
constexpr int kStages = 6;
constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kStaging + kBarBytes + 1024;
static_assert(kSmem <= 232448, "shared memory per CTA");
// barriers (the same offsets in both CTAs of a pair)
constexpr int kFull = 0;                   // [stages] leader: the stage's bytes of both CTAs landed
constexpr int kEmpty = kFull + kStages;    // [stages] the stage's MMAs completed
constexpr int kAccFull = kEmpty + kStages; // [2] the accumulator is complete
constexpr int kAccEmpty = kAccFull + 2;    // [2] leader: the epilogues have drained it
constexpr int kDrain = kAccEmpty + 2;
constexpr int kBars = kDrain + 1;
static_assert(kBars * 8 + 16 <= kBarBytes, "barrier area");

struct ProductArgs {
    int m, n, k;           // rows and columns of the result, length of the products
    int batch;
    float4* factors;       // this step's of every matrix, kMaxOrthogonalizeSteps apart
    const double2* starts; // |G|_F of every matrix, and with eps
    int steps;
    float coefficients[3 * kMaxOrthogonalizeSteps];
    // result = alpha * (A or X) + beta * accumulator, with the matrix's factors (a, unit, b, c) and powers of two
    // `on_x` (the addend) and `on_acc`; with the diagonals, in FP32: A's sum_i and B's d_i,
    //   gram:   on_acc accumulator; sum_i = diag_acc accumulator_ii
    //   square: on_x (b + c (sum_i + sum_j)) A + on_acc c accumulator; d_i = b sum_i + c (sum_i^2 + diag_acc accumulator_ii)
    //   update: on_x (a + unit d_i) X + on_acc unit accumulator
    float on_x, on_acc, diag_acc;
    float* sums;           // A's diagonal [batch][fours]: written by gram (diag_acc accumulator_ii), read by square
    float2* diagonal;      // with B's diagonal d_i (a + unit d_i, unit) [batch][fours]: written by square, read by update
    int fours;             // m, rounded up to a multiple of 4
    const __half* addend;  // square: A; update: X [batch][m][pitch]
    int64_t pitch;
    __half* rest;          // update: X's rest, blocks of 128 x 128 in the order of the epilogue's lanes
    int rest_rows, rest_cols;  // blocks of a matrix
    uint16_t* out;         // where the results go: last: bf16; small products: also A, B or X
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
    int e, row, col;  // matrix, first row and column
};
// The symmetric products (gram, square) have tiles on and below the diagonal only, row by row; the others go
// down the columns, so that the left operand (m x m) stays in L2 and X is read once.  (Tiles of 256 x 128 by
// pairs: 3.25 against 2.82 ms for 32 of 1408 x 2048, 9.4 against 6.8 for 20480 x 5120; their stages want
// 96 bytes per cycle and SM of L2 where 256 x 256 want 64.)
template <int SIDE>
__host__ __device__ __forceinline__ int64_t tiles_of(bool symmetric, int64_t m, int64_t n)
{
    const int64_t rows = (m + SIDE - 1) / SIDE;
    return symmetric ? rows * (rows + 1) / 2 : rows * ((n + SIDE - 1) / SIDE);
}
template <int SIDE, bool SYMMETRIC>
__device__ __forceinline__ Tile tile_at(int64_t t, int per, int m)
{
    Tile r;
    r.e = static_cast<int>(t / per);
    const int l = static_cast<int>(t - static_cast<int64_t>(r.e) * per);
    if (SYMMETRIC) {
        int k = static_cast<int>((sqrtf(8.0f * l + 1.0f) - 1.0f) * 0.5f);
        while (k * (k + 1) / 2 > l) --k;
        while ((k + 1) * (k + 2) / 2 <= l) ++k;
        r.row = k * SIDE;
        r.col = (l - k * (k + 1) / 2) * SIDE;
    } else {
        const int rows = (m + SIDE - 1) / SIDE;
        r.row = l % rows * SIDE;
        r.col = l / rows * SIDE;
    }
    return r;
}

// 16 values of 2 bytes, 32-byte aligned: one load of a whole sector.
__device__ __forceinline__ void load16(const __half* src, const void* base, int64_t bytes, int* status, uint32_t* v)
{
    if (kBoundsCheck && !(in_buffer(reinterpret_cast<const uint4*>(src), base, bytes, status) &&
                          in_buffer(reinterpret_cast<const uint4*>(src) + 1, base, bytes, status))) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0;
        return;
    }
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(src));
}
// Value k (0 .. N - 1) of v, which becomes 0; 0 for another k.
template <int N>
__device__ __forceinline__ float take(uint32_t* v, int k)
{
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        r = i == k ? v[i] : r;
        v[i] = i == k ? 0u : v[i];
    }
    return __uint_as_float(r);
}
// The l of a matrix's first X 2^-l: 0 where |G|_F / (|G|_F + eps) is 1 / 2 or more, otherwise (by the exponents)
// what leaves 1 / 4 .. 1 of it.
__device__ __forceinline__ int start_power(double root, double norm)
{
    return root > 0.0 && root < 0.5 * norm ? (__double2hiint(root) >> 20) - (__double2hiint(norm) >> 20) + 1 : 0;
}
// The steps' factors (a, unit, b, c) of the matrices, a lane for each, by the loading warp of every CTA of the first
// gram when its loads are on their way: nothing waits for it there (in prepare_kernel they took 3 % of a step of 1024
// of 128 x 512 in registers, a matrix after the other 1 %).
__device__ __forceinline__ void write_factors(const ProductArgs& p, int lane)
{
    const int64_t bytes = 16 * static_cast<int64_t>(p.batch) * kMaxOrthogonalizeSteps;
    const int64_t ctas = gridDim.x;
    for (int64_t e = blockIdx.x + lane * ctas; e < p.batch; e += 32 * ctas) {
        const double2 start = ld_checked(p.starts + e, p.starts, 16 * static_cast<int64_t>(p.batch), p.dev_status);
        float4* const factors = p.factors + e * kMaxOrthogonalizeSteps;
        int low = start_power(start.x, start.y);
        if (low == 0) {  // as for most
            for (int i = 0; i < p.steps; ++i)
                st_checked(factors + i, make_float4(p.coefficients[3 * i], 1.0f, p.coefficients[3 * i + 1],
                                                    p.coefficients[3 * i + 2]),
                           p.factors, bytes, p.dev_status);
            continue;
        }
        double bound = start.x / start.y;
        for (int i = 0; i < p.steps; ++i) {
            const double ca = p.coefficients[3 * i], cb = p.coefficients[3 * i + 1], cc = p.coefficients[3 * i + 2];
            const double square = bound * bound;
            bound *= fabs(ca) + square * (fabs(cb) + square * fabs(cc));
            int next = 0;  // X 2^-next behind the step; behind the last one X itself
            if (low < 0 && i + 1 < p.steps && bound > 0.0 && bound < 0.5) frexp(bound, &next);
            const double b = ldexp(cb, 2 * low), c = ldexp(cc, 4 * low);
            int unit = 0;  // B is held times 2^-unit
            if (low < 0) frexp(fmax(fabs(b), fabs(c)), &unit);
            st_checked(factors + i,
                       make_float4(static_cast<float>(ldexp(ca, low - next)), static_cast<float>(ldexp(1.0, unit + low - next)),
                                   static_cast<float>(ldexp(b, -unit)), static_cast<float>(ldexp(c, -unit))),
                       p.factors, bytes, p.dev_status);
            low = next;
        }
    }
}
// What a product's lane takes its row's values times: the addend (its diagonal's part included), the accumulator, and
// (square) A's diagonal in the value's column.
struct Weights {
    float alpha, beta, gamma;
    float own;  // square: A's diagonal in the row
    float4 f;   // square: the matrix's factors
};
template <int OP>
__device__ __forceinline__ Weights weights_of(const ProductArgs& p, int64_t e, int row)
{
    Weights w = {0.0f, p.on_acc, 0.0f, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
    if (OP == kSquare) {
        const int64_t rows = static_cast<int64_t>(p.batch) * p.fours;
        w.own = row < p.m ? ld_checked(p.sums + e * p.fours + row, p.sums, 4 * rows, p.dev_status) : 0.0f;
        w.f = ld_checked(p.factors + e * kMaxOrthogonalizeSteps, p.factors,
                         16 * ((static_cast<int64_t>(p.batch) - 1) * kMaxOrthogonalizeSteps + 1), p.dev_status);
        w.gamma = p.on_x * w.f.w;
        w.alpha = fmaf(w.gamma, w.own, p.on_x * w.f.z);
        w.beta = p.on_acc * w.f.w;
    } else if (OP != kGram) {
        const int64_t rows = static_cast<int64_t>(p.batch) * p.fours;
        const float2 d = row < p.m ? ld_checked(p.diagonal + e * p.fours + row, p.diagonal, 8 * rows, p.dev_status)
                                   : make_float2(0.0f, 0.0f);
        w.alpha = p.on_x * d.x;
        w.beta = p.on_acc * d.y;
    }
    return w;
}
// A's diagonal in four rows from `row` on, a multiple of 4 (rows behind m hold anything: nothing of them is kept).
__device__ __forceinline__ float4 diagonal_four(const float* d, const ProductArgs& p, int64_t e, int row)
{
    if (row >= p.fours) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    return ld_checked(reinterpret_cast<const float4*>(d + e * p.fours + row), d,
                      4 * static_cast<int64_t>(p.batch) * p.fours, p.dev_status);
}
// Keeps a row's diagonal value of A (gram), or what update makes of B's (square), from its accumulator.
template <int OP>
__device__ __forceinline__ void keep_diagonal(const ProductArgs& p, int64_t e, int row, float acc, const Weights& w)
{
    if (row >= p.m) return;
    const int64_t rows = static_cast<int64_t>(p.batch) * p.fours;
    if (OP == kGram) {
        st_checked(p.sums + e * p.fours + row, p.diag_acc * acc, p.sums, 4 * rows, p.dev_status);
    } else {
        const float d = fmaf(w.f.z, w.own, fmaf(w.f.w * w.own, w.own, w.f.w * p.diag_acc * acc));
        st_checked(p.diagonal + e * p.fours + row, make_float2(fmaf(w.f.y, d, w.f.x), w.f.y), p.diagonal, 8 * rows,
                   p.dev_status);
    }
}
__device__ __forceinline__ float2 halves(uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Warp 0 loads, warp 1 issues the MMAs behind the gate warp, warps 2..9 turn accumulators into results; two
// accumulators, so that a tile's results are written while the next one is multiplied.  In a pair
// (cta_group::2) each CTA holds half of either operand's rows and the accumulator of its 128 rows.
//   What bounds it (B200): a step of K of a pair's tile takes 0.385 us with all SMs at work, 1.6 PFLOP/s, which is
// also the rate of cuBLAS's bf16 product on this GPU: the power limit (clocks fall to 1.4 .. 1.6 GHz; the tensor pipe
// is busy 76 % of those cycles) and the 83 bytes per ns that every SM then reads from L2.  20480 x 5120: gram 370 us,
// square 101, update 777 (2 KB of X and its rest in and out per row of a tile on top).  Single CTAs are bound by
// the 124 bytes per ns that an SM can read: 0.27 us for a step of a quarter of that work.
template <int CG, int OP, bool FIRST>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_d, const __grid_constant__ CUtensorMap map_t,
                   const ProductArgs p)
{
    constexpr int SIDE = kBlock * CG, SLICE = SIDE / 2;  // of a tile; columns of an epilogue warp
    constexpr bool SYMMETRIC = OP == kGram || OP == kSquare;
    constexpr bool ACROSS = OP == kUpdate || OP == kLast;  // the right operand's rows run along K
    constexpr uint32_t IDESC = (1u << 4) | (ACROSS ? 1u << 16 : 0u) | (static_cast<uint32_t>(SIDE >> 3) << 17) |
                               (static_cast<uint32_t>(SIDE >> 4) << 24);
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
    const int per = static_cast<int>(tiles_of<SIDE>(SYMMETRIC, p.m, p.n));
    const int64_t total = static_cast<int64_t>(p.batch) * per;
    const int depth = (p.k + kDepth - 1) / kDepth;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(kFull + s), 1);
            mbar_init(bar(kEmpty + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(kAccFull + b), 1);
            mbar_init(bar(kAccEmpty + b), CG * kEpiWarps);
        }
        mbar_init(bar(kDrain), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_b)) : "memory");
    }
    if (warp == 1) {
        if (CG == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(2 * SIDE)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(2 * SIDE)
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
            const Tile c = tile_at<SIDE, SYMMETRIC>(t, per, p.m);
            const int ya = c.row + rank * kBlock, yb = c.col + rank * kBlock;
            for (int d = 0; d < depth; ++d) {
                if (!wait_bounded(bar(kEmpty + stage), phase ^ 1, abort_flag, p.dev_status)) {
                    ok = false;
                    break;
                }
                if (kBoundsCheck && !(gemm::tma_box_start_ok(d * kDepth, ya, 2, p.dev_status) &&
                                      gemm::tma_box_start_ok(yb, d * kDepth, 2, p.dev_status) &&
                                      c.e < p.batch)) {
                    record_bounds_error(p.dev_status);
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                const uint32_t full = CG == 2 ? leader_address(bar(kFull + stage)) : bar(kFull + stage);
                const uint32_t at = smem_u32(smem + stage * kStageBytes);
                if (rank == 0) mbar_expect_tx(bar(kFull + stage), CG * kStageBytes);
                load_3d<CG>(at, &map_a, d * kDepth, ya, c.e, full);
                if (ACROSS) {
                    load_3d<CG>(at + kLeftBytes, &map_b, yb, d * kDepth, c.e, full);
                    load_3d<CG>(at + kLeftBytes + kBoxBytes, &map_b, yb + 64, d * kDepth, c.e, full);
                } else {
                    load_3d<CG>(at + kLeftBytes, &map_b, d * kDepth, yb, c.e, full);
                    load_3d<CG>(at + kLeftBytes + kBoxBytes, &map_b, d * kDepth, yb + 64, c.e, full);
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
                    if (n) wait_bounded(bar(kFull + s), (n - 1) & 1, abort_flag, nullptr, true, 100000000ull);
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
            const uint32_t acc = tmem + (it & 1) * SIDE;
            for (int d = 0; d < depth; ++d) {
                named_sync(kGateBar + stage, 64);
                if (lane == 0) {
                    tc_fence_after();
                    const uint64_t da = desc_sw128(s0 + stage * kStageBytes);
                    const uint64_t db = ACROSS ? desc_across(s0 + stage * kStageBytes + kLeftBytes)
                                               : desc_sw128(s0 + stage * kStageBytes + kLeftBytes);
#pragma unroll
                    for (int k = 0; k < kDepth / 16; ++k)  // 32 bytes of a row, or 16 rows, further on
                        mma_f16<CG>(acc, da + 2 * k, db + (ACROSS ? 128 : 2) * k, IDESC, (d | k) != 0 ? 1u : 0u);
                    mma_commit<CG>(bar(kEmpty + stage));
                    if (d + 1 == depth) mma_commit<CG>(bar(kAccFull + (it & 1)));
                }
                __syncwarp();
                if (++stage == kStages) stage = 0;
            }
        }
        // every MMA completes before the tensor memory can be freed
        if (lane == 0 && it > 0) {
            mma_commit<CG>(bar(kDrain));
            wait_bounded(bar(kDrain), 0, abort_flag, nullptr, true);
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
                        ok = wait_bounded(bar(kAccEmpty + (it & 1)), ((it >> 1) & 1) ^ 1, abort_flag,
                                          p.dev_status);
                    if (ok) ok = wait_bounded(bar(kFull + stage), phase, abort_flag, p.dev_status);
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
        const int q = warp & 3, half = (warp - kFirstEpi) >> 2;
        const uint32_t stage_buf = smem_u32(staging + (warp - kFirstEpi) * kStaging);
        const int64_t addend_bytes = 2 * static_cast<int64_t>(p.batch) * p.m * p.pitch;
        const int64_t rest_bytes = 2LL * kRestBlock * p.batch * p.rest_rows * p.rest_cols;
        int it = 0;
        for (int64_t t = worker; t < total; t += workers, ++it) {
            const Tile c = tile_at<SIDE, SYMMETRIC>(t, per, p.m);
            const int buf = it & 1;
            const int r0 = c.row + rank * kBlock + 32 * q;  // the warp's rows (one per lane)
            const int row = r0 + lane;
            const int c0 = c.col + half * SLICE;            // its columns
            // what the accumulator is added to, 32 columns (half h of 64) at a time: A or X of the lane's row, and X's rest
            uint32_t add[OP == kGram ? 1 : 32], rest[ACROSS ? 32 : 1];
            auto rest_at = [&](int col) -> __half* {
                const int br = r0 / kBlock, bc = col / kBlock;
                if (br >= p.rest_rows || bc >= p.rest_cols) return nullptr;
                return p.rest + ((static_cast<int64_t>(c.e) * p.rest_rows + br) * p.rest_cols + bc) * kRestBlock +
                       ((q * 16 + (col % kBlock) / 8) * 32 + lane) * 8;
            };
            auto fetch = [&](int col, int h) {
                if (OP != kGram) {
#pragma unroll
                    for (int g = 2 * h; g < 2 * h + 2; ++g) {
                        if (row < p.m && col + 16 * g < p.pitch)
                            load16(p.addend + (static_cast<int64_t>(c.e) * p.m + row) * p.pitch + col + 16 * g, p.addend,
                                   addend_bytes, p.dev_status, add + 8 * g);
                        else
#pragma unroll
                            for (int i = 0; i < 8; ++i) add[8 * g + i] = 0;
                    }
                }
                if (ACROSS) {
                    const __half* const at = rest_at(col);
#pragma unroll
                    for (int g = 4 * h; g < 4 * h + 4; ++g) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (at)
                            v = ld_checked(reinterpret_cast<const uint4*>(at) + 32 * g, p.rest, rest_bytes, p.dev_status);
                        rest[4 * g] = v.x; rest[4 * g + 1] = v.y; rest[4 * g + 2] = v.z; rest[4 * g + 3] = v.w;
                    }
                }
            };
            fetch(c0, 0);  // on its way while the products are summed
            fetch(c0, 1);
            // what the lane's row takes, A's or B's diagonal in it included
            const Weights by_row = weights_of<OP>(p, c.e, row);
            bool ready = lane == 0 ? wait_bounded(bar(kAccFull + buf), (it >> 1) & 1, abort_flag, p.dev_status) : false;
            ready = __shfl_sync(0xFFFFFFFFu, ready ? 1 : 0, 0) != 0;
            if (!ready) break;
            tc_fence_after();
            // 32 columns of the accumulator
            auto accumulator = [&](int at, uint32_t* v) {
                tmem_ld32(tmem + (static_cast<uint32_t>(32 * q) << 16) + buf * SIDE + half * SLICE + 32 * at, v);
                tmem_wait_ld();
                if (at == SLICE / 32 - 1) {  // the last of the warp's slice is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_leader<CG>(bar(kAccEmpty + buf));
                }
            };
#pragma unroll 1
            for (int w = 0; w < SLICE / 64; ++w) {
                const int col = c0 + 64 * w;
                uint32_t packed[32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[32];
                    accumulator(2 * w + h, v);
                    if (SYMMETRIC && r0 == col + 32 * h)  // the diagonal's block
                        keep_diagonal<OP>(p, c.e, row, take<32>(v, lane), by_row);
                    float4 across = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // A's diagonal in four columns
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int i = 16 * h + j;
                        if (OP == kSquare && j % 2 == 0) across = diagonal_four(p.sums, p, c.e, col + 2 * i);
                        float2 f = make_float2(by_row.beta * __uint_as_float(v[2 * j]), by_row.beta * __uint_as_float(v[2 * j + 1]));
                        if (OP != kGram) {
                            float2 x = halves(add[i]), by = make_float2(by_row.alpha, by_row.alpha);
                            if (OP == kSquare) {  // H D + D H
                                by.x += by_row.gamma * (j % 2 ? across.z : across.x);
                                by.y += by_row.gamma * (j % 2 ? across.w : across.y);
                            }
                            if (ACROSS) {
                                const float2 r = halves(rest[i]);
                                x.x += r.x * kRestUnit;
                                x.y += r.y * kRestUnit;
                            }
                            f.x += by.x * x.x;
                            f.y += by.y * x.y;
                        }
                        packed[i] = OP == kLast ? pack_bf16(f.x, f.y) : pack_half(f.x, f.y);
                        if (OP == kUpdate) {
                            const float2 o = halves(packed[i]);
                            rest[i] = pack_half((f.x - o.x) * (1.0f / kRestUnit), (f.y - o.y) * (1.0f / kRestUnit));
                        }
                    }
                    if (OP == kUpdate) {
                        __half* const at = rest_at(col);
#pragma unroll
                        for (int g = 4 * h; at && g < 4 * h + 4; ++g)
                            st_checked(reinterpret_cast<uint4*>(at) + 32 * g,
                                       make_uint4(rest[4 * g], rest[4 * g + 1], rest[4 * g + 2], rest[4 * g + 3]), p.rest,
                                       rest_bytes, p.dev_status);
                    }
                    if (w + 1 < SLICE / 64) fetch(col + 64, h);  // under the other half's work
                }
                const bool inside = r0 < p.m && col < p.n;
                const bool direct = OP != kLast || !p.transposed;
                // a symmetric result's other half; a tile on the diagonal holds both
                const bool turned = SYMMETRIC ? c.row != c.col : (OP == kLast && p.transposed);
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
    if (FIRST && warp == 0) write_factors(p, lane);

    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if (CG == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * SIDE)
                         : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * SIDE)
                         : "memory");
    }
}

// ---- the steps' small products ---------------------------------------------------------------
//
// Where larger tiles are too few for the SMs, CTAs take one of 128 x 64 each; or a cluster of 2 or 4 takes one: each
// CTA sums a part of K, copies to every other CTA of the cluster the sums of that one's columns (bulk copies
// between shared memories), and writes the results of its own.  The order of the additions is that of the parts.
//   What bounds it (B200, 512 x 512, clusters of 4): latency.  Of 4.9 us per product 1.3 lie between the kernels, 1.4
// until the sums of 2 steps of K are there, 1.2 in the exchange, 1.0 in the results.  Tiles of 128 x 128 by clusters
// exchange twice the sums and took 6.4 us; written straight to the other CTAs' memory by the lanes the sums took
// 2.2 us instead of 0.6 + 0.6.

constexpr int kNarrow = 64;                     // columns of a tile
constexpr int kNarrowStage = kLeftBytes + kBoxBytes;
constexpr int kNarrowStages = 6;
constexpr int kExchange = kBlock * kNarrow * 4; // the sums of a CTA's columns from all parts
constexpr int kNarrowEpi = 8;                   // epilogue warps, two per lane quarter, half of the columns each
constexpr int kNarrowGate = 2 + kNarrowEpi;     // the issuer's gate, as in the kernel of the larger tiles
constexpr int kNarrowThreads = 32 * (kNarrowGate + 1);
constexpr int kNarrowBar = 2;                   // named barriers from 2: issuer and gate (1 is the epilogue's)
constexpr int kNarrowSmem = kNarrowStages * kNarrowStage + kExchange + kBarBytes + 1024;
static_assert(kNarrowSmem <= 232448 && (2 * kNarrowStages + 2) * 8 + 16 <= kBarBytes, "shared memory per CTA");

__host__ __device__ __forceinline__ int64_t narrow_tiles(bool symmetric, int64_t m, int64_t n)
{
    const int64_t rows = (m + kBlock - 1) / kBlock;
    // below the diagonal and in its blocks
    return symmetric ? rows * (rows - 1) + (m - (rows - 1) * kBlock + kNarrow - 1) / kNarrow
                           + 2 * (rows - 1) : rows * ((n + kNarrow - 1) / kNarrow);
}
template <bool SYMMETRIC>
__device__ __forceinline__ Tile narrow_tile_at(int t, int per, int m)
{
    Tile r;
    r.e = t / per;
    const int l = t - r.e * per;
    if (SYMMETRIC) {  // 2 k + 2 tiles in row k of tiles (the last row may lack its last one)
        int k = static_cast<int>((sqrtf(4.0f * l + 1.0f) - 1.0f) * 0.5f);
        while (k * (k + 1) > l) --k;
        while ((k + 1) * (k + 2) <= l) ++k;
        r.row = k * kBlock;
        r.col = (l - k * (k + 1)) * kNarrow;
    } else {
        const int rows = (m + kBlock - 1) / kBlock;
        r.row = l % rows * kBlock;
        r.col = l / rows * kNarrow;
    }
    return r;
}

// `bytes` of this CTA's shared memory to the same place of CTA `cta`, whose barrier counts them.
__device__ __forceinline__ void copy_to_cta(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar, uint32_t cta)
{
    asm volatile(
        "{\n\t.reg .b32 to, there;\n\t"
        "mapa.shared::cluster.u32 to, %0, %4;\n\t"
        "mapa.shared::cluster.u32 there, %3, %4;\n\t"
        "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [to], [%1], %2, [there];\n\t}" ::"r"(dst),
        "r"(src), "r"(bytes), "r"(bar), "r"(cta)
        : "memory");
}

template <int OP, int PARTS, bool FIRST>
__global__ void __launch_bounds__(kNarrowThreads, 1)
    narrow_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const ProductArgs p)
{
    constexpr bool SYMMETRIC = OP == kGram || OP == kSquare;
    constexpr bool ACROSS = OP == kUpdate || OP == kLast;
    constexpr uint32_t IDESC = (1u << 4) | (ACROSS ? 1u << 16 : 0u) | (static_cast<uint32_t>(kNarrow >> 3) << 17) |
                               (static_cast<uint32_t>(kBlock >> 4) << 24);
    constexpr int FULL = 0, EMPTY = kNarrowStages, ACC_FULL = 2 * kNarrowStages, SUMS = ACC_FULL + 1;
    constexpr int WIDTH = kNarrow / PARTS;                 // columns that a CTA writes
    constexpr int SHARE = WIDTH * kBlock;                  // their sums from one part
    constexpr int GROUPS = WIDTH / 16;                     // of 8 columns of a warp
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    float4* exchange = reinterpret_cast<float4*>(smem + kNarrowStages * kNarrowStage);
    // the shares for the others take the stages' place when the products are summed
    float4* shares = reinterpret_cast<float4*>(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kNarrowStages * kNarrowStage + kExchange);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kNarrowStages + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PARTS > 1 ? static_cast<int>(cluster_rank()) : 0;
    const Tile c = narrow_tile_at<SYMMETRIC>(static_cast<int>(blockIdx.x) / PARTS,
                                             static_cast<int>(narrow_tiles(SYMMETRIC, p.m, p.n)), p.m);
    const int depth = (p.k + kDepth - 1) / kDepth;
    const int first = depth * rank / PARTS, last = depth * (rank + 1) / PARTS;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kNarrowStages + 2; ++i) mbar_init(bar(i), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_b)) : "memory");
    }
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kNarrow)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (PARTS > 1 && threadIdx.x == 0) mbar_expect_tx(bar(SUMS), (PARTS - 1) * SHARE * 4);
    if (PARTS > 1) cluster_sync();  // the cluster's CTAs run, and count, before one copies to another
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // everything this kernel reads is the work of the kernels ahead
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // the epilogue's rows and, in groups of 8, columns; what the sums are added to
    const int q = warp & 3, half = warp >= 6 ? 1 : 0;
    const int row = c.row + 32 * q + lane, col0 = c.col + rank * WIDTH + half * (WIDTH / 2);
    const bool writes = warp >= 2 && warp < kNarrowGate && row < p.m;
    uint32_t v[32];  // sums of the lane's row, 32 columns
    Weights by_row = {};
    const int64_t plane = static_cast<int64_t>(c.e) * p.m;
    const int64_t matrix_values = static_cast<int64_t>(p.batch) * p.m * p.pitch;
    uint4 add[GROUPS], rest[GROUPS];
    uint4* rest_at = nullptr;
    const int64_t rest_bytes = 2LL * kRestBlock * p.batch * p.rest_rows * p.rest_cols;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- loads ----------------
            asm volatile("fence.proxy.async;" ::: "memory");  // copies written by ordinary stores
            uint32_t fills = 0;
            for (int d = first; d < last; ++d, ++fills) {
                const int stage = static_cast<int>(fills % kNarrowStages);
                if (!wait_bounded(bar(EMPTY + stage), (fills / kNarrowStages & 1) ^ 1, abort_flag, p.dev_status)) break;
                if (kBoundsCheck && !(gemm::tma_box_start_ok(d * kDepth, c.row, 2, p.dev_status) &&
                                      gemm::tma_box_start_ok(c.col, d * kDepth, 2, p.dev_status) && c.e < p.batch)) {
                    record_bounds_error(p.dev_status);
                    *abort_flag = 1;
                    break;
                }
                const uint32_t full = bar(FULL + stage), at = smem_u32(smem + stage * kNarrowStage);
                mbar_expect_tx(full, kNarrowStage);
                load_3d<1>(at, &map_a, d * kDepth, c.row, c.e, full);
                load_3d<1>(at + kLeftBytes, &map_b, ACROSS ? c.col : d * kDepth, ACROSS ? d * kDepth : c.col, c.e, full);
            }
            if (*abort_flag)  // copies already issued land before the CTA can exit
                for (uint32_t s = 0; s < kNarrowStages; ++s) {
                    const uint32_t n = fills > s ? (fills - s + kNarrowStages - 1) / kNarrowStages : 0u;
                    if (n) wait_bounded(bar(FULL + s), (n - 1) & 1, abort_flag, nullptr, true);
                }
        }
        __syncwarp();
        if (FIRST) write_factors(p, lane);
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        uint32_t fills = 0;
        for (int d = first; d < last; ++d, ++fills) {
            const int stage = static_cast<int>(fills % kNarrowStages);
            named_sync(kNarrowBar + stage, 64);
            if (lane == 0) {
                tc_fence_after();
                const uint32_t at = smem_u32(smem + stage * kNarrowStage);
                const uint64_t da = desc_sw128(at), db = ACROSS ? desc_across(at + kLeftBytes) : desc_sw128(at + kLeftBytes);
#pragma unroll
                for (int k = 0; k < kDepth / 16; ++k)
                    mma_f16<1>(tmem, da + 2 * k, db + (ACROSS ? 128 : 2) * k, IDESC, fills != 0 || k != 0 ? 1u : 0u);
                mma_commit<1>(bar(EMPTY + stage));
                if (d + 1 == last) mma_commit<1>(bar(ACC_FULL));
            }
            __syncwarp();
        }
        // the tensor memory is freed behind them
        if (lane == 0) wait_bounded(bar(ACC_FULL), 0, abort_flag, nullptr, true);
        __syncwarp();
    } else if (warp == kNarrowGate) {
        bool ok = true;
        uint32_t fills = 0;
        for (int d = first; d < last; ++d, ++fills) {
            const int stage = static_cast<int>(fills % kNarrowStages);
            if (lane == 0 && ok)
                ok = wait_bounded(bar(FULL + stage), fills / kNarrowStages & 1, abort_flag, p.dev_status);
            __syncwarp();
            named_sync(kNarrowBar + stage, 64);
        }
    } else {
        // ---------------- sums to the CTAs that write them ----------------
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            add[g] = rest[g] = make_uint4(0, 0, 0, 0);
            const int col = col0 + 8 * g;
            if (OP != kGram && writes && col < p.pitch)
                add[g] = ld_checked(reinterpret_cast<const uint4*>(p.addend + (plane + row) * p.pitch + col), p.addend,
                                    2 * matrix_values, p.dev_status);
            if (ACROSS) {
                rest_at = reinterpret_cast<uint4*>(p.rest) +
                          (((static_cast<int64_t>(c.e) * p.rest_rows + c.row / kBlock) * p.rest_cols + c.col / kBlock) *
                               (kRestBlock / 8) + (q * 16 + col0 % kBlock / 8) * 32 + lane);
                rest[g] = ld_checked(rest_at + 32 * g, p.rest, rest_bytes, p.dev_status);
            }
        }
        by_row = weights_of<OP>(p, c.e, row);
        bool ready = lane == 0 ? wait_bounded(bar(ACC_FULL), 0, abort_flag, p.dev_status) : false;
        ready = __shfl_sync(0xFFFFFFFFu, ready ? 1 : 0, 0) != 0;
        if (ready) {
            tc_fence_after();
            tmem_ld32(tmem + (static_cast<uint32_t>(32 * q) << 16) + 32 * half, v);
            tmem_wait_ld();
            if (PARTS > 1) {
                float4* dst = shares + 8 * half * kBlock + 32 * q + lane;  // [owner][4 columns][row]
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dst[i * kBlock] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                  __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
                fence_async_smem();
            }
        }
        if (PARTS > 1) {
            named_sync(1, 32 * kNarrowEpi);
            const int owner = static_cast<int>(threadIdx.x) - 64;
            if (ready && owner < PARTS && owner != rank)
                copy_to_cta(smem_u32(exchange + rank * (SHARE / 4)), smem_u32(shares + owner * (SHARE / 4)), SHARE * 4,
                            bar(SUMS), static_cast<uint32_t>(owner));
            if (lane == 0) wait_bounded(bar(SUMS), 0, abort_flag, p.dev_status);
            __syncwarp();
        }
    }
    // the cluster's CTAs stay until each has what the others sent
    if (PARTS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (writes) {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int col = col0 + 8 * g;
            if (col >= p.n) break;
            float f[8];
            if (PARTS == 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * g + i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = 0.0f;
#pragma unroll
                for (int i = 0; i < PARTS; ++i) {
                    const float4* src = (i == rank ? shares : exchange) + i * (SHARE / 4) +
                                        (half * (WIDTH / 8) + 2 * g) * kBlock + 32 * q + lane;
                    const float4 lo = src[0], hi = src[kBlock];
                    f[0] += lo.x; f[1] += lo.y; f[2] += lo.z; f[3] += lo.w;
                    f[4] += hi.x; f[5] += hi.y; f[6] += hi.z; f[7] += hi.w;
                }
            }
            if (SYMMETRIC && row >= col && row < col + 8) {  // the diagonal
                uint32_t bits[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) bits[i] = __float_as_uint(f[i]);
                keep_diagonal<OP>(p, c.e, row, take<8>(bits, row - col), by_row);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(bits[i]);
            }
            const uint32_t aw[4] = {add[g].x, add[g].y, add[g].z, add[g].w};
            const uint32_t rw[4] = {rest[g].x, rest[g].y, rest[g].z, rest[g].w};
            uint32_t o[4], r[4];
            float4 across = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // A's diagonal in four columns
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 x = make_float2(by_row.beta * f[2 * i], by_row.beta * f[2 * i + 1]);
                if (OP != kGram) {
                    float2 to = halves(aw[i]), by = make_float2(by_row.alpha, by_row.alpha);
                    if (OP == kSquare) {  // H D + D H
                        if (i % 2 == 0) across = diagonal_four(p.sums, p, c.e, col + 2 * i);
                        by.x += by_row.gamma * (i % 2 ? across.z : across.x);
                        by.y += by_row.gamma * (i % 2 ? across.w : across.y);
                    }
                    if (ACROSS) {
                        const float2 s = halves(rw[i]);
                        to.x += s.x * kRestUnit;
                        to.y += s.y * kRestUnit;
                    }
                    x.x += by.x * to.x;
                    x.y += by.y * to.y;
                }
                o[i] = OP == kLast ? pack_bf16(x.x, x.y) : pack_half(x.x, x.y);
                if (OP == kUpdate) {
                    const float2 w = halves(o[i]);
                    r[i] = pack_half((x.x - w.x) * (1.0f / kRestUnit), (x.y - w.y) * (1.0f / kRestUnit));
                }
            }
            if (OP == kUpdate) st_checked(rest_at + 32 * g, make_uint4(r[0], r[1], r[2], r[3]), p.rest, rest_bytes, p.dev_status);
            // rows of the intermediate matrices end on 128 bytes
            const int64_t out_values = OP == kLast ? (p.batch - 1) * p.out_stride + ((p.transposed ? p.n : p.m) - 1) * p.ldo +
                                                         (p.transposed ? p.m : p.n)
                                                   : static_cast<int64_t>(p.batch) * p.m * p.ldo;
            uint16_t* const out = p.out + c.e * p.out_stride;
            if (OP != kLast || !p.transposed) {
                uint16_t* dst = out + static_cast<int64_t>(row) * p.ldo + col;
                if (OP != kLast || p.by_tma) {
                    st_checked(reinterpret_cast<uint4*>(dst), make_uint4(o[0], o[1], o[2], o[3]), p.out, 2 * out_values,
                               p.dev_status);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (col + i < p.n)
                            st_checked(dst + i, static_cast<uint16_t>(o[i / 2] >> (16 * (i & 1))), p.out, 2 * out_values,
                                       p.dev_status);
                }
            }
            if (SYMMETRIC ? c.row / kBlock != c.col / kBlock : (OP == kLast && p.transposed)) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (col + i < p.n)
                        st_checked(out + static_cast<int64_t>(col + i) * p.ldo + row,
                                   static_cast<uint16_t>(o[i / 2] >> (16 * (i & 1))), p.out, 2 * out_values, p.dev_status);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kNarrow) : "memory");
    }
    __syncwarp();
    if (PARTS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- the norm and the scaled copies --------------------------------------------------------

constexpr int kNormThreads = 256;

struct PrepareArgs {
    const void* g;
    int64_t rows, cols, ldg, g_stride;  // of G
    int64_t m, n, pitch;                // of X (G or G^T) and of its FP16 copy
    int batch, transposed;
    int by_fours;                       // G's rows can be read four values at a time
    int parts;                          // partial sums per matrix
    double* partials;                   // [batch][parts]
    __half* rest;
    int rest_rows, rest_cols;
    __half* x;
    double scale, eps;
    double2* starts;                    // [batch]: |G|_F, and with eps
    int* dev_status;
};

template <bool F32>
__device__ __forceinline__ float element(const PrepareArgs& a, int64_t at, int64_t bytes)
{
    if (F32) return ldg_checked(static_cast<const float*>(a.g) + at, a.g, bytes, a.dev_status);
    const uint16_t v = ldg_checked(static_cast<const uint16_t*>(a.g) + at, a.g, bytes, a.dev_status);
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// Four of them (by_fours: 16-byte, bf16 8-byte aligned).
template <bool F32>
__device__ __forceinline__ float4 four(const PrepareArgs& a, int64_t at, int64_t bytes)
{
    if (F32)
        return ldg_checked(reinterpret_cast<const float4*>(static_cast<const float*>(a.g) + at), a.g, bytes, a.dev_status);
    const uint2 v = ldg_checked(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.g) + at), a.g, bytes,
                                a.dev_status);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
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

// Partial sums of the squares, in FP64: no value of FP32 or bf16 leaves its range when squared.  Bound by HBM: B200,
// 20480 x 5120 FP32 69 us (6.1 TB/s).
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
    const int warps = kNormThreads / 32, lane = threadIdx.x & 31;
    for (int64_t i = blockIdx.x * warps + (threadIdx.x >> 5); i < a.rows * pieces;
         i += static_cast<int64_t>(gridDim.x) * warps) {
        const int64_t r = i / pieces, c0 = (i - r * pieces) * 1024;
        const int64_t end = c0 + 1024 < a.cols ? c0 + 1024 : a.cols;
        const int64_t base = e * a.g_stride + r * a.ldg;
        if (a.by_fours) {
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int64_t c = c0 + 4 * (lane + 32 * k);
                v[k] = c < end ? four<F32>(a, base + c, bytes) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const double x = v[k].x, y = v[k].y, z = v[k].z, w = v[k].w;
                sum += x * x + y * y + (z * z + w * w);
            }
        } else {
#pragma unroll 8
            for (int64_t c = c0 + lane; c < end; c += 32) {
                const double v = element<F32>(a, base + c, bytes);
                sum += v * v;
            }
        }
    }
    sum = block_sum(sum, shared);
    if (threadIdx.x == 0)
        st_checked(a.partials + e * a.parts + blockIdx.x, sum, a.partials,
                   8 * static_cast<int64_t>(a.batch) * a.parts, a.dev_status);
}

// X times the scale over the norm: in FP16 row by row, and the rest to it in the order of the products' epilogue.
// A CTA takes pieces of 32 rows x 128 columns of X through shared memory (G^T: both sides stay coalesced), all
// of a piece's loads in flight.  Bound by HBM and the passes between barriers: B200, 32 of 1408 x 2048 FP32 146 us
// (5.1 TB/s), 20480 x 5120 (turned) 181 us (4.6 TB/s); with FP64 products and loads one by one 186 and 209.
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
    // the scale as a power of two and the rest of it: no product of a value with either leaves FP32 on the way,
    // and the result is rounded once
    float power = 0.0f, factor = 0.0f;
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
            const double root = sqrt(sum), norm = root + a.eps;
            if (l == 0 && threadIdx.x == 0)
                st_checked(a.starts + e, make_double2(root, norm), a.starts, 16 * static_cast<int64_t>(a.batch),
                           a.dev_status);
            // norm 2^l, in its exponent (an ldexp behind the division took 40 registers instead of 32)
            const double divisor = __hiloint2double(__double2hiint(norm) + start_power(root, norm) * (1 << 20),
                                                    __double2loint(norm));
            // zeros stay zeros, whatever eps: its inverse may leave FP32
            const double scale = sum > 0.0 ? a.scale / divisor : 0.0;
            int exponent = 0;
            const double mantissa = frexp(scale, &exponent);
            power = ldexpf(1.0f, exponent / 2);
            factor = static_cast<float>(ldexp(mantissa, exponent - exponent / 2));
            have = e;
            if (!finite && l == 0 && threadIdx.x == 0 && a.dev_status) atomicOr(a.dev_status, 1);  // NONFINITE
        }
        __syncthreads();  // the piece before has left the tile
        // values that are not there, or of a matrix that is not finite, count as zeros
        auto scaled = [&](float v, bool there) { return there && finite ? v * power * factor : 0.0f; };
        if (a.transposed) {
            const int64_t r = r0 + lane;
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int64_t cc = c0 + warp + 8 * k;
                v[k] = r < a.m && cc < a.n ? element<F32>(a, e * a.g_stride + cc * a.ldg + r, bytes) : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) tile[lane][warp + 8 * k] = scaled(v[k], true);
        } else if (a.by_fours) {
            float4 v[4];
            const int64_t cc = c0 + 4 * lane;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t r = r0 + warp + 8 * k;
                v[k] = r < a.m && cc < a.n ? four<F32>(a, e * a.g_stride + r * a.ldg + cc, bytes)
                                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4*>(&tile[warp + 8 * k][4 * lane]) =
                    make_float4(scaled(v[k].x, true), scaled(v[k].y, true), scaled(v[k].z, true), scaled(v[k].w, true));
        } else {
            for (int r = warp; r < 32; r += kNormThreads / 32)
#pragma unroll
                for (int c = lane; c < 128; c += 32) {
                    const bool there = r0 + r < a.m && c0 + c < a.n;
                    tile[r][c] = scaled(there ? element<F32>(a, e * a.g_stride + (r0 + r) * a.ldg + c0 + c, bytes) : 0.0f,
                                        there);
                }
        }
        __syncthreads();
        const int64_t block = (e * a.rest_rows + r0 / kBlock) * a.rest_cols + c0 / kBlock;
        uint4* dst = reinterpret_cast<uint4*>(a.rest + block * kRestBlock) + (r0 % kBlock) / 32 * 16 * 32;
        const int64_t rest_bytes = 2LL * kRestBlock * a.batch * a.rest_rows * a.rest_cols;
        for (int c8 = warp; c8 < 16; c8 += kNormThreads / 32) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = *reinterpret_cast<const float2*>(&tile[lane][8 * c8 + 2 * i]);
                const float2 h = halves(pack_half(f.x, f.y));
                o[i] = pack_half((f.x - h.x) * (1.0f / kRestUnit), (f.y - h.y) * (1.0f / kRestUnit));
            }
            st_checked(dst + c8 * 32 + lane, make_uint4(o[0], o[1], o[2], o[3]), a.rest, rest_bytes, a.dev_status);
        }
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

template <int CG>
auto product_of(int op)
{
    switch (op) {
        case kFirst: return product_kernel<CG, kGram, true>;
        case kGram: return product_kernel<CG, kGram, false>;
        case kSquare: return product_kernel<CG, kSquare, false>;
        case kUpdate: return product_kernel<CG, kUpdate, false>;
        default: return product_kernel<CG, kLast, false>;
    }
}
template <int PARTS>
auto narrow_of(int op)
{
    switch (op) {
        case kFirst: return narrow_kernel<kGram, PARTS, true>;
        case kGram: return narrow_kernel<kGram, PARTS, false>;
        case kSquare: return narrow_kernel<kSquare, PARTS, false>;
        case kUpdate: return narrow_kernel<kUpdate, PARTS, false>;
        default: return narrow_kernel<kLast, PARTS, false>;
    }
}
auto narrow_of(int op, int parts)
{
    return parts == 1 ? narrow_of<1>(op) : (parts == 2 ? narrow_of<2>(op) : narrow_of<4>(op));
}

// Once per device: the kernels' shared memory, and how many pairs and clusters of 1, 2, 4 can run at once.
struct Resident {
    int singles, pairs, clusters[3];  // clusters of 2^i CTAs
};
cudaError_t resident_on_device(int sm_count, Resident* out)
{
    constexpr int kDevices = 64;
    static Resident known[kDevices] = {};
    static std::mutex mutex;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= kDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mutex);
    Resident& r = known[device];
    if (r.singles == 0) {
        cudaError_t e = cudaSuccess;
        for (int op = kGram; op <= kFirst; ++op) {
            const cudaFuncAttribute attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
            if ((e = cudaFuncSetAttribute(product_of<1>(op), attr, kSmem)) != cudaSuccess) return e;
            if ((e = cudaFuncSetAttribute(product_of<2>(op), attr, kSmem)) != cudaSuccess) return e;
            for (int parts = 1; parts <= 4; parts *= 2)
                if ((e = cudaFuncSetAttribute(narrow_of(op, parts), attr, kNarrowSmem)) != cudaSuccess) return e;
        }
        for (int i = 0; i < 3; ++i) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 1u << i;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            cfg.gridDim = dim3(static_cast<unsigned>(sm_count >> i << i));
            cfg.blockDim = dim3(kNarrowThreads);
            cfg.dynamicSmemBytes = kNarrowSmem;
            e = cudaOccupancyMaxActiveClusters(&r.clusters[i], narrow_of(kGram, 1 << i), &cfg);
            if (e != cudaSuccess) return e;
            if (i == 1) {
                cfg.blockDim = dim3(kThreads);
                cfg.dynamicSmemBytes = kSmem;
                e = cudaOccupancyMaxActiveClusters(&r.pairs, product_of<2>(kGram), &cfg);
                if (e != cudaSuccess) return e;
            }
        }
        if (r.pairs < 1) return cudaErrorInvalidConfiguration;
        r.singles = sm_count;
    }
    *out = r;
    return cudaSuccess;
}

// How a product is spread over the SMs: tiles of 128 x 128 by single CTAs, of 256 x 256 by pairs, or (parts > 0) a
// tile of 128 x 64 by a cluster of `parts` (all of which are resident at once).  Chosen by estimated time; the estimate
// ranks the ways and predicts none (update of 1024 x 4096 12.6 us where it takes 17, its gram 13.9 where it takes 9).  Whole
// calls with one way for all three products, us (B200; singles / pairs / clusters of 1, 2, 4):
//   512 x 512     116 / 154 / 100, 91, 81      1024 x 1024   143 / 187 / 141, 153, 291
//   768 x 3000    184 / 229 / 222, 241, 392    2048 x 2048   270 / 279 / 558, ..
//   16 of 256 x 512  108 / 133 / 117, ..       2816 x 2816   614 / 451 / 1346, ..
// and with the choice 81, 124, 151, 248, 102, 440.
// Over 46 sizes from 128 x 512 to 2688 x 4096, in batches of 1 to 64, no other way for one of the products was more
// than 4 % faster than the choice (1536 x 4096: updates by pairs 331, by singles 350; 16 of 768 x 2048: gram by pairs 569, by
// singles 599).
struct Plan {
    int cg, parts;
    int64_t workers;
};
Plan plan_of(bool symmetric, int64_t batch, int64_t m, int64_t n, int64_t k, const Resident& r)
{
    // us: a step of K (see the kernels), what a wave of single tiles adds, and the rest of a kernel.  A pair's tile takes
    // at least its results' 5 us, which lie under the next one's products
    const int64_t depth = (k + kDepth - 1) / kDepth;
    const int64_t small = batch * tiles_of<128>(symmetric, m, n), large = batch * tiles_of<256>(symmetric, m, n);
    const int64_t narrow = batch * narrow_tiles(symmetric, m, n);
    const double single = static_cast<double>((small + r.singles - 1) / r.singles) *
                              (static_cast<double>(depth) * 0.27 + 1.0) + 4.0;
    const double tile = static_cast<double>(depth) * 0.385;
    const double pair = static_cast<double>((large + r.pairs - 1) / r.pairs - 1) * (tile > 5.0 ? tile : 5.0) + tile + 6.4;
    Plan best = pair <= single ? Plan{2, 0, large < r.pairs ? large : r.pairs}
                               : Plan{1, 0, small < r.singles ? small : r.singles};
    double time = pair <= single ? pair : single;
    for (int i = 0; i < 3; ++i) {
        const int64_t parts = int64_t(1) << i;
        if (parts > depth || narrow > r.clusters[i]) continue;
        const double clusters = static_cast<double>((depth + parts - 1) / parts) * 0.3 + (parts == 1 ? 3.7 : 4.3);
        if (clusters <= time) {
            time = clusters;
            best = Plan{1, static_cast<int>(parts), narrow};
        }
    }
    return best;
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
    int64_t m, n, x_pitch, a_pitch, rest_rows, rest_cols;
    int parts;
    size_t partials, starts, factors, rest, x, a, sums, diagonal;  // bytes
};

Sizes sizes_of(int64_t batch, int64_t rows, int64_t cols)
{
    Sizes s;
    s.m = rows < cols ? rows : cols;
    s.n = rows < cols ? cols : rows;
    s.x_pitch = (s.n + 63) / 64 * 64;  // rows of whole 128-byte lines
    s.a_pitch = (s.m + 63) / 64 * 64;
    s.rest_rows = (s.m + kBlock - 1) / kBlock;
    s.rest_cols = (s.n + kBlock - 1) / kBlock;
    // partial sums: 16 K values each, no more than fill the SMs several times
    int64_t parts = (rows * cols + 16383) / 16384;
    const int64_t most = batch < 592 ? 592 / batch : 1;
    s.parts = static_cast<int>(parts < most ? parts : most);
    s.partials = round256(8 * static_cast<size_t>(batch) * s.parts);
    s.starts = round256(sizeof(double2) * static_cast<size_t>(batch));
    s.factors = round256(sizeof(float4) * static_cast<size_t>(batch) * kMaxOrthogonalizeSteps);
    s.rest = round256(2 * static_cast<size_t>(kRestBlock) * batch * s.rest_rows * s.rest_cols);
    s.x = round256(2 * static_cast<size_t>(batch) * s.m * s.x_pitch);
    s.a = round256(2 * static_cast<size_t>(batch) * s.m * s.a_pitch);
    s.sums = round256(4 * static_cast<size_t>(batch) * ((s.m + 3) / 4 * 4));
    s.diagonal = round256(8 * static_cast<size_t>(batch) * ((s.m + 3) / 4 * 4));
    return s;
}

}  // namespace

size_t orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols)
{
    const Sizes s = sizes_of(batch, rows, cols);
    return 256 + s.partials + s.starts + s.factors + s.rest + 2 * s.x + 2 * s.a + s.sums + s.diagonal;
}

cudaError_t orthogonalize_ways(int64_t batch, int64_t rows, int64_t cols, int sm_count, int* ways)
{
    Resident resident;
    const cudaError_t e = resident_on_device(sm_count, &resident);
    if (e != cudaSuccess) return e;
    const Sizes z = sizes_of(batch, rows, cols);
    const Plan plans[3] = {plan_of(true, batch, z.m, z.m, z.n, resident), plan_of(true, batch, z.m, z.m, z.m, resident),
                           plan_of(false, batch, z.m, z.n, z.m, resident)};
    for (int i = 0; i < 3; ++i) ways[i] = plans[i].parts > 0 ? plans[i].parts : plans[i].cg * kBlock;
    return cudaSuccess;
}

cudaError_t launch_orthogonalize(const OrthogonalizeArgs& g, int sm_count, cudaStream_t s)
{
    Resident resident;
    cudaError_t e = resident_on_device(sm_count, &resident);
    if (e != cudaSuccess) return e;
    const Sizes z = sizes_of(g.batch, g.rows, g.cols);
    const bool transposed = g.rows > g.cols;
    // on a 256-byte boundary: rows are read 32 bytes at a time
    uint8_t* at = reinterpret_cast<uint8_t*>(round256(reinterpret_cast<uintptr_t>(g.workspace)));
    double* partials = reinterpret_cast<double*>(at);
    double2* starts = reinterpret_cast<double2*>(at += z.partials);
    float4* factors = reinterpret_cast<float4*>(at += z.starts);
    __half* rest = reinterpret_cast<__half*>(at += z.factors);
    __half* x[2];
    x[0] = reinterpret_cast<__half*>(at += z.rest);
    x[1] = reinterpret_cast<__half*>(at += z.x);
    __half* a = reinterpret_cast<__half*>(at += z.x);
    __half* b = reinterpret_cast<__half*>(at += z.a);
    float* sums = reinterpret_cast<float*>(at += z.a);
    float2* diagonal = reinterpret_cast<float2*>(at += z.sums);

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
    const int64_t size = g.f32 ? 4 : 2;
    pa.by_fours = reinterpret_cast<uintptr_t>(g.g) % (4 * size) == 0 && g.cols % 4 == 0 && g.ldg % 4 == 0 && g.g_stride % 4 == 0;
    pa.parts = z.parts;
    pa.partials = partials;
    pa.rest = rest;
    pa.rest_rows = static_cast<int>(z.rest_rows);
    pa.rest_cols = static_cast<int>(z.rest_cols);
    pa.x = x[0];
    pa.scale = S;
    pa.eps = g.eps;
    pa.starts = starts;
    pa.dev_status = g.dev_status;

    // left operands in boxes of 128 rows x 64 of K, right ones of 64 rows (across: of K) x 64, stores of 32 x 64
    // or, turned, 64 x 32
    CUtensorMap x_left[2], x_right[2], x_store[2], a_left, a_right, b_left, a_store, b_store, a_turn, b_turn, out_store;
    bool ok = true;
    auto map_of = [&](CUtensorMap* map, __half* data, int64_t cols, int64_t pitch, int box_x, int box_y, bool swizzle) {
        ok = ok && make_map(map, data, cols, z.m, g.batch, pitch, z.m * pitch, box_x, box_y, swizzle);
    };
    for (int i = 0; i < 2; ++i) {
        map_of(&x_left[i], x[i], z.n, z.x_pitch, kDepth, kBlock, true);
        map_of(&x_right[i], x[i], z.n, z.x_pitch, 64, 64, true);
        map_of(&x_store[i], x[i], z.n, z.x_pitch, 64, 32, true);
    }
    map_of(&a_left, a, z.m, z.a_pitch, kDepth, kBlock, true);
    map_of(&a_right, a, z.m, z.a_pitch, 64, 64, true);
    map_of(&b_left, b, z.m, z.a_pitch, kDepth, kBlock, true);
    map_of(&a_store, a, z.m, z.a_pitch, 64, 32, true);
    map_of(&b_store, b, z.m, z.a_pitch, 64, 32, true);
    map_of(&a_turn, a, z.m, z.a_pitch, 32, 64, false);
    map_of(&b_turn, b, z.m, z.a_pitch, 32, 64, false);
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
    const int64_t pieces = g.batch * ((z.m + 31) / 32) * z.rest_cols;
    const dim3 prepare_grid(static_cast<unsigned>(pieces < 8 * sm_count ? pieces : 8 * sm_count));
    e = launch_chained(g.f32 ? prepare_kernel<true> : prepare_kernel<false>, prepare_grid, kNormThreads, 0, 1, s, pa);
    if (e != cudaSuccess) return e;

    ProductArgs p = {};
    p.batch = static_cast<int>(g.batch);
    p.sums = sums;
    p.diagonal = diagonal;
    p.fours = static_cast<int>((z.m + 3) / 4 * 4);
    p.rest = rest;
    p.rest_rows = pa.rest_rows;
    p.rest_cols = pa.rest_cols;
    p.transposed = transposed;
    p.by_tma = by_tma;
    p.dev_status = g.dev_status;
    p.starts = starts;
    p.steps = g.steps;
    for (int i = 0; i < 3 * g.steps; ++i) p.coefficients[i] = g.coefficients[i];
    auto product = [&](int op, int64_t n, int64_t k, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& md,
                       const CUtensorMap& mt, const __half* addend, int64_t pitch, __half* out, double on_x,
                       double on_acc, double diag_acc) {
        p.m = static_cast<int>(z.m);
        p.n = static_cast<int>(n);
        p.k = static_cast<int>(k);
        p.addend = addend;
        p.pitch = pitch;
        p.on_x = static_cast<float>(on_x);
        p.on_acc = static_cast<float>(on_acc);
        p.diag_acc = static_cast<float>(diag_acc);
        p.out = op == kLast ? static_cast<uint16_t*>(g.out) : reinterpret_cast<uint16_t*>(out);
        p.ldo = op == kLast ? g.ldo : (op == kUpdate ? z.x_pitch : z.a_pitch);
        p.out_stride = op == kLast ? g.out_stride : z.m * p.ldo;
        const Plan plan = plan_of(op != kUpdate && op != kLast, g.batch, z.m, n, k, resident);
        if (plan.parts > 0)
            return launch_chained(narrow_of(op, plan.parts), dim3(static_cast<unsigned>(plan.parts * plan.workers)),
                                  kNarrowThreads, kNarrowSmem, plan.parts, s, ma, mb, p);
        return launch_chained(plan.cg == 1 ? product_of<1>(op) : product_of<2>(op),
                              dim3(static_cast<unsigned>(plan.cg * plan.workers)), kThreads, kSmem, plan.cg, s, ma, mb, md,
                              mt, p);
    };
    int now = 0;
    for (int i = 0; i < g.steps; ++i) {
        const bool last = i + 1 == g.steps;
        p.factors = factors + i;
        // A = X X^T from the products of S X
        e = product(i == 0 ? kFirst : kGram, z.m, z.n, x_left[now], x_right[now], a_store, a_turn, nullptr, z.a_pitch, a, 0.0,
                    kScaleA / (S * S), 1.0 / (S * S));
        if (e != cudaSuccess) return e;
        // B = b A + c A^2 with A = H + D
        e = product(kSquare, z.m, z.m, a_left, a_right, b_store, b_turn, a, z.a_pitch, b, kScaleB / kScaleA,
                    kScaleB / kScaleA / kScaleA, 1.0 / kScaleA / kScaleA);
        if (e != cudaSuccess) return e;
        // X <- (a + F) X + E X with B = E + F
        const double unit = last ? 1.0 / S : 1.0;
        e = product(last ? kLast : kUpdate, z.n, z.m, b_left, x_right[now], last ? out_store : x_store[now ^ 1],
                    last ? out_store : a_turn, x[now], z.x_pitch, x[now ^ 1], unit, unit / kScaleB, 0.0);
        if (e != cudaSuccess) return e;
        now ^= 1;
    }
    return cudaSuccess;
}

}  // namespace nvfp4
