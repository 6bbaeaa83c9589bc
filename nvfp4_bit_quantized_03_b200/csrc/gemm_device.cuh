// Building blocks of the block-scaled FP4 GEMM kernels (gemm.cu: one product; gemm_grouped.cu: the
// products of a mixture layer's experts): the pair tile's shape and shared-memory plan, mbarrier
// waits bounded in time, TMA copies, the tcgen05 operations, the decode factor, the epilogue's
// stores and the tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cfloat>
#include <cstdint>
#include <mutex>

#include "bounds_check.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace gemm {

constexpr int CTA_M = 128;              // A rows per CTA (tensor-memory lanes)
constexpr int PAIR_M = 2 * CTA_M;       // rows of a pair tile
constexpr int BN = 256;                 // columns of a pair tile (B rows), N of the MMA
constexpr int B_ROWS = BN / 2;          // B rows each CTA loads
constexpr int BK = 256;                 // K elements per pipeline stage (128 bytes per row)
constexpr int MMA_K = 64;               // K per tcgen05.mma of kind::mxf4nvf4
constexpr int A_BYTES = CTA_M * BK / 2;  // 16 KB
constexpr int B_BYTES = B_ROWS * BK / 2;  // 16 KB
constexpr int SF_TILE = 512;            // 128 rows x 4 blocks of scales
constexpr int SFA_BYTES = (BK / MMA_K) * SF_TILE;      // 2 KB: this CTA's 128 A rows
constexpr int SFB_BYTES = 2 * (BK / MMA_K) * SF_TILE;  // 4 KB: all 256 B rows of the tile
constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;  // 38 KB
constexpr int NUM_SF_WARPS = 4;         // one per 32-lane quarter of tensor memory
constexpr int NUM_EPI_WARPS = 16;       // four per lane quarter, 64 accumulator columns each
constexpr int FIRST_SF_WARP = 2;
constexpr int FIRST_EPI_WARP = FIRST_SF_WARP + NUM_SF_WARPS;
constexpr int GATE_WARP = FIRST_EPI_WARP + NUM_EPI_WARPS;
constexpr int THREADS = 32 * (GATE_WARP + 1);
constexpr uint32_t GATE_BAR0 = 3;       // named barriers 3 .. 3 + STAGES - 1: issuer + gate
constexpr uint32_t GATE_THREADS = 64;   // (1 is the epilogue's)
constexpr int TMEM_COLS = 512;
constexpr int ACC_COL = 0;              // accumulator: columns [0, 256)
constexpr int SF_COL = BN;              // scales: 48 columns per stage from column 256
constexpr int SF_COLS_PER_STAGE = (BK / MMA_K) * (4 + 8);
constexpr int BAR_BYTES = 256;

// Pipeline shape per output type.  Five operand stages either way.  A tile's output (64 KB per
// CTA in bf16, 128 KB in FP32) goes out through a 2 KB staging buffer per epilogue warp: TMA
// store rounds of 32 rows x 64 bytes, two for bf16 and four for FP32.  (With 512-byte buffers,
// eight bf16 rounds whose store round trips follow one another bounded the epilogue: B200,
// 8192 x 20480 x K, 0.421 -> 0.365 ms at K = 5120 and 0.322 -> 0.114 ms at K = 1024; delays
// that paced the small rounds away from the next tile's loads no longer help.  FP32 rows
// stored straight from registers were slower than the staged boxes: 0.387 against 0.375 ms at
// 20480 x 5120 x 8192, 0.200 against 0.146 ms at 8192 x 20480 x 1024.)
template <bool BF16>
struct Pipe {
    static constexpr int STAGES = 5;
    static constexpr int STAGING_BYTES = 2048;  // per epilogue warp
    static constexpr int SMEM_BYTES =
        STAGES * STAGE_BYTES + NUM_EPI_WARPS * STAGING_BYTES + BAR_BYTES + 1024;
    // shared-memory barrier slots (the same offsets in both CTAs of a pair)
    static constexpr int BAR_FULL = 0;                     // [STAGES] this CTA's TMA bytes landed
    static constexpr int BAR_EMPTY = BAR_FULL + STAGES;    // [STAGES] the stage's MMAs completed
    static constexpr int BAR_SF = BAR_EMPTY + STAGES;      // [STAGES] leader: both CTAs' scales in TMEM
    static constexpr int BAR_ACC_FULL = BAR_SF + STAGES;   // the tile's accumulator is complete
    static constexpr int BAR_ACC_EMPTY = BAR_ACC_FULL + 1; // leader: both CTAs' epilogues drained it
    static constexpr int BAR_DRAIN = BAR_ACC_EMPTY + 1;    // teardown after an abort
    static constexpr int NUM_BARS = BAR_DRAIN + 1;
    static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
    static_assert(NUM_BARS * 8 + 16 <= BAR_BYTES, "barrier area (+ TMEM slot, abort and go flags)");
    static_assert(SF_COL + STAGES * SF_COLS_PER_STAGE <= TMEM_COLS, "tensor memory budget");
};
constexpr unsigned long long WAIT_LIMIT_NS = 2000000000ull;  // 2 s per wait
constexpr int kDevTimeoutBit = 2;       // NVFP4_DEVSTAT_TIMEOUT

static_assert(STAGE_BYTES % 1024 == 0, "stages must keep 1024-byte alignment (128B swizzle)");

// Instruction descriptor of tcgen05.mma kind::mxf4nvf4: A and B E2M1 (format 1), both
// K-major, N >> 3 at bit 17, M >> 4 at bit 24 (M = 256: the pair's rows), dense K = 64; bit 23
// selects the scale type: 0 = UE4M3 (NVFP4), 1 = UE8M0 (MXFP4, whose 32-block scales fill both
// 16-element slots).
constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(BN >> 3) << 17) |
                           (static_cast<uint32_t>(PAIR_M >> 4) << 24);
constexpr uint32_t IDESC_UE8M0 = IDESC | (1u << 23);

__device__ __forceinline__ uint32_t smem_u32(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t globaltimer()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// ---- mbarrier ----------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// Arrive on the barrier at the same shared-memory offset in CTA `cta` of the cluster (this
// CTA's own when cta is its rank).  The arrive keeps the default (CTA-scope release)
// semantics: what it publishes to the peer is tensor-memory traffic, which the tcgen05 fences
// around it order (tcgen05.fence::before_thread_sync here, ::after_thread_sync after the wait);
// a cluster-scope release costs about half a microsecond per arrive on B200.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar, uint32_t cta)
{
    asm volatile(
        "{\n\t.reg .b32 remote;\n\t"
        "mapa.shared::cluster.u32 remote, %0, %1;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [remote];\n\t}" ::"r"(bar),
        "r"(cta)
        : "memory");
}
// Non-blocking test of the phase with the given parity.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of both CTAs of the pair.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Wait for the phase of `bar` with the given parity to complete.  Gives up when another
// role has aborted (unless `ignore_abort`) or after WAIT_LIMIT_NS, which it reports.
static __device__ __noinline__ bool wait_bounded_slow(uint32_t bar, uint32_t parity,
                                               volatile int* abort_flag, int* dev_status,
                                               bool ignore_abort, unsigned long long limit_ns)
{
    const uint64_t t0 = globaltimer();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 31u) == 0) {
            if (!ignore_abort && *abort_flag) return false;
            if (globaltimer() - t0 > limit_ns) {
                *abort_flag = 1;
                if (dev_status) atomicOr(dev_status, kDevTimeoutBit);
                return false;
            }
        }
    }
}
// For the accumulator hand-off between the MMA issuer and the epilogue, where the waiting
// thread is alone and the wake-up latency of a suspended try_wait shows in every tile: spin on
// the non-blocking test, with the same time limit and abort handling as wait_bounded.
static __device__ __noinline__ bool wait_spin(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                       int* dev_status)
{
    if (mbar_test_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t i = 1;; ++i) {
        if (mbar_test_wait(bar, parity)) return true;
        if ((i & 63u) == 0) {
            if (*abort_flag) return false;
            if (globaltimer() - t0 > WAIT_LIMIT_NS) {
                *abort_flag = 1;
                if (dev_status) atomicOr(dev_status, kDevTimeoutBit);
                return false;
            }
        }
    }
}

// Named barrier among `threads` threads (whole warps), id 1..15.
__device__ __forceinline__ void named_sync(uint32_t id, uint32_t threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The common case -- the phase has already completed -- costs one try_wait, inline.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity,
                                             volatile int* abort_flag, int* dev_status,
                                             bool ignore_abort = false,
                                             unsigned long long limit_ns = WAIT_LIMIT_NS)
{
    if (mbar_try_wait(bar, parity)) return true;
    return wait_bounded_slow(bar, parity, abort_flag, dev_status, ignore_abort, limit_ns);
}

// ---- TMA / bulk copies -------------------------------------------------------------------
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int32_t x,
                                            int32_t y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x,
                                            int32_t y, int32_t z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t x,
                                             int32_t y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(x), "r"(y), "r"(src)
        : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Debug builds (bounds_check.cuh): a tiled TMA box must start at non-negative coordinates with
// its innermost coordinate on a 16-byte boundary (x * element bytes); a start beyond the far
// edge is legal (loads zero-fill, stores are clipped).  Records NVFP4_DEVSTAT_BOUNDS otherwise.
__device__ __forceinline__ bool tma_box_start_ok(int x, int y, int elem_bytes, int* dev_status)
{
    if (x >= 0 && y >= 0 && (x * elem_bytes) % 16 == 0) return true;
    record_bounds_error(dev_status);
    return false;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- tcgen05 -----------------------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor, K-major with 128-byte swizzle: rows of 128 bytes, groups
// of 8 rows 1024 bytes apart (stride byte offset), version 1, layout type 2.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}
// Register -> tensor memory stores of one warp's 32 lanes: 16 or 32 consecutive columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
        "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One block-scaled MMA of the pair, issued by the leader CTA: D (256 x 256, rows 0-127 in the
// leader's tensor memory, 128-255 in the peer's) += A . B^T over K = 64, where the descriptors'
// shared-memory offsets select each CTA's 128 A rows and 128 B rows, and the scale addresses
// each CTA's own scale columns (its A rows, all 256 B rows).
template <bool MX>
__device__ __forceinline__ void mma_nvf4_pair(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                              uint32_t sfa, uint32_t sfb, uint32_t accumulate)
{
    constexpr uint32_t idesc = MX ? IDESC_UE8M0 : IDESC;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X "
        "[%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}

// Arrive on the barrier at offset `bar` of both CTAs once every MMA the leader issued so far
// has completed.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(0x3))
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
        "[%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
          "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
          "=r"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Tensor encode scale of an operand, as the quantizer computed it; see Alpha below.
__device__ __forceinline__ float operand_scale(float amax)
{
    if (amax == 0.0f) return 1.0f;
    const float s = __fdiv_rn(2688.0f, amax);
    return s > FLT_MAX ? FLT_MAX : s;
}

// The epilogue's decode factor 1 / (S_enc,A S_enc,B), applied as two FP32 multiplies
// D = (acc * a1) * a2.  The product of two FP32 encode scales spans 2^-256 .. 2^256, beyond
// FP32, so it is formed in FP64 (the 24 x 24-bit product is exact, the reciprocal rounded
// once) and split into a1 = m 2^e1 (m in [1, 2), e1 = e clamped to [-100, 70]) and the power
// of two a2 = 2^(e - e1).  A non-zero accumulator lies in [2^-20, 2^54] (products of E2M1
// values, at least 1/2, and E4M3 scales, at least 2^-9; K < 2^31 terms of at most 6^2 448^2),
// so acc * a1 is always a normal FP32 value and the only rounding that matters is the last
// one.  When e - e1 falls outside [-149, 127] it is clamped: then every non-zero |acc| / (S_A
// S_B) is below 2^-194 or above 2^177, and the clamped product rounds to the same 0 or Inf.
// Non-finite operands (amax = Inf) give 0; MXFP4 operands carry no tensor scale (a1 = a2 = 1).
struct Alpha {
    float a1, a2;
};

__device__ __forceinline__ float pow2f(int e)  // 2^e for e in [-149, 127], exact
{
    return e >= -126 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23)
                     : __uint_as_float(1u << (e + 149));
}

template <bool MX>
__device__ __forceinline__ Alpha epilogue_alpha(float amax_a, float amax_b)
{
    const bool finite = (amax_a < INFINITY) && (amax_b < INFINITY) && amax_a >= 0.0f &&
                        amax_b >= 0.0f;
    if (!finite) return Alpha{0.0f, 1.0f};
    if (MX) return Alpha{1.0f, 1.0f};
    const double alpha = 1.0 / (static_cast<double>(operand_scale(amax_a)) *
                                static_cast<double>(operand_scale(amax_b)));
    const int e = static_cast<int>((__double_as_longlong(alpha) >> 52) & 0x7FF) - 1023;
    const int e1 = e < -100 ? -100 : (e > 70 ? 70 : e);
    int e2 = e - e1;
    e2 = e2 < -149 ? -149 : (e2 > 127 ? 127 : e2);
    // alpha * 2^-(e - e1) by exponent arithmetic on the FP64 pattern (exact), then to FP32
    const double scaled = __longlong_as_double(__double_as_longlong(alpha) -
                                               (static_cast<long long>(e - e1) << 52));
    return Alpha{__double2float_rn(scaled), pow2f(e2)};
}

__device__ __forceinline__ float apply_alpha(uint32_t acc_bits, const Alpha& al)
{
    return __fmul_rn(__fmul_rn(__uint_as_float(acc_bits), al.a1), al.a2);
}

// One epilogue warp's 32 x 64 slice of the tile (row `lane`, values v[0..63] in FP32 bits) to
// global memory, scaled by alpha and converted, through the warp's staging buffer with TMA bulk
// tensor stores.
//  * bf16: 2 rounds of 64 bytes (32 columns) of every row; FP32: 4 rounds of 64 bytes
//    (16 columns).  Boxes of 32 rows x 64 bytes: row `lane` sits at lane * 64 with its four
//    16-byte chunks permuted by the 64-byte swizzle (chunk c at c ^ ((row / 2) % 4)), which
//    keeps the warp's 16-byte shared stores conflict-free and which the tensor map undoes.
// Each round waits only for the previous box to leave the buffer.
// With AMAX (bf16 only) the warp also folds its slice into the two maxima the next quantizer
// of D needs: m_plain, the largest |bf16| bit pattern (in the low 16 bits of each half), and
// m_rht, the largest |v| bit pattern of the random Hadamard transform of every 16 consecutive
// rows (lanes 0-15 and 16-31; lane = row) before its x1/4: the sign of row i flips when bit i of
// sign_mask is set, then butterflies of widths 1, 2, 4, 8 across lanes (shfl_xor), the lower
// lane keeping a + b and the upper a - b -- the same FP32 operations, in the same order, as the
// quantizer's transform of the bf16 values.
template <bool BF16, bool AMAX = false>
__device__ __forceinline__ void store_slice(const uint32_t* v, const Alpha& alpha, uint32_t stage_buf,
                                            int lane, const CUtensorMap* tmap_d, int n0, int y,
                                            int M, int N, uint32_t* m_plain = nullptr,
                                            uint32_t* m_rht = nullptr, uint32_t flip = 0,
                                            int* dev_status = nullptr)
{
    constexpr int CHUNKS = 4;                        // 16-byte chunks per box row
    constexpr int COLS = CHUNKS * (BF16 ? 8 : 4);    // columns per box row
    const uint32_t row_base = stage_buf + 16 * CHUNKS * lane;
    const uint32_t swz = (lane >> 1) & 3;
#pragma unroll
    for (int r = 0; r < 64 / COLS; ++r) {
        if (lane == 0) bulk_wait_read();  // the previous box has left the buffer
        __syncwarp();
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            uint32_t o[4];
            if (BF16) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int j = r * COLS + c * 8 + 2 * h;
                    const __nv_bfloat162 b2 =
                        __floats2bfloat162_rn(apply_alpha(v[j], alpha), apply_alpha(v[j + 1], alpha));
                    o[h] = *reinterpret_cast<const uint32_t*>(&b2);
                }
                if (AMAX) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) *m_plain = __vmaxu2(*m_plain, o[h] & 0x7FFF7FFFu);
                    float f[8];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        f[2 * h] = __uint_as_float((o[h] << 16) ^ flip);
                        f[2 * h + 1] = __uint_as_float((o[h] & 0xFFFF0000u) ^ flip);
                    }
#pragma unroll
                    for (int w = 1; w < 16; w <<= 1) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float other = __shfl_xor_sync(0xFFFFFFFFu, f[k], w);
                            f[k] = (lane & w) ? __fsub_rn(other, f[k]) : __fadd_rn(f[k], other);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *m_rht = max(*m_rht, __float_as_uint(f[k]) & 0x7FFFFFFFu);
                }
            } else {
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    o[h] = __float_as_uint(apply_alpha(v[r * 16 + c * 4 + h], alpha));
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row_base + 16 * (c ^ swz)),
                         "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                         : "memory");
        }
        fence_async_smem();
        __syncwarp();
        const int x = n0 + r * COLS;
        if (lane == 0 && y < M && x < N &&
            (!kBoundsCheck || tma_box_start_ok(x, y, BF16 ? 2 : 4, dev_status)))
            tma_store_2d(tmap_d, stage_buf, x, y);
    }
}

// ---- host side ---------------------------------------------------------------------------

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// 2D map over a codes buffer (rows x K/2 bytes), boxes of `box_rows` x 128 bytes, 128-byte
// swizzle, zero fill outside the tensor (boxes may start beyond the last row).
inline bool make_codes_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box_rows)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(BK / 2), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3D map over a scale buffer in the MMA layout, as 32-bit words: x = the 128 words of one
// 512-byte tile, y = the K tile (4 blocks = 64 elements of K), z = the 128-row group; boxes of
// 4 K tiles x `groups` row groups, zero fill beyond the buffer (ragged K, padding groups).
inline bool make_scales_map(CUtensorMap* map, const uint8_t* scales, int64_t rows, int64_t K, int groups)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {SF_TILE / 4, static_cast<cuuint64_t>(K / MMA_K),
                                static_cast<cuuint64_t>((rows + 127) / 128)};
    const cuuint64_t strides[2] = {SF_TILE, static_cast<cuuint64_t>(K / MMA_K) * SF_TILE};
    const cuuint32_t box[3] = {SF_TILE / 4, BK / MMA_K, static_cast<cuuint32_t>(groups)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(scales), dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2D map over D (rows x N elements, row stride ldd) for the epilogue's bulk tensor stores
// (the map clips rows beyond M): boxes of 32 rows x 64 bytes with the 64-byte swizzle.
inline bool make_output_map(CUtensorMap* map, void* D, int64_t M, int64_t N, int64_t ldd, bool bf16)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const int64_t esize = bf16 ? 2 : 4;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ldd * esize)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(64 / esize), 32};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, D,
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gemm
}  // namespace nvfp4
