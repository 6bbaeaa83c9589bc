// Block-scaled NVFP4 products over the experts of a mixture layer, on the sm_100a tcgen05 tensor
// cores.  The rows of an expert-ordered matrix belong to experts in turn: expert e owns the rows
// offsets[e] .. offsets[e + 1], a multiple of 128, known only on the device.
//   by rows : D[r, n] = sum_k A[r, k] B_e[n, k] for the rows r of every expert e (forward and data
//             gradient).  The E matrices B_e are slices of one operand: N rows each, stacked
//             (forward, W), or K columns each, side by side (data gradient, W^T).
//   by K    : D_e[m, n] = sum over the columns r of expert e of A[m, r] B[n, r] (weight
//             gradient), zero for an expert without rows.
//
// The pipeline is the single product's (gemm.cu): persistent CTA pairs over 256 x 256 tiles, one
// tcgen05.mma.cta_group::2 accumulation each, TMA producer, scale stagers, gate, issuer and
// epilogue warps.  What differs is the schedule: every CTA reads the offsets once, keeps them and
// the running count of 256-row tiles in shared memory (4 bytes an expert), and each role finds a
// tile's expert by binary search.  No host knowledge of the routing is needed, so a call can be
// captured and replayed.  A tile may cover rows of the next expert (regions are multiples of 128,
// tiles of 256) and a K block columns of it: such rows are computed and not stored, such columns are
// loaded and not multiplied.
//
// B200, by rows: 8192 tokens to 8 of 64 experts, 4096 -> 2048, bf16 out: 265-290 us (1.1 TFLOP, 3.8-4.1
// PFLOP/s, the single product's rate at such K less the half tiles); one token to 8 experts, 4096
// -> 4096: 23 us against 11.6 for its weights' bytes.  By K: 36700 rows, 32 x 2048 x 4096 FP32 out,
// 250-290 us; the 2.1 GB output of 64 experts alone takes 390 us (5.5 TB/s), with 1024 rows each 475.
// Tried on both ends and not kept (same results):
//  * loading only the 32-row quarters of A with tokens: 16 K blocks 14.4 against 12.1 us, the
//    smaller boxes land later; skipping the empty half of a tile: the same time;
//  * L2 prefetch of the weights ahead of the ring, by box or by row: one token 31-32 against 29 us;
//  * by K with 4 stages and two staging buffers, or 128-byte output boxes: 261 against 252 us, and the
//    same change by rows 418 against 388: the fifth stage is worth more.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "gemm_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
using namespace gemm;
namespace {

struct GroupedParams {
    const int32_t* offsets;  // experts + 1 row offsets
    int experts;
    int rows;                // rows of the expert-ordered operands
    const float* amax_a;
    const float* amax_b;
    int M;                   // by K: rows of each D_e
    int N;                   // columns of D
    int K;                   // by rows: reduction length
    int b_row_step;          // by rows: B_e starts at row e * b_row_step, column e * b_k_step
    int b_k_step;
    int* dev_status;
};

// The schedule's tables behind the barriers: offsets / 128 and the 256-row tiles before each expert.
constexpr int SCHEDULE_BYTES = 2 * 2 * (kMaxExperts + 1);
template <bool BF16>
constexpr int grouped_smem()
{
    return Pipe<BF16>::SMEM_BYTES + SCHEDULE_BYTES;
}
static_assert(grouped_smem<true>() <= 232448 && grouped_smem<false>() <= 232448,
              "shared memory per CTA");

struct Tile {
    int a_row, b_row;     // first rows of the operands
    int a_k, b_k;         // first elements along K
    int steps;            // K steps of 64
    int d_row, d_end;     // first output row, end of the expert's output rows
    int col;              // first output column
    __device__ int k_blocks() const { return (steps + BK / MMA_K - 1) / (BK / MMA_K); }
};

struct Schedule {
    uint16_t* off128;  // [experts + 1] offsets / 128
    uint16_t* first;   // [experts + 1] row tiles of the experts before
    int experts, tiles_m, tiles_n, M, K, b_row_step, b_k_step;

    template <bool BY_K>
    __device__ int total() const
    {
        return (BY_K ? experts * tiles_m : first[experts]) * tiles_n;
    }
    template <bool BY_K>
    __device__ int steps(int t) const
    {
        if (!BY_K) return K / MMA_K;
        const int e = t / (tiles_m * tiles_n);
        const int n = off128[e + 1] - off128[e];
        return n > 0 ? n * (128 / MMA_K) : 0;
    }
    // Row tiles innermost: the pairs at work share an expert's weights, each stripe of which is
    // then read from memory about once.
    template <bool BY_K>
    __device__ Tile tile(int t) const
    {
        Tile c;
        if (BY_K) {
            const int per = tiles_m * tiles_n, e = t / per, local = t - e * per;
            const int tn = local / tiles_m, tm = local - tn * tiles_m;
            c.a_row = tm * PAIR_M;
            c.b_row = tn * BN;
            c.a_k = c.b_k = off128[e] * 128;
            c.steps = steps<true>(t);
            c.d_row = e * M + tm * PAIR_M;
            c.d_end = (e + 1) * M;
            c.col = tn * BN;
            return c;
        }
        int lo = 0, hi = experts;  // first[lo] * tiles_n <= t < first[hi] * tiles_n
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] * tiles_n <= t) lo = mid;
            else hi = mid;
        }
        const int n = max(1, first[lo + 1] - first[lo]), local = t - first[lo] * tiles_n;
        const int tn = local / n, tm = local - tn * n;
        c.a_row = c.d_row = off128[lo] * 128 + tm * PAIR_M;
        c.d_end = off128[lo + 1] * 128;
        c.b_row = lo * b_row_step + tn * BN;
        c.a_k = 0;
        c.b_k = lo * b_k_step;
        c.steps = K / MMA_K;
        c.col = tn * BN;
        return c;
    }
};

// Fill the tables: thread e takes expert e, the running tile counts are an inclusive scan in
// `scratch` (32 words).  Offsets outside the matrix are clamped to it.
__device__ __forceinline__ void build_schedule(const Schedule& s, const int32_t* offsets, int rows,
                                               int* scratch)
{
    static_assert(THREADS >= kMaxExperts + 1, "a thread per table entry");
    const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
    int o = 0, tiles = 0;
    if (e <= s.experts) {
        o = min(max(offsets[e], 0), rows) / 128;
        if (e < s.experts) tiles = max(0, (min(max(offsets[e + 1], 0), rows) / 128 - o + 1) / 2);
    }
    int sum = tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += v;
    }
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += scratch[w];
    if (e <= s.experts) {
        s.off128[e] = static_cast<uint16_t>(o);
        s.first[e] = static_cast<uint16_t>(sum - tiles);
    }
    __syncthreads();
}

template <bool BF16, bool BY_K>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    gemm_grouped_kernel(const __grid_constant__ CUtensorMap tmap_a,
                     const __grid_constant__ CUtensorMap tmap_b,
                     const __grid_constant__ CUtensorMap tmap_sfa,
                     const __grid_constant__ CUtensorMap tmap_sfb,
                     const __grid_constant__ CUtensorMap tmap_d, const GroupedParams p)
{
    using P = Pipe<BF16>;
    constexpr int STAGES = P::STAGES, STAGING_BYTES = P::STAGING_BYTES;
    constexpr int BAR_FULL = P::BAR_FULL, BAR_EMPTY = P::BAR_EMPTY, BAR_SF = P::BAR_SF;
    constexpr int BAR_ACC_FULL = P::BAR_ACC_FULL, BAR_ACC_EMPTY = P::BAR_ACC_EMPTY;
    constexpr int BAR_DRAIN = P::BAR_DRAIN, NUM_BARS = P::NUM_BARS;
    extern __shared__ uint8_t smem_raw[];
    // Both CTAs of a pair lay out their shared memory identically: the MMA, the commits and
    // the remote arrivals address the peer's buffers and barriers by the same offsets.
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* staging = smem + STAGES * STAGE_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(staging + NUM_EPI_WARPS * STAGING_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NUM_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* epi_go = abort_flag + 1;  // the epilogue's waiter tells the other warps
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();             // 0: leader (issues the MMAs), 1: peer
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
    Schedule sch;
    sch.off128 = reinterpret_cast<uint16_t*>(bars) + BAR_BYTES / 2;
    sch.first = sch.off128 + kMaxExperts + 1;
    sch.experts = p.experts;
    sch.tiles_m = BY_K ? (p.M + PAIR_M - 1) / PAIR_M : 0;
    sch.tiles_n = (p.N + BN - 1) / BN;
    sch.K = p.K;
    sch.b_row_step = p.b_row_step;
    sch.b_k_step = p.b_k_step;
    sch.M = p.M;
    build_schedule(sch, p.offsets, p.rows, reinterpret_cast<int*>(staging));
    const int total = sch.total<BY_K>();

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(BAR_FULL + s), 1);
            mbar_init(bar(BAR_EMPTY + s), 1);
            mbar_init(bar(BAR_SF + s), 2 * NUM_SF_WARPS);
        }
        mbar_init(bar(BAR_ACC_FULL), 1);
        mbar_init(bar(BAR_ACC_EMPTY), 2 * NUM_EPI_WARPS);  // every epilogue warp of the pair
        mbar_init(bar(BAR_DRAIN), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_b)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_sfa)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_sfb)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_d)) : "memory");
    }
    if (warp == 1) {
        // one warp of each CTA allocates the pair's tensor memory (the same columns in both)
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers are initialised before either signals the other
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        // Four copies per stage: this CTA's A box and B box (128 rows x 128 bytes each, 128-byte
        // swizzle) and two boxes of the scale maps: this CTA's 128 A rows and both 128-row
        // groups of the tile's B rows, 4 scale tiles (one 256-wide K block) each.  Every box is
        // full size: the maps zero-fill rows, row groups and K tiles beyond the matrices.
        int stage = 0;
        uint32_t phase = 0;
        uint32_t fills = 0;  // stages filled so far
        bool ok = true;
        auto load_b = [&](const Tile& c, int kb, uint32_t st, uint32_t full) {
            tma_load_2d(st + A_BYTES, &tmap_b, c.b_k / 2 + kb * (BK / 2),
                        c.b_row + static_cast<int>(rank) * B_ROWS, full);
            tma_load_3d(st + A_BYTES + B_BYTES + SFA_BYTES, &tmap_sfb, 0,
                        c.b_k / MMA_K + kb * (BK / MMA_K), c.b_row / CTA_M, full);
        };
        // By rows the weights do not come from the kernel ahead: the ring is filled with them while
        // it ends.
        uint32_t ahead = 0;
        if (!BY_K && !kBoundsCheck) {
            for (int t = cluster; t < total && ahead < STAGES; t += clusters) {
                const Tile c = sch.tile<BY_K>(t);
                for (int kb = 0; kb < c.k_blocks() && ahead < STAGES; ++kb, ++ahead) {
                    const uint32_t full = bar(BAR_FULL + ahead);
                    mbar_expect_tx(full, STAGE_BYTES);
                    load_b(c, kb, smem_u32(smem + ahead * STAGE_BYTES), full);
                }
            }
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
        for (int t = cluster; t < total && ok; t += clusters) {
            const Tile c = sch.tile<BY_K>(t);
            const int ya = c.a_row + static_cast<int>(rank) * CTA_M;  // this CTA's A rows
            for (int kb = 0; kb < c.k_blocks(); ++kb) {
                if (!wait_bounded(bar(BAR_EMPTY + stage), phase ^ 1, abort_flag, p.dev_status)) {
                    ok = false;
                    break;
                }
                const int xa = c.a_k / 2 + kb * (BK / 2);
                if (kBoundsCheck && !(tma_box_start_ok(xa, ya, 1, p.dev_status) &&
                                      tma_box_start_ok(c.b_k / 2 + kb * (BK / 2), c.b_row, 1,
                                                       p.dev_status))) {
                    // no copy for this stage: the roles waiting for it stop at the abort flag
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                const uint32_t full = bar(BAR_FULL + stage);
                const uint32_t st = smem_u32(smem + stage * STAGE_BYTES);
                if (fills >= ahead) {
                    mbar_expect_tx(full, STAGE_BYTES);
                    load_b(c, kb, st, full);
                }
                tma_load_2d(st, &tmap_a, xa, ya, full);
                tma_load_3d(st + A_BYTES + B_BYTES, &tmap_sfa, 0,
                            c.a_k / MMA_K + kb * (BK / MMA_K), ya / CTA_M, full);
                ++fills;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) {
            // Let every copy already issued land before the CTA can exit: slot s was filled
            // n_s times, and its last fill completes phase n_s - 1 of its full barrier.
            for (int s = 0; s < STAGES; ++s) {
                // (a slot with only its weights under way never completes: such an abort can only
                // come from a wait that ran out, after every slot was filled once)
                const uint32_t n_s = fills > static_cast<uint32_t>(s)
                                         ? (fills - static_cast<uint32_t>(s) + STAGES - 1) / STAGES
                                         : 0u;
                if (n_s) wait_bounded(bar(BAR_FULL + s), (n_s - 1) & 1, abort_flag, nullptr, true);
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer (leader CTA) ----------------
        // As in the single product (gemm.cu): the warp meets the gate at the slot's named barrier and
        // lane 0 issues; the loop is unrolled over the ring's slots so that each slot's descriptors,
        // scale columns and barriers are constants.  Experts without K steps are skipped by every
        // role but the epilogue.
        const uint32_t s0 = smem_u32(smem);
        uint64_t da[STAGES], db[STAGES];
        uint32_t tc[STAGES];
#pragma unroll
        for (int j = 0; j < STAGES; ++j) {
            da[j] = desc_sw128(s0 + j * STAGE_BYTES);
            db[j] = desc_sw128(s0 + j * STAGE_BYTES + A_BYTES);
            tc[j] = tmem_base + SF_COL + j * SF_COLS_PER_STAGE;
        }
        const uint32_t acc = tmem_base + ACC_COL;
        bool any = false;
        int left = 0;  // K steps of the tile that no issued block covers
        int t = cluster;
        for (; t < total && (left = sch.steps<BY_K>(t)) == 0;) t += clusters;
        int steps = left;
        bool live = t < total;
        while (live) {
#pragma unroll
            for (int j = 0; j < STAGES; ++j) {
                if (!live) break;
                named_sync(GATE_BAR0 + j, GATE_THREADS);
                const bool more = left > BK / MMA_K;
                const uint32_t add = left != steps ? 1u : 0u;  // not the tile's first block
                if (lane == 0) {
                    tc_fence_after();
                    // K step k: scales of A in columns tc + 4k, of B in tc + 16 + 8k
                    if (left >= BK / MMA_K) {
                        mma_nvf4_pair<false>(acc, da[j], db[j], tc[j], tc[j] + 16, add);
                        mma_nvf4_pair<false>(acc, da[j] + 2, db[j] + 2, tc[j] + 4, tc[j] + 24, 1u);
                        mma_nvf4_pair<false>(acc, da[j] + 4, db[j] + 4, tc[j] + 8, tc[j] + 32, 1u);
                        mma_nvf4_pair<false>(acc, da[j] + 6, db[j] + 6, tc[j] + 12, tc[j] + 40, 1u);
                    } else {
                        // 1..3 K steps; the rest of the block belongs to the next expert
                        for (int k = 0; k < left; ++k)
                            mma_nvf4_pair<false>(acc, da[j] + 2 * k, db[j] + 2 * k, tc[j] + 4 * k,
                                                 tc[j] + 16 + 8 * k, k != 0 ? 1u : add);
                    }
                    mma_commit_pair(bar(BAR_EMPTY + j));
                    if (!more) mma_commit_pair(bar(BAR_ACC_FULL));
                }
                __syncwarp();
                any = true;
                if (!more) {
                    for (t += clusters; t < total && (left = sch.steps<BY_K>(t)) == 0;) t += clusters;
                    steps = left;
                    live = t < total;
                } else {
                    left -= BK / MMA_K;
                }
            }
        }
        // every MMA this CTA pair issued completes before the tensor memory can be freed
        if (lane == 0 && any) {
            mma_commit_pair(bar(BAR_DRAIN));
            wait_bounded(bar(BAR_DRAIN), 0, abort_flag, nullptr, true);
        }
    } else if (warp == GATE_WARP && rank == 0) {
        // ---------------- the issuer's gate (leader CTA) ----------------
        // For each K block in the issuer's order: at a tile start, wait until both CTAs'
        // epilogues have drained the accumulator; wait until both CTAs' stagers have put the
        // slot's scales in tensor memory (which they do after the slot's TMA bytes landed);
        // then meet the issuer.  After an abort (or a timeout here) it stops waiting but keeps
        // meeting the issuer, K block for K block.
        // (every role that waits with a time limit starts its clock when the kernel ahead has ended)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        int stage = 0, it = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = cluster; t < total; t += clusters) {
            const int num_kb = (sch.steps<BY_K>(t) + BK / MMA_K - 1) / (BK / MMA_K);
            if (BY_K && num_kb == 0) continue;
            for (int kb = 0; kb < num_kb; ++kb) {
                if (lane == 0 && ok) {
                    // suspending waits (try_wait): a spinning gate takes issue slots from the
                    // stagers and epilogue warps of its scheduler (0.5 % slower, FP32 out)
                    if (kb == 0)
                        ok = wait_bounded(bar(BAR_ACC_EMPTY), (it & 1) ^ 1, abort_flag,
                                          p.dev_status);
                    if (ok) ok = wait_bounded(bar(BAR_SF + stage), phase, abort_flag, p.dev_status);
                }
                __syncwarp();
                named_sync(GATE_BAR0 + stage, GATE_THREADS);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            ++it;
        }
    } else if (warp >= FIRST_SF_WARP && warp < FIRST_SF_WARP + NUM_SF_WARPS) {
        // ---------------- scale stagers (both CTAs) ----------------
        // Tensor-memory layout the block-scaled MMA reads, in each CTA: row r's four E4M3
        // scales of one K step sit in lane r % 32 of every lane quarter, column r / 32.  Byte
        // 16 l of a 512-byte scale tile holds exactly those 4 columns for rows l, l + 32, l + 64,
        // l + 96, so lane l of each quarter's warp loads 16 bytes per tile and stores them.
        // Row groups beyond M or N and K tiles beyond K arrive zero-filled from the scale maps,
        // so padding rows (whose codes are zero-filled too) multiply to zero, never to NaN.
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int q = warp & 3;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = cluster; t < total && ok; t += clusters) {
            const int num_kb = (sch.steps<BY_K>(t) + BK / MMA_K - 1) / (BK / MMA_K);
            for (int kb = 0; kb < num_kb; ++kb) {
                bool ready = lane == 0 ? wait_bounded(bar(BAR_FULL + stage), phase, abort_flag,
                                                      p.dev_status)
                                       : false;
                ready = __shfl_sync(0xFFFFFFFFu, ready ? 1 : 0, 0) != 0;
                if (!ready) {
                    ok = false;
                    break;
                }
                __syncwarp();
                const uint8_t* sf = smem + stage * STAGE_BYTES + A_BYTES + B_BYTES;
                uint32_t ra[16], rb[32];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 v = *reinterpret_cast<const uint4*>(sf + k * SF_TILE + 16 * lane);
                    ra[4 * k] = v.x;
                    ra[4 * k + 1] = v.y;
                    ra[4 * k + 2] = v.z;
                    ra[4 * k + 3] = v.w;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 v = *reinterpret_cast<const uint4*>(
                            sf + SFA_BYTES + h * (SFB_BYTES / 2) + k * SF_TILE + 16 * lane);
                        const int c = 4 * (2 * k + h);
                        rb[c] = v.x;
                        rb[c + 1] = v.y;
                        rb[c + 2] = v.z;
                        rb[c + 3] = v.w;
                    }
                }
                const uint32_t taddr = tmem_base + SF_COL + stage * SF_COLS_PER_STAGE +
                                       (static_cast<uint32_t>(32 * q) << 16);
                tmem_st16(taddr, ra);       // A: columns 4k + j
                tmem_st32(taddr + 16, rb);  // B: columns 16 + 8k + 4h + j
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(bar(BAR_SF + stage), 0);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp >= FIRST_EPI_WARP && warp < FIRST_EPI_WARP + NUM_EPI_WARPS) {
        // ---------------- epilogue (both CTAs) ----------------
        const int q = warp & 3;                         // TMEM lane quarter this warp may access
        const int chunk = (warp - FIRST_EPI_WARP) >> 2; // accumulator columns [64 chunk, +64)
        const uint32_t stage_buf = smem_u32(staging + (warp - FIRST_EPI_WARP) * STAGING_BYTES);
        // NVFP4: undo both tensor scales; MXFP4 has none (its amax only flags bad data)
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the quantizer's amax
        const Alpha alpha = epilogue_alpha<false>(*p.amax_a, *p.amax_b);
        int it = 0;  // tiles with an accumulator so far
        constexpr uint32_t EPI_THREADS = 32 * NUM_EPI_WARPS;
        const bool waiter = warp == FIRST_EPI_WARP && lane == 0;
        for (int t = cluster; t < total; t += clusters) {
            const Tile c = sch.tile<BY_K>(t);
            uint32_t v[64];
            if (BY_K && c.steps == 0) {
                // an expert without tokens: its product is zero
#pragma unroll
                for (int j = 0; j < 64; ++j) v[j] = 0u;
            } else {
                // one thread spins on the accumulator barrier and releases the other epilogue
                // warps through a named barrier (a hardware barrier: nobody else polls)
                if (waiter) *epi_go = wait_spin(bar(BAR_ACC_FULL), it & 1, abort_flag, p.dev_status);
                named_sync(1, EPI_THREADS);
                if (!*epi_go) break;
                tc_fence_after();
                const uint32_t taddr = tmem_base + ACC_COL + (static_cast<uint32_t>(32 * q) << 16) +
                                       64 * chunk;
                tmem_ld32(taddr, v);  // row `lane` of the quarter, columns [64 chunk, +64)
                tmem_ld32(taddr + 32, v + 32);
                tmem_wait_ld();
                tc_fence_before();
                // this warp holds its slice: its arrival releases its part of the accumulator
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(bar(BAR_ACC_EMPTY), 0);
                ++it;
            }
            // first output row of this warp's slice: the CTA's half of the pair tile
            const int y = c.d_row + static_cast<int>(rank) * CTA_M + 32 * q;
            store_slice<BF16>(v, alpha, stage_buf, lane, &tmap_d, c.col + 64 * chunk, y, c.d_end, p.N,
                              nullptr, nullptr, 0, p.dev_status);
        }
        if (lane == 0) bulk_wait_all();
    }

    // Neither CTA frees its tensor memory or exits while the pair's MMAs or the peer's
    // arrivals may still reach it.
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

}  // namespace

cudaError_t launch_gemm_grouped(const GroupedGemmArgs& g, int sm_count, cudaStream_t s)
{
    // Once per device: the kernels' shared-memory limit and the number of resident CTA pairs.
    constexpr int kDevices = 64;
    static int max_pairs[kDevices] = {};
    static std::mutex configure_mutex;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices)
        return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(configure_mutex);
        if (max_pairs[dev] == 0) {
            const void* kernels[4] = {reinterpret_cast<const void*>(gemm_grouped_kernel<true, false>),
                                      reinterpret_cast<const void*>(gemm_grouped_kernel<false, false>),
                                      reinterpret_cast<const void*>(gemm_grouped_kernel<true, true>),
                                      reinterpret_cast<const void*>(gemm_grouped_kernel<false, true>)};
            int pairs = sm_count / 2;
            for (int i = 0; i < 4; ++i) {
                const int smem = i % 2 ? grouped_smem<false>() : grouped_smem<true>();
                const cudaError_t e = cudaFuncSetAttribute(
                    kernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
                if (e != cudaSuccess) return e;
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3(static_cast<unsigned>(sm_count & ~1), 1, 1);
                cfg.blockDim = dim3(THREADS, 1, 1);
                cfg.dynamicSmemBytes = static_cast<size_t>(smem);
                int n = 0;
                if (cudaOccupancyMaxActiveClusters(&n, kernels[i], &cfg) == cudaSuccess && n >= 1 &&
                    n < pairs)
                    pairs = n;
            }
            (void)cudaGetLastError();  // a failed occupancy query leaves no sticky error
            max_pairs[dev] = pairs > 0 ? pairs : 1;
        }
    }
    // operand shapes: by rows A is rows x K and B has every expert's slice; by K both run along the
    // expert-ordered rows
    const int64_t a_rows = g.by_k ? g.M : g.rows, a_k = g.by_k ? g.rows : g.K;
    const int64_t d_rows = g.by_k ? g.experts * g.M : g.rows;
    CUtensorMap ma, mb, msa, msb, md;
    if (!make_codes_map(&ma, g.a_codes, a_rows, a_k, CTA_M) ||
        !make_codes_map(&mb, g.b_codes, g.b_rows, g.b_cols, B_ROWS) ||
        !make_scales_map(&msa, g.a_scales, a_rows, a_k, 1) ||
        !make_scales_map(&msb, g.b_scales, g.b_rows, g.b_cols, 2) ||
        !make_output_map(&md, g.D, d_rows, g.N, g.ldd, g.out_bf16 != 0))
        return cudaErrorInvalidValue;
    GroupedParams p;
    p.offsets = g.offsets;
    p.experts = static_cast<int>(g.experts);
    p.rows = static_cast<int>(g.rows);
    p.amax_a = g.a_amax;
    p.amax_b = g.b_amax;
    p.M = static_cast<int>(g.M);
    p.N = static_cast<int>(g.N);
    p.K = static_cast<int>(g.K);
    p.b_row_step = static_cast<int>(g.b_row_step);
    p.b_k_step = static_cast<int>(g.b_k_step);
    p.dev_status = g.dev_status;
    // most tiles the routing can give: one partly filled row tile per 128 rows
    const int64_t tiles_n = (g.N + BN - 1) / BN;
    const int64_t tiles = g.by_k ? g.experts * ((g.M + PAIR_M - 1) / PAIR_M) * tiles_n
                                 : g.rows / 128 * tiles_n;
    const int grid = 2 * static_cast<int>(tiles < max_pairs[dev] ? tiles : max_pairs[dev]);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(g.out_bf16 ? grouped_smem<true>() : grouped_smem<false>());
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = g.after_quantizer ? 1 : 0;
    if (g.by_k && g.out_bf16)
        return cudaLaunchKernelEx(&cfg, gemm_grouped_kernel<true, true>, ma, mb, msa, msb, md, p);
    if (g.by_k)
        return cudaLaunchKernelEx(&cfg, gemm_grouped_kernel<false, true>, ma, mb, msa, msb, md, p);
    if (g.out_bf16)
        return cudaLaunchKernelEx(&cfg, gemm_grouped_kernel<true, false>, ma, mb, msa, msb, md, p);
    return cudaLaunchKernelEx(&cfg, gemm_grouped_kernel<false, false>, ma, mb, msa, msb, md, p);
}

}  // namespace nvfp4
