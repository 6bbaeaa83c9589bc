// Block-scaled NVFP4 GEMM on the sm_100a tcgen05 tensor cores: D = A . B^T.
//
// Method: "Pretraining Large Language Models with NVFP4" (gist.science summary), Resumen
// tecnico section 2, "Formato NVFP4": E2M1 operands with one E4M3 scale per 16 elements and
// an FP32 scale per tensor, multiplied natively by Blackwell tensor cores.
//
// Design: persistent CTA pairs (clusters of two CTAs on one TPC), one per two SMs, over
// 256 x 256 output tiles; each pair tile is one tcgen05.mma.cta_group::2 accumulation (M 256,
// N 256, K 64 per instruction) whose A rows and B rows are split between the two CTAs, so each
// SM reads 128 A rows and 128 B rows per K block: 38 KB per 256-wide K block where a single-CTA
// 128 x 256 tile needs 54 KB for the same work.  23 warps per CTA:
//   warp 0      TMA producer (both CTAs): per 256-wide K block, this CTA's A (128 x 128 B) and
//               B (128 x 128 B) code boxes with 128-byte swizzle, this CTA's 128 rows of A
//               scales (four 512-byte tiles of the MMA scale layout) and all 256 rows of B
//               scales (eight), each set one 3-D tensor copy over the tiles, into a
//               shared-memory ring of 5 stages.
//   warps 2-5   scale stagers, one per 32-lane quarter of tensor memory (both CTAs): move each
//               stage's scales shared -> registers -> tensor memory (tcgen05.st), then arrive on
//               the leader CTA's stage barrier.  (tcgen05.cp from the MMA thread would use the
//               tensor pipe: measured on B200, twelve 32x128b copies per K block lengthen the
//               block's four MMAs from 278 ns to 458 ns.)
//   warp 1      tensor-memory owner (both CTAs, allocated for the pair) and, in the leader CTA,
//               the MMA issuer (one thread): per K block, four kind::mxf4nvf4 block-scaled MMAs
//               (E4M3 scales, or UE8M0 for MXFP4 operands), then one commit that releases the
//               stage in both CTAs.
//   warp 22     the issuer's gate (leader CTA): waits until both CTAs' stagers have arrived
//               (and, at a tile start, both epilogues have drained the accumulator), then
//               meets the issuer at the slot's named barrier.  The issuer polls no mbarrier:
//               measured on B200, a barrier poll in the issuing thread between two K blocks
//               idles the tensor pipe 80-200 ns per K block (pair M256 N256 K64 MMAs:
//               278 ns per four behind a named barrier, 480 ns with a commit and a poll).
//   warps 6-21  epilogue (both CTAs): each warp drains one 32-lane quarter x 64 columns of its
//               CTA's 128 x 256 half of the accumulator (tcgen05.ld), releases it to the leader,
//               scales by 1 / (S_enc,A S_enc,B) and writes it while the next tile computes,
//               through a 2 KB per-warp staging buffer with TMA bulk tensor stores (2 rounds for
//               bf16, 4 for FP32; clipped at the matrix edge).  With the fused amax, the bf16
//               epilogue also reduces max |D| and, by 16-lane shuffles across rows,
//               max |RHT(D)| for the next quantization of D.
// No load is multicast: every CTA loads its own operands from this GPU's memory.
// Every wait on an mbarrier is bounded in time; on expiry the kernel records
// NVFP4_DEVSTAT_TIMEOUT, drains its in-flight copies and MMAs (again with a limit), meets its
// peer at a cluster barrier, frees its tensor memory and returns.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "gemm_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
using namespace gemm;
namespace {

struct Params {
    uint32_t* amax_out;  // fused maxima (bf16 output only): [max |D|, max |RHT(D)|] as FP32 bits
    uint32_t sign_mask;  // RHT signs for amax_out[1]
    const float* amax_a;
    const float* amax_b;
    void* D;
    int64_t ldd;
    int M, N, K;
    int out_bf16;
    int group_m;         // row tiles per raster group (tile_coords)
    int* dev_status;
};

// Pair-tile order: groups of G row tiles, each group's row tiles innermost and its column tiles
// outer, so that the pairs working at the same time share A and B tiles in L2 (G per shape,
// set by the host).
__device__ __forceinline__ void tile_coords(int t, int tiles_m, int tiles_n, int G, int& tm,
                                            int& tn)
{
    const int group = t / (G * tiles_n);
    const int first = group * G;
    const int gsz = min(G, tiles_m - first);
    const int local = t - group * G * tiles_n;
    tm = first + local % gsz;
    tn = local / gsz;
}

template <bool BF16, bool MX, bool AMAX = false>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    gemm_nvf4_kernel(const __grid_constant__ CUtensorMap tmap_a,
                     const __grid_constant__ CUtensorMap tmap_b,
                     const __grid_constant__ CUtensorMap tmap_sfa,
                     const __grid_constant__ CUtensorMap tmap_sfb,
                     const __grid_constant__ CUtensorMap tmap_d, const Params p)
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
    const int tiles_m = (p.M + PAIR_M - 1) / PAIR_M, tiles_n = (p.N + BN - 1) / BN;
    const int total = tiles_m * tiles_n;
    const int num_kb = (p.K + BK - 1) / BK;
    const int k_steps_total = p.K / MMA_K;

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
        for (int t = cluster; t < total && ok; t += clusters) {
            int tm, tn;
            tile_coords(t, tiles_m, tiles_n, p.group_m, tm, tn);
            const int ga = tm * 2 + static_cast<int>(rank);  // this CTA's 128-row group of A
            for (int kb = 0; kb < num_kb; ++kb) {
                if (!wait_bounded(bar(BAR_EMPTY + stage), phase ^ 1, abort_flag, p.dev_status)) {
                    ok = false;
                    break;
                }
                if (kBoundsCheck &&
                    !(tma_box_start_ok(kb * (BK / 2), ga * CTA_M, 1, p.dev_status) &&
                      kb * (BK / 2) < p.K / 2 &&
                      tma_box_start_ok(kb * (BK / 2), tn * BN + static_cast<int>(rank) * B_ROWS, 1,
                                       p.dev_status))) {
                    // no copy for this stage: the roles waiting for it stop at the abort flag
                    record_bounds_error(p.dev_status);
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                const uint32_t full = bar(BAR_FULL + stage);
                const uint32_t st = smem_u32(smem + stage * STAGE_BYTES);
                mbar_expect_tx(full, STAGE_BYTES);
                tma_load_2d(st, &tmap_a, kb * (BK / 2), ga * CTA_M, full);
                tma_load_2d(st + A_BYTES, &tmap_b, kb * (BK / 2),
                            tn * BN + static_cast<int>(rank) * B_ROWS, full);
                tma_load_3d(st + A_BYTES + B_BYTES, &tmap_sfa, 0, kb * (BK / MMA_K), ga, full);
                tma_load_3d(st + A_BYTES + B_BYTES + SFA_BYTES, &tmap_sfb, 0, kb * (BK / MMA_K),
                            2 * tn, full);
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
                const uint32_t n_s = fills > static_cast<uint32_t>(s)
                                         ? (fills - static_cast<uint32_t>(s) + STAGES - 1) / STAGES
                                         : 0u;
                if (n_s) wait_bounded(bar(BAR_FULL + s), (n_s - 1) & 1, abort_flag, nullptr, true);
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer (leader CTA) ----------------
        // The MMA instructions issue at about the rate the tensor pipe executes them, so every
        // instruction this thread runs between two K blocks leaves the pipe idle.  The whole
        // warp meets the gate warp at the slot's named barrier (the gate has seen the slot's
        // operands and scales land); lane 0 then issues.  The loop is unrolled over the ring's
        // slots, which it visits in order across tiles as the producer, the stagers and the
        // gate do, so each slot's descriptors, scale columns, barriers and named barrier are
        // constants.  Descriptors address shared memory through a 14-bit start-address field
        // (address / 16): a slot is STAGE_BYTES / 16 further on, a K step 32 bytes (2 units).
        // After an abort the gate keeps meeting the issuer, which then runs its schedule on
        // stale operands (in bounds, results discarded) rather than leave a barrier unmet.
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
        const bool k_full = (k_steps_total % (BK / MMA_K)) == 0;  // every stage has 4 K steps
        bool any = false;
        int kb = 0, t = cluster;
        bool live = t < total;
        while (live) {
#pragma unroll
            for (int j = 0; j < STAGES; ++j) {
                if (!live) break;
                named_sync(GATE_BAR0 + j, GATE_THREADS);
                const bool more = kb + 1 < num_kb;
                if (lane == 0) {
                    tc_fence_after();
                    // K step k: scales of A in columns tc + 4k, of B in tc + 16 + 8k
                    if (k_full || more) {
                        mma_nvf4_pair<MX>(acc, da[j], db[j], tc[j], tc[j] + 16, kb != 0 ? 1u : 0u);
                        mma_nvf4_pair<MX>(acc, da[j] + 2, db[j] + 2, tc[j] + 4, tc[j] + 24, 1u);
                        mma_nvf4_pair<MX>(acc, da[j] + 4, db[j] + 4, tc[j] + 8, tc[j] + 32, 1u);
                        mma_nvf4_pair<MX>(acc, da[j] + 6, db[j] + 6, tc[j] + 12, tc[j] + 40, 1u);
                    } else {
                        const int nk = k_steps_total - kb * (BK / MMA_K);  // 1..3 K steps left
                        for (int k = 0; k < nk; ++k)
                            mma_nvf4_pair<MX>(acc, da[j] + 2 * k, db[j] + 2 * k, tc[j] + 4 * k,
                                              tc[j] + 16 + 8 * k, (kb | k) != 0 ? 1u : 0u);
                    }
                    mma_commit_pair(bar(BAR_EMPTY + j));
                    if (!more) mma_commit_pair(bar(BAR_ACC_FULL));
                }
                __syncwarp();
                any = true;
                if (!more) {
                    kb = 0;
                    t += clusters;
                    live = t < total;
                } else {
                    ++kb;
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
        int stage = 0, it = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = cluster; t < total; t += clusters, ++it) {
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
        }
    } else if (warp >= FIRST_SF_WARP && warp < FIRST_SF_WARP + NUM_SF_WARPS) {
        // ---------------- scale stagers (both CTAs) ----------------
        // Tensor-memory layout the block-scaled MMA reads, in each CTA: row r's four E4M3
        // scales of one K step sit in lane r % 32 of every lane quarter, column r / 32.  Byte
        // 16 l of a 512-byte scale tile holds exactly those 4 columns for rows l, l + 32, l + 64,
        // l + 96, so lane l of each quarter's warp loads 16 bytes per tile and stores them.
        // Row groups beyond M or N and K tiles beyond K arrive zero-filled from the scale maps,
        // so padding rows (whose codes are zero-filled too) multiply to zero, never to NaN.
        const int q = warp & 3;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = cluster; t < total && ok; t += clusters) {
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
        const Alpha alpha = epilogue_alpha<MX>(*p.amax_a, *p.amax_b);
        int it = 0;
        uint32_t m_plain = 0, m_rht = 0;  // fused maxima (AMAX)
        const uint32_t flip = ((p.sign_mask >> (lane & 15)) & 1u) ? 0x80000000u : 0u;
        constexpr uint32_t EPI_THREADS = 32 * NUM_EPI_WARPS;
        const bool waiter = warp == FIRST_EPI_WARP && lane == 0;
        for (int t = cluster; t < total; t += clusters, ++it) {
            // one thread spins on the accumulator barrier and releases the other epilogue
            // warps through a named barrier (a hardware barrier: nobody else polls)
            if (waiter) *epi_go = wait_spin(bar(BAR_ACC_FULL), it & 1, abort_flag, p.dev_status);
            named_sync(1, EPI_THREADS);
            if (!*epi_go) break;
            tc_fence_after();
            uint32_t v[64];
            const uint32_t taddr = tmem_base + ACC_COL + (static_cast<uint32_t>(32 * q) << 16) +
                                   64 * chunk;
            tmem_ld32(taddr, v);  // row `lane` of the quarter, columns [64 chunk, +64)
            tmem_ld32(taddr + 32, v + 32);
            tmem_wait_ld();
            tc_fence_before();
            // this warp holds its slice: its arrival releases its part of the accumulator
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(bar(BAR_ACC_EMPTY), 0);

            int tm, tn;
            tile_coords(t, tiles_m, tiles_n, p.group_m, tm, tn);
            // first output row of this warp's slice: the CTA's half of the pair tile
            const int y = tm * PAIR_M + static_cast<int>(rank) * CTA_M + 32 * q;
            const int n0 = tn * BN + 64 * chunk;  // first output column
            store_slice<BF16, AMAX>(v, alpha, stage_buf, lane, &tmap_d, n0, y, p.M, p.N, &m_plain,
                                    &m_rht, flip, p.dev_status);
        }
        if (lane == 0) bulk_wait_all();
        if (AMAX) {
            m_plain = __reduce_max_sync(0xFFFFFFFFu, max(m_plain & 0xFFFFu, m_plain >> 16) << 16);
            m_rht = __reduce_max_sync(0xFFFFFFFFu, m_rht);
            if (lane == 0) {
                atomicMax(p.amax_out, m_plain);
                // x1/4 once, on the maximum (rounding is monotone)
                atomicMax(p.amax_out + 1, __float_as_uint(__fmul_rn(__uint_as_float(m_rht), 0.25f)));
            }
        }
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

// Self-test of the bounded waits: one thread waits on an mbarrier that nothing arrives at, with
// the GEMM's own wait routine and a limit of `limit_ns`; the wait gives up, records
// NVFP4_DEVSTAT_TIMEOUT and the kernel returns.
__global__ void wait_selftest_kernel(int* dev_status, unsigned long long limit_ns)
{
    __shared__ __align__(8) uint64_t never;
    __shared__ int abort_flag;
    if (threadIdx.x != 0) return;
    mbar_init(smem_u32(&never), 1);
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    wait_bounded(smem_u32(&never), 0, &abort_flag, dev_status, false, limit_ns);
}

}  // namespace

cudaError_t launch_wait_selftest(int* dev_status, unsigned long long limit_ns, cudaStream_t s)
{
    wait_selftest_kernel<<<1, 32, 0, s>>>(dev_status, limit_ns);
    return cudaGetLastError();
}

cudaError_t launch_gemm(const GemmArgs& g, int sm_count, cudaStream_t s)
{
    // Once per device: the kernels' shared-memory limit is raised and the number of CTA pairs
    // that can be resident at once is looked up (the persistent grid is one wave of pairs).
    constexpr int kDevices = 64;
    static int max_pairs[kDevices] = {};
    static std::mutex configure_mutex;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices)
        return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(configure_mutex);
        if (max_pairs[dev] == 0) {
            cudaError_t e = cudaSuccess;
            const void* kernels[5] = {
                reinterpret_cast<const void*>(gemm_nvf4_kernel<true, false>),
                reinterpret_cast<const void*>(gemm_nvf4_kernel<false, false>),
                reinterpret_cast<const void*>(gemm_nvf4_kernel<true, true>),
                reinterpret_cast<const void*>(gemm_nvf4_kernel<false, true>),
                reinterpret_cast<const void*>(gemm_nvf4_kernel<true, false, true>)};
            const int smem[5] = {Pipe<true>::SMEM_BYTES, Pipe<false>::SMEM_BYTES,
                                 Pipe<true>::SMEM_BYTES, Pipe<false>::SMEM_BYTES,
                                 Pipe<true>::SMEM_BYTES};
            for (int i = 0; i < 5 && e == cudaSuccess; ++i)
                e = cudaFuncSetAttribute(kernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem[i]);
            if (e != cudaSuccess) return e;
            int pairs = 0;
            for (int i = 0; i < 5; ++i) {
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3(static_cast<unsigned>(sm_count & ~1), 1, 1);
                cfg.blockDim = dim3(THREADS, 1, 1);
                cfg.dynamicSmemBytes = static_cast<size_t>(smem[i]);
                int n = 0;
                if (cudaOccupancyMaxActiveClusters(&n, kernels[i], &cfg) != cudaSuccess || n < 1)
                    n = sm_count / 2;
                pairs = (i == 0 || n < pairs) ? n : pairs;
            }
            (void)cudaGetLastError();  // a failed occupancy query leaves no sticky error
            max_pairs[dev] = pairs > 0 ? pairs : 1;
        }
    }
    CUtensorMap ma, mb, msa, msb, md;
    if (!make_codes_map(&ma, g.a_codes, g.M, g.K, CTA_M) ||
        !make_codes_map(&mb, g.b_codes, g.N, g.K, B_ROWS) ||
        !make_scales_map(&msa, g.a_scales, g.M, g.K, 1) ||
        !make_scales_map(&msb, g.b_scales, g.N, g.K, 2) ||
        !make_output_map(&md, g.D, g.M, g.N, g.ldd, g.out_bf16 != 0))
        return cudaErrorInvalidValue;
    Params p;
    p.amax_a = g.a_amax;
    p.amax_b = g.b_amax;
    p.D = g.D;
    p.ldd = g.ldd;
    p.M = static_cast<int>(g.M);
    p.N = static_cast<int>(g.N);
    p.K = static_cast<int>(g.K);
    p.out_bf16 = g.out_bf16;
    // Raster: the operand with fewer rows stays resident in L2 while the other streams through
    // about once.  A (M rows) no larger than B: every row tile of a column tile in turn (A
    // resident, each B stripe read once); otherwise groups of 4 row tiles across all column
    // tiles (B resident, each A stripe read once).  B200: 8192 x 20480 x 5120 0.358 ms with
    // all 32 row tiles per group against 0.375 with 8; 20480 x 5120 x 8192 0.389 with 4
    // against 0.398 with 8.
    {
        const int tiles_m = static_cast<int>((g.M + PAIR_M - 1) / PAIR_M);
        p.group_m = g.M <= g.N ? tiles_m : (tiles_m < 4 ? tiles_m : 4);
    }
    p.dev_status = g.dev_status;
    p.amax_out = g.amax_out;
    p.sign_mask = g.sign_mask;
    const int64_t tiles = ((g.M + PAIR_M - 1) / PAIR_M) * ((g.N + BN - 1) / BN);
    const int pairs = static_cast<int>(tiles < max_pairs[dev] ? tiles : max_pairs[dev]);
    const int grid = 2 * pairs;  // clusters of two CTAs (__cluster_dims__)
    if (g.amax_out) {
        // fused maxima of the bf16 output for the next quantizer (the API allows it only there)
        if (!g.out_bf16 || g.mx) return cudaErrorInvalidValue;
        const cudaError_t e = cudaMemsetAsync(g.amax_out, 0, 2 * sizeof(uint32_t), s);
        if (e != cudaSuccess) return e;
        gemm_nvf4_kernel<true, false, true>
            <<<grid, THREADS, Pipe<true>::SMEM_BYTES, s>>>(ma, mb, msa, msb, md, p);
    } else if (g.out_bf16 && !g.mx)
        gemm_nvf4_kernel<true, false><<<grid, THREADS, Pipe<true>::SMEM_BYTES, s>>>(ma, mb, msa, msb, md, p);
    else if (!g.mx)
        gemm_nvf4_kernel<false, false><<<grid, THREADS, Pipe<false>::SMEM_BYTES, s>>>(ma, mb, msa, msb, md, p);
    else if (g.out_bf16)
        gemm_nvf4_kernel<true, true><<<grid, THREADS, Pipe<true>::SMEM_BYTES, s>>>(ma, mb, msa, msb, md, p);
    else
        gemm_nvf4_kernel<false, true><<<grid, THREADS, Pipe<false>::SMEM_BYTES, s>>>(ma, mb, msa, msb, md, p);
    return cudaGetLastError();
}

}  // namespace nvfp4
