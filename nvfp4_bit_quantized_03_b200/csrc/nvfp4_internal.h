// Internal interfaces between the C ABI (api.cu) and the kernels (quantize.cu, gemm.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#ifdef __CUDACC__
#include "bounds_check.cuh"
#endif

namespace nvfp4 {

// Upper bound on the CTAs of the amax pass, i.e. on the partial maxima in the workspace.
constexpr int kMaxPartials = 2048;

// Where a quantize kernel gets the tensor amax from: the partial maxima written by the
// amax pass (FP32 bit patterns), or a caller-given FP32 value.
// The ten Philox-4x32-10 round keys of a seed: round i uses (seed low + i * 0x9E3779B9,
// seed high + i * 0xBB67AE85).
struct PhiloxKeys {
    uint32_t k0[10], k1[10];
};

inline PhiloxKeys philox_round_keys(uint64_t seed)
{
    PhiloxKeys k;
    uint32_t a = static_cast<uint32_t>(seed), b = static_cast<uint32_t>(seed >> 32);
    for (int i = 0; i < 10; ++i) {
        k.k0[i] = a;
        k.k1[i] = b;
        a += 0x9E3779B9u;
        b += 0xBB67AE85u;
    }
    return k;
}

struct QuantSource {
    const uint32_t* partials;
    int n_partials;
    const float* amax_given;  // non-null: use *amax_given, ignore the partials
};

// Which row of x a row of an expert-ordered matrix holds.  Maps come from device memory that the
// caller wrote, so every index is checked against its range before it is used.
struct RowMap {
    const int32_t* row_token;  // [rows] token of each row, negative: a row of zeros
    const int32_t* pair_row;   // [tokens * k] row of each pair, negative: none
    const int32_t* used;       // rows in use (the last of the region offsets)
    int64_t tokens, k;
    int64_t rows;              // rows of the expert-ordered matrix
    int64_t x_rows;            // rows of x: tokens when gathering, else the matrix's rows
    bool gather;               // x has a row per token; otherwise it is in expert order itself
    int* dev_status;           // of the debug build's checks

#ifdef __CUDACC__
    __device__ __forceinline__ int64_t token_of(int64_t r) const
    {
        return ld_checked(row_token + r, row_token, 4 * rows, dev_status);
    }
    __device__ __forceinline__ int64_t used_rows(int64_t rows) const
    {
        const int64_t n = *used;
        return n < 0 ? 0 : (n < rows ? n : rows) & ~static_cast<int64_t>(127);
    }
    // row of x behind row r, or -1
    __device__ __forceinline__ int64_t source(int64_t r) const
    {
        const int64_t t = token_of(r);
        if (t < 0 || t >= tokens) return -1;
        return gather ? t : r;
    }
    // row of the pair (t, j), or -1
    __device__ __forceinline__ int64_t pair_target(int64_t t, int64_t j, int64_t rows) const
    {
        const int64_t r = ld_checked(pair_row + t * k + j, pair_row, 4 * tokens * k, dev_status);
        return r < rows ? r : -1;
    }
#endif
};

struct TileArgs {
    const uint16_t* x;
    int64_t rows, cols, ld;
    QuantSource src;      // amax of the row-wise output (of every output outside the dual mode)
    QuantSource src_col;  // dual mode (row-wise + RHT column-wise): amax of the column output
    uint8_t* row_codes;
    uint8_t* row_scales;
    float* row_amax;
    uint8_t* col_codes;
    uint8_t* col_scales;
    float* col_amax;
    uint32_t sign_mask;
    PhiloxKeys keys;      // round keys of the SR seed
    uint64_t offset;
    uint64_t offset_col;  // dual mode: SR stream of the column output
    int* dev_status;
    RowMap map;           // grouped passes only
};

int amax_grid(int64_t rows, int64_t cols, bool rht, int sm_count);
cudaError_t launch_amax(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, bool rht,
                        uint32_t sign_mask, uint32_t* partials, int grid, int* dev_status,
                        cudaStream_t s);
// One pass for both maxima of the dual mode: amax of RHT(x) along the rows into
// `partials_rht` and amax of x into `partials_plain` (grid entries each).
cudaError_t launch_amax_dual(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld,
                             uint32_t sign_mask, uint32_t* partials_rht,
                             uint32_t* partials_plain, int grid, int* dev_status,
                             cudaStream_t s);
cudaError_t launch_quant_rowwise(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld,
                                 const QuantSource& src, float* amax_out0, float* amax_out1,
                                 uint8_t* codes, uint8_t* scales, bool sr, uint64_t seed,
                                 uint64_t offset, int* dev_status, int sm_count, cudaStream_t s);
cudaError_t launch_quant_tile(const TileArgs& a, bool row, bool col, bool block2d, bool rht,
                              bool sr, bool mx, int sm_count, cudaStream_t s);
// The same passes over an expert-ordered matrix.  amax: plain (`partials`), RHT (`partials`), or
// both (`partials_plain` not null).
int amax_grouped_grid(int64_t rows, int64_t cols, bool rht, const RowMap& map, int sm_count);
// Whether the gathered row-wise RTN pass computes the amax itself (n_partials 0, no amax pass).
bool grouped_amax_is_small(int64_t cols, const RowMap& map);
cudaError_t launch_amax_grouped(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, bool rht,
                                uint32_t sign_mask, uint32_t* partials, uint32_t* partials_plain,
                                int grid, const RowMap& map, int* dev_status, cudaStream_t s);
cudaError_t launch_quant_grouped_rows(const TileArgs& a, bool sr, int sm_count, cudaStream_t s);
cudaError_t launch_quant_grouped_tile(const TileArgs& a, bool row, bool sr, int sm_count,
                                      cudaStream_t s);
// Debug build only: one checked store just past a buffer's declared end (refused, recorded as
// NVFP4_DEVSTAT_BOUNDS); cudaErrorNotSupported in the normal build.
cudaError_t launch_bounds_selftest(int* dev_status, cudaStream_t s);

struct GemmArgs {
    const uint8_t* a_codes;
    const uint8_t* a_scales;
    const float* a_amax;
    const uint8_t* b_codes;
    const uint8_t* b_scales;
    const float* b_amax;
    int64_t M, N, K;
    void* D;
    int64_t ldd;
    int out_bf16;
    int* dev_status;
    bool mx;  // MXFP4 operands: E8M0 scales (each 32-block's byte in both 16-slots), no tensor scale
    uint32_t* amax_out;  // non-null: fused [max |D|, max |RHT(D)|] (FP32 bits) of a bf16 D
    uint32_t sign_mask;  // RHT signs for amax_out[1]
};

cudaError_t launch_gemm(const GemmArgs& g, int sm_count, cudaStream_t s);

// Experts of a mixture layer: the grouped products keep 4 bytes of schedule per expert in the
// shared memory that their pipeline leaves.
constexpr int kMaxExperts = 512;

// Products over the experts (gemm_grouped.cu).  By rows: A is rows x K in expert order, B holds
// expert e's N x K matrix from row e * b_row_step and column e * b_k_step of a b_rows x b_cols
// operand, D is rows x N.  By K: A is M x rows and B is N x rows (b_rows = N, b_cols = rows), D is
// (experts * M) x N.
struct GroupedGemmArgs {
    bool by_k;
    const uint8_t* a_codes;
    const uint8_t* a_scales;
    const float* a_amax;
    const uint8_t* b_codes;
    const uint8_t* b_scales;
    const float* b_amax;
    int64_t b_rows, b_cols, b_row_step, b_k_step;
    const int32_t* offsets;
    int64_t experts, rows;
    int64_t M, N, K;
    void* D;
    int64_t ldd;
    int out_bf16;
    int* dev_status;
    // The kernel ahead on the stream is the quantizer of A (and B by K), and what that waited for is
    // after everything else this product reads: the product may be launched before it ends.
    bool after_quantizer;
};

// Routing (route.cu).  The plan's first pass counts each kPlanPairs pairs apart; it needs no
// workspace when there are no more.
constexpr int kPlanPairs = 1024;
// From so many chunks on a pass between adds their counts up, instead of every chunk those of all
// (B200, 256 experts, with against without: 16 chunks 10.1 / 11.3 us, 128 11.4 / 15.8, 1024 22 / 140, 4096
// 73 / 1825; 64 experts, 64 chunks 10.0 / 10.1).
constexpr int kPlanScan = 16;
cudaError_t launch_route(const void* logits, bool bf16, int64_t T, int64_t E, int64_t ld,
                         const float* bias, bool sigmoid, bool renorm, int groups, int top_groups,
                         int k, float scale, int32_t* experts, float* weights, int* dev_status,
                         cudaStream_t s);
cudaError_t launch_route_backward(const void* logits, bool bf16, int64_t T, int64_t E, int64_t ld,
                                  const int32_t* experts, const float* dweights, bool sigmoid,
                                  bool renorm, int k, float scale, void* dlogits, int64_t ldd,
                                  int* dev_status, cudaStream_t s);
cudaError_t launch_plan(const int32_t* experts, int64_t pairs, int k, int E, int64_t rows,
                        int32_t* offsets, int32_t* pair_row, int32_t* row_token, int32_t* counts,
                        int* dev_status, cudaStream_t s);

// Expert rows to tokens and back (combine.cu).
struct CombineArgs {
    RowMap map;
    int64_t rows, cols;
    const uint16_t* y;
    int64_t ldy;
    const float* weights;
    void* out;            // combine: tokens x cols
    const void* dout;     // backward: tokens x cols
    int64_t ldo;          // row stride of out or dout
    uint16_t* dy;
    int64_t lddy;
    float* dweights;
    int* dev_status;
};
cudaError_t launch_combine(const CombineArgs& a, bool f32, int sm_count, cudaStream_t s);
cudaError_t launch_combine_backward(const CombineArgs& a, bool f32, int sm_count, cudaStream_t s);

// Norms and rotation of queries and keys (qk_norm.cu): index 0 the queries, 1 the keys.
constexpr int kMaxHeadDim = 512;     // a head's units of 16 values fill at most one warp
constexpr int kMaxHeadCtas = 592;    // CTAs of the gradient (4 per SM), i.e. rows of its partial sums
struct HeadsView {
    void* data;
    int64_t heads, token_stride, head_stride;  // strides in elements
};
struct HeadsArgs {
    HeadsView x[2];       // heads before the norm
    HeadsView z[2];       // after the rotation (backward: its gradients)
    HeadsView dx[2];      // backward: gradients of x
    const float* weight[2];
    float* dweight[2];
    float* partials;      // backward: a row of D sums per CTA
    const int32_t* positions;
    const float* table;   // table_rows x rotary: cosines, then sines
    int64_t tokens, table_rows;
    int D, rotary;
    float eps, inv_D;
    int lanes;            // lanes per head (set by the launch, as below)
    int slices;           // items a token's heads are split into
    int q_ctas;           // backward: the CTAs of the queries
    int* dev_status;
};
cudaError_t launch_qk_norm_rope(HeadsArgs a, bool in_f32, bool out_f32, bool interleaved, int sm_count,
                                cudaStream_t s);
int qk_backward_ctas(int64_t tokens, int64_t heads_q, int64_t heads_k, int64_t D);
cudaError_t launch_qk_norm_rope_backward(HeadsArgs a, bool x_f32, bool z_f32, bool dx_f32, bool interleaved,
                                         cudaStream_t s);

// Newton-Schulz orthogonalisation (orthogonalize.cu).
constexpr int kMaxOrthogonalizeSteps = 32;
struct OrthogonalizeArgs {
    const void* g;            // batch matrices rows x cols
    bool f32;                 // FP32, otherwise bf16
    int64_t batch, rows, cols, ldg, g_stride;
    int steps;
    const float* coefficients;  // host: steps x (a, b, c)
    double eps;
    void* out;                // bf16, as g
    int64_t ldo, out_stride;
    void* workspace;
    int* dev_status;
};
size_t orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols);
cudaError_t orthogonalize_ways(int64_t batch, int64_t rows, int64_t cols, int sm_count, int* ways);
cudaError_t launch_orthogonalize(const OrthogonalizeArgs& g, int sm_count, cudaStream_t s);

cudaError_t launch_gemm_grouped(const GroupedGemmArgs& g, int sm_count, cudaStream_t s);
// A kernel whose only thread waits, with the GEMM's bounded-wait routine, on an mbarrier that
// nothing completes; it records NVFP4_DEVSTAT_TIMEOUT after limit_ns and returns.
cudaError_t launch_wait_selftest(int* dev_status, unsigned long long limit_ns, cudaStream_t s);

}  // namespace nvfp4
