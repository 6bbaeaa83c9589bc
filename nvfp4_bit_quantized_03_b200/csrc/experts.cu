// C entry points of the mixture-of-experts operators (include/nvfp4.h): argument checks, workspace
// carving and dispatch to route.cu, quantize.cu, gemm_grouped.cu and combine.cu.  As everywhere in
// the library: no allocation, no synchronization, and nothing queued when an argument is invalid.
#include <cuda_runtime.h>

#include <cstdint>

#include "api_common.h"

using namespace nvfp4;

namespace {

constexpr int64_t kRegion = 128;                  // expert regions are multiples of this many rows
constexpr int64_t kMaxRows = kRegion * 0xFFFF;    // the grouped schedule keeps 16-bit region counts
constexpr int64_t kMaxPerToken = 32;              // a token's experts fill at most one warp

bool routing_sizes_ok(int64_t T, int64_t k, int64_t E)
{
    return T >= 1 && T < kMaxDim && E >= 1 && E <= kMaxExperts && k >= 1 && k <= kMaxPerToken &&
           T * k < kMaxDim;
}

nvfp4_status check_plan(const nvfp4_expert_plan* p)
{
    if (!p || !p->offsets || !p->pair_row || !p->row_token) return NVFP4_ERR_NULL;
    const int64_t need = nvfp4_expert_rows(p->tokens, p->k, p->experts);
    if (need == 0 || p->rows < need || p->rows % kRegion || p->rows > kMaxRows)
        return NVFP4_ERR_SHAPE;
    if (!aligned4(p->offsets) || !aligned4(p->pair_row) || !aligned4(p->row_token))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

RowMap row_map(const nvfp4_expert_plan& p, bool gather, int* dev_status)
{
    RowMap m;
    m.row_token = p.row_token;
    m.pair_row = p.pair_row;
    m.used = p.offsets + p.experts;
    m.tokens = p.tokens;
    m.k = p.k;
    m.rows = p.rows;
    m.x_rows = gather ? p.tokens : p.rows;
    m.gather = gather;
    m.dev_status = dev_status;
    return m;
}

nvfp4_status check_logits(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld,
                          int score, int k)
{
    if (!logits) return NVFP4_ERR_NULL;
    if (dtype != NVFP4_OUT_F32 && dtype != NVFP4_OUT_BF16) return NVFP4_ERR_ARG;
    if (score != NVFP4_SCORE_SOFTMAX && score != NVFP4_SCORE_SIGMOID) return NVFP4_ERR_ARG;
    if (!routing_sizes_ok(T, k, E) || k > E || ld < E) return NVFP4_ERR_SHAPE;
    const uintptr_t mask = dtype == NVFP4_OUT_F32 ? 3u : 1u;
    if (reinterpret_cast<uintptr_t>(logits) & mask) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

nvfp4_status check_rows_matrix(const void* x, int64_t cols, int64_t ld, int64_t per16)
{
    if (!x) return NVFP4_ERR_NULL;
    if (cols < 8 || cols >= kMaxDim || cols % 8 || ld < cols) return NVFP4_ERR_SHAPE;
    if (ld % per16 || !aligned16(x)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

nvfp4_status check_gemm_output(const void* D, int d_dtype, int64_t N, int64_t ldd)
{
    if (!D) return NVFP4_ERR_NULL;
    if (d_dtype != NVFP4_OUT_F32 && d_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_ARG;
    if (N < 16 || N % 16 || N >= kMaxDim || ldd < N) return NVFP4_ERR_SHAPE;
    if (!aligned16(D) || (ldd * (d_dtype == NVFP4_OUT_F32 ? 4 : 2)) % 16) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

void set_operands(GroupedGemmArgs& g, const nvfp4_operand& A, const nvfp4_operand& B)
{
    g.a_codes = static_cast<const uint8_t*>(A.codes);
    g.a_scales = static_cast<const uint8_t*>(A.scales);
    g.a_amax = A.amax;
    g.b_codes = static_cast<const uint8_t*>(B.codes);
    g.b_scales = static_cast<const uint8_t*>(B.scales);
    g.b_amax = B.amax;
    g.b_rows = B.rows;
    g.b_cols = B.cols;
}

}  // namespace

extern "C" {

int64_t nvfp4_expert_rows(int64_t T, int64_t k, int64_t E)
{
    if (!routing_sizes_ok(T, k, E)) return 0;
    // most rows that P pairs in at most n regions need: P + 127 n, in whole regions
    const int64_t pairs = T * k, n = pairs < E ? pairs : E;
    const int64_t rows = (pairs + n * (kRegion - 1)) / kRegion * kRegion;
    return rows <= kMaxRows ? rows : 0;
}

size_t nvfp4_expert_plan_workspace_bytes(int64_t T, int64_t k, int64_t E)
{
    if (!routing_sizes_ok(T, k, E)) return 0;
    const int64_t chunks = (T * k + kPlanPairs - 1) / kPlanPairs;
    return chunks > 1 ? sizeof(int32_t) * static_cast<size_t>((chunks + 1) * E) : 0;
}

nvfp4_status nvfp4_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld,
                         const float* bias, int score, int groups, int top_groups, int k,
                         int renormalize, float scale, int32_t* experts, float* weights,
                         int* dev_status, void* stream)
{
    nvfp4_status st = check_logits(logits, dtype, T, E, ld, score, k);
    if (st != NVFP4_OK) return st;
    if (!experts || !weights) return NVFP4_ERR_NULL;
    if (groups < 1 || groups > 32 || E % groups || top_groups < 1 || top_groups > groups ||
        k > E / groups * top_groups)
        return NVFP4_ERR_SHAPE;
    if (!aligned4(bias) || !aligned4(experts) || !aligned4(weights)) return NVFP4_ERR_ALIGN;
    int sms = 0;
    if ((st = current_device(&sms)) != NVFP4_OK) return st;
    return from_cuda(launch_route(logits, dtype == NVFP4_OUT_BF16, T, E, ld, bias,
                                  score == NVFP4_SCORE_SIGMOID, renormalize != 0, groups, top_groups,
                                  k, scale, experts, weights, dev_status,
                                  static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_route_backward(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld,
                                  const int32_t* experts, const float* dweights, int score, int k,
                                  int renormalize, float scale, void* dlogits, int64_t ldd,
                                  int* dev_status, void* stream)
{
    nvfp4_status st = check_logits(logits, dtype, T, E, ld, score, k);
    if (st != NVFP4_OK) return st;
    if (!experts || !dweights || !dlogits) return NVFP4_ERR_NULL;
    if (ldd < E) return NVFP4_ERR_SHAPE;
    const uintptr_t mask = dtype == NVFP4_OUT_F32 ? 3u : 1u;
    if (!aligned4(experts) || !aligned4(dweights) || (reinterpret_cast<uintptr_t>(dlogits) & mask))
        return NVFP4_ERR_ALIGN;
    int sms = 0;
    if ((st = current_device(&sms)) != NVFP4_OK) return st;
    return from_cuda(launch_route_backward(logits, dtype == NVFP4_OUT_BF16, T, E, ld, experts,
                                           dweights, score == NVFP4_SCORE_SIGMOID, renormalize != 0,
                                           k, scale, dlogits, ldd, dev_status,
                                           static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_plan_experts(const int32_t* experts, const nvfp4_expert_plan* plan,
                                void* workspace, int* dev_status, void* stream)
{
    if (!experts) return NVFP4_ERR_NULL;
    nvfp4_status st = check_plan(plan);
    if (st != NVFP4_OK) return st;
    if (!aligned4(experts) || !aligned16(workspace)) return NVFP4_ERR_ALIGN;
    if (!workspace && nvfp4_expert_plan_workspace_bytes(plan->tokens, plan->k, plan->experts))
        return NVFP4_ERR_NULL;
    int sms = 0;
    if ((st = current_device(&sms)) != NVFP4_OK) return st;
    return from_cuda(launch_plan(experts, plan->tokens * plan->k, static_cast<int>(plan->k),
                                 static_cast<int>(plan->experts), plan->rows, plan->offsets,
                                 plan->pair_row, plan->row_token, static_cast<int32_t*>(workspace),
                                 dev_status, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_quantize_grouped(const void* x_bf16, int64_t cols, int64_t ld,
                                    const nvfp4_expert_plan* plan, uint16_t sign_mask,
                                    unsigned flags, uint64_t seed, uint64_t offset,
                                    const nvfp4_operand* out_row, const nvfp4_operand* out_col,
                                    void* workspace, int* dev_status, void* stream)
{
    const bool want_row = flags & NVFP4_ROWWISE, want_col = flags & NVFP4_COLWISE;
    const bool sr = flags & NVFP4_SR, given = flags & NVFP4_AMAX_GIVEN, gather = flags & NVFP4_GATHER;
    if (flags & ~static_cast<unsigned>(NVFP4_ROWWISE | NVFP4_COLWISE | NVFP4_SR | NVFP4_AMAX_GIVEN |
                                       NVFP4_GATHER))
        return NVFP4_ERR_ARG;
    if (!want_row && !want_col) return NVFP4_ERR_ARG;
    nvfp4_status st = check_plan(plan);
    if (st != NVFP4_OK) return st;
    if ((st = check_rows_matrix(x_bf16, cols, ld, 8)) != NVFP4_OK) return st;
    if (cols % 16 || (want_row && cols % 64)) return NVFP4_ERR_SHAPE;
    const int64_t rows = plan->rows;
    if (want_row && (st = check_operand(out_row, rows, cols)) != NVFP4_OK) return st;
    if (want_col && (st = check_operand(out_col, cols, rows)) != NVFP4_OK) return st;
    if (!given && !workspace) return NVFP4_ERR_NULL;
    if (!aligned16(workspace)) return NVFP4_ERR_ALIGN;
    int sms = 0;
    if ((st = current_device(&sms)) != NVFP4_OK) return st;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    TileArgs a{};
    a.x = static_cast<const uint16_t*>(x_bf16);
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    a.map = row_map(*plan, gather, dev_status);
    if (given) {
        a.src.amax_given = want_row ? out_row->amax : nullptr;
        a.src_col.amax_given = want_col ? out_col->amax : nullptr;
    } else if (want_col || sr || !grouped_amax_is_small(cols, a.map)) {
        // [RHT partials][plain partials], as in nvfp4_quantize_row_rht
        uint32_t* rht = static_cast<uint32_t*>(workspace);
        uint32_t* plain = rht + kMaxPartials;
        const int grid = amax_grouped_grid(rows, cols, want_col, a.map, sms);
        a.src.partials = plain;
        a.src_col.partials = rht;
        a.src.n_partials = a.src_col.n_partials = grid;
        st = from_cuda(launch_amax_grouped(a.x, rows, cols, ld, want_col, sign_mask,
                                           want_col ? rht : plain, want_row ? plain : nullptr, grid,
                                           a.map, dev_status, s));
        if (st != NVFP4_OK) return st;
    }
    if (want_row) {
        a.row_codes = static_cast<uint8_t*>(out_row->codes);
        a.row_scales = static_cast<uint8_t*>(out_row->scales);
        a.row_amax = out_row->amax;
    } else {
        a.src = a.src_col;  // the single-output kernels read `src`
    }
    if (want_col) {
        a.col_codes = static_cast<uint8_t*>(out_col->codes);
        a.col_scales = static_cast<uint8_t*>(out_col->scales);
        a.col_amax = out_col->amax;
    }
    a.sign_mask = sign_mask;
    a.keys = philox_round_keys(seed);
    a.offset = offset;
    a.offset_col = offset + 1;
    a.dev_status = dev_status;
    if (!want_col) return from_cuda(launch_quant_grouped_rows(a, sr, sms, s));
    return from_cuda(launch_quant_grouped_tile(a, want_row, sr, sms, s));
}

static nvfp4_status gemm_by_rows(const nvfp4_operand* A, const nvfp4_operand* B,
                                 const nvfp4_expert_plan* plan, void* D, int d_dtype, int64_t ldd,
                                 bool after_quantizer, int* dev_status, void* stream)
{
    nvfp4_status st = check_plan(plan);
    if (st != NVFP4_OK) return st;
    if (!A || !B) return NVFP4_ERR_NULL;
    const int64_t E = plan->experts, K = A->cols;
    if ((st = check_operand(A, plan->rows, K)) != NVFP4_OK) return st;
    if ((st = check_operand(B, B->rows, B->cols)) != NVFP4_OK) return st;
    if (K < 64 || K % 64 || K >= kMaxDim || B->rows < 16 || B->rows >= kMaxDim || B->cols >= kMaxDim)
        return NVFP4_ERR_SHAPE;
    GroupedGemmArgs g{};
    set_operands(g, *A, *B);
    if (B->cols == K && B->rows % E == 0) {  // stacked by rows
        g.N = B->rows / E;
        g.b_row_step = g.N;
        if (E > 1 && g.N % 128) return NVFP4_ERR_SHAPE;
    } else if (B->cols == K * E) {           // side by side
        g.N = B->rows;
        g.b_k_step = K;
    } else {
        return NVFP4_ERR_SHAPE;
    }
    if ((st = check_gemm_output(D, d_dtype, g.N, ldd)) != NVFP4_OK) return st;
    g.offsets = plan->offsets;
    g.experts = E;
    g.rows = plan->rows;
    g.K = K;
    g.D = D;
    g.ldd = ldd;
    g.out_bf16 = d_dtype == NVFP4_OUT_BF16;
    g.dev_status = dev_status;
    g.after_quantizer = after_quantizer;
    if (plan->rows / 128 * ((g.N + 255) / 256) >= kMaxDim) return NVFP4_ERR_SHAPE;
    int sms = 0;
    if ((st = current_device(&sms)) != NVFP4_OK) return st;
    return from_cuda(launch_gemm_grouped(g, sms, static_cast<cudaStream_t>(stream)));
}

static nvfp4_status gemm_by_k(const nvfp4_operand* A, const nvfp4_operand* B,
                              const nvfp4_expert_plan* plan, void* D, int d_dtype, int64_t ldd,
                              bool after_quantizer, int* dev_status, void* stream)
{
    nvfp4_status st = check_plan(plan);
    if (st != NVFP4_OK) return st;
    if (!A || !B) return NVFP4_ERR_NULL;
    const int64_t E = plan->experts;
    if ((st = check_operand(A, A->rows, plan->rows)) != NVFP4_OK) return st;
    if ((st = check_operand(B, B->rows, plan->rows)) != NVFP4_OK) return st;
    if (A->rows < 128 || A->rows % 128 || A->rows * E >= kMaxDim) return NVFP4_ERR_SHAPE;
    if ((st = check_gemm_output(D, d_dtype, B->rows, ldd)) != NVFP4_OK) return st;
    GroupedGemmArgs g{};
    set_operands(g, *A, *B);
    g.by_k = true;
    g.M = A->rows;
    g.N = B->rows;
    g.offsets = plan->offsets;
    g.experts = E;
    g.rows = plan->rows;
    g.D = D;
    g.ldd = ldd;
    g.out_bf16 = d_dtype == NVFP4_OUT_BF16;
    g.dev_status = dev_status;
    g.after_quantizer = after_quantizer;
    if (E * ((g.M + 255) / 256) * ((g.N + 255) / 256) >= kMaxDim) return NVFP4_ERR_SHAPE;
    int sms = 0;
    if ((st = current_device(&sms)) != NVFP4_OK) return st;
    return from_cuda(launch_gemm_grouped(g, sms, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_gemm_grouped(const nvfp4_operand* A, const nvfp4_operand* B,
                                const nvfp4_expert_plan* plan, void* D, int d_dtype, int64_t ldd,
                                int* dev_status, void* stream)
{
    return gemm_by_rows(A, B, plan, D, d_dtype, ldd, false, dev_status, stream);
}

nvfp4_status nvfp4_gemm_grouped_k(const nvfp4_operand* A, const nvfp4_operand* B,
                                  const nvfp4_expert_plan* plan, void* D, int d_dtype, int64_t ldd,
                                  int* dev_status, void* stream)
{
    return gemm_by_k(A, B, plan, D, d_dtype, ldd, false, dev_status, stream);
}

size_t nvfp4_experts_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t rows, int64_t I,
                                     int64_t O)
{
    const int64_t need = nvfp4_expert_rows(T, k, E);
    if (need == 0 || rows < need || rows % kRegion || rows > kMaxRows || I <= 0 || O <= 0 || I % 64 ||
        O % 128)
        return 0;
    const size_t fprop = operand_bytes(rows, I), dgrad = operand_bytes(rows, O);
    const size_t wgrad = operand_bytes(O, rows) + operand_bytes(I, rows);
    size_t m = fprop > dgrad ? fprop : dgrad;
    m = m > wgrad ? m : wgrad;
    return m + round256(nvfp4_workspace_bytes(128, 128, 0));
}

static nvfp4_status check_experts(const nvfp4_expert_plan* plan, int64_t I, int64_t O,
                                  const void* workspace)
{
    const nvfp4_status st = check_plan(plan);
    if (st != NVFP4_OK) return st;
    if (!workspace) return NVFP4_ERR_NULL;
    if (I < 64 || I % 64 || O < 128 || O % 128 || I >= kMaxDim || O >= kMaxDim ||
        O * plan->experts >= kMaxDim)
        return NVFP4_ERR_SHAPE;
    // the products' tile counts (checked by them too, but after the quantization is queued)
    const int64_t ti = (I + 255) / 256, to = (O + 255) / 256;
    if (plan->rows / kRegion * (ti > to ? ti : to) >= kMaxDim || plan->experts * to * ti >= kMaxDim)
        return NVFP4_ERR_SHAPE;
    return aligned16(workspace) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

nvfp4_status nvfp4_experts_fprop(const void* X, int64_t ldx, int gather, const nvfp4_operand* W,
                                 const nvfp4_expert_plan* plan, int64_t I, int64_t O, void* Y,
                                 int y_dtype, int64_t ldy, void* workspace, int* dev_status,
                                 void* stream)
{
    nvfp4_status st = check_experts(plan, I, O, workspace);
    if (st != NVFP4_OK) return st;
    // everything the product checks, before the quantization is queued
    if ((st = check_operand(W, plan->experts * O, I)) != NVFP4_OK) return st;
    if ((st = check_gemm_output(Y, y_dtype, O, ldy)) != NVFP4_OK) return st;
    Carver c{static_cast<uint8_t*>(workspace)};
    const nvfp4_operand a = c.operand(plan->rows, I);
    if ((st = nvfp4_quantize_grouped(X, I, ldx, plan, 0, NVFP4_ROWWISE | (gather ? NVFP4_GATHER : 0),
                                     0, 0, &a, nullptr, c.at, dev_status, stream)) != NVFP4_OK)
        return st;
    return gemm_by_rows(&a, W, plan, Y, y_dtype, ldy, true, dev_status, stream);
}

nvfp4_status nvfp4_experts_dgrad(const void* dY, int64_t lddy, const nvfp4_operand* Wt,
                                 const nvfp4_expert_plan* plan, int64_t I, int64_t O, uint64_t seed,
                                 uint64_t offset, void* dX, int dx_dtype, int64_t lddx,
                                 void* workspace, int* dev_status, void* stream)
{
    nvfp4_status st = check_experts(plan, I, O, workspace);
    if (st != NVFP4_OK) return st;
    if ((st = check_operand(Wt, I, plan->experts * O)) != NVFP4_OK) return st;
    if ((st = check_gemm_output(dX, dx_dtype, I, lddx)) != NVFP4_OK) return st;
    Carver c{static_cast<uint8_t*>(workspace)};
    const nvfp4_operand a = c.operand(plan->rows, O);
    if ((st = nvfp4_quantize_grouped(dY, O, lddy, plan, 0, NVFP4_ROWWISE | NVFP4_SR, seed, offset, &a,
                                     nullptr, c.at, dev_status, stream)) != NVFP4_OK)
        return st;
    return gemm_by_rows(&a, Wt, plan, dX, dx_dtype, lddx, true, dev_status, stream);
}

nvfp4_status nvfp4_experts_wgrad(const void* dY, int64_t lddy, const void* X, int64_t ldx, int gather,
                                 const nvfp4_expert_plan* plan, int64_t I, int64_t O,
                                 uint16_t sign_mask, uint64_t seed, uint64_t offset, void* dW,
                                 int dw_dtype, int64_t lddw, void* workspace, int* dev_status,
                                 void* stream)
{
    nvfp4_status st = check_experts(plan, I, O, workspace);
    if (st != NVFP4_OK) return st;
    if ((st = check_gemm_output(dW, dw_dtype, I, lddw)) != NVFP4_OK) return st;
    if ((st = check_rows_matrix(X, I, ldx, 8)) != NVFP4_OK) return st;
    Carver c{static_cast<uint8_t*>(workspace)};
    const nvfp4_operand a = c.operand(O, plan->rows), b = c.operand(I, plan->rows);
    if ((st = nvfp4_quantize_grouped(dY, O, lddy, plan, sign_mask, NVFP4_COLWISE | NVFP4_SR, seed,
                                     offset, nullptr, &a, c.at, dev_status, stream)) != NVFP4_OK)
        return st;
    if ((st = nvfp4_quantize_grouped(X, I, ldx, plan, sign_mask,
                                     NVFP4_COLWISE | (gather ? NVFP4_GATHER : 0), 0, 0, nullptr, &b,
                                     c.at, dev_status, stream)) != NVFP4_OK)
        return st;
    return gemm_by_k(&a, &b, plan, dW, dw_dtype, lddw, true, dev_status, stream);
}

nvfp4_status nvfp4_combine(const void* Y_bf16, int64_t cols, int64_t ldy,
                           const nvfp4_expert_plan* plan, const float* weights, void* out,
                           int out_dtype, int64_t ldo, int* dev_status, void* stream)
{
    nvfp4_status st = check_plan(plan);
    if (st != NVFP4_OK) return st;
    if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_ARG;
    if ((st = check_rows_matrix(Y_bf16, cols, ldy, 8)) != NVFP4_OK) return st;
    if ((st = check_rows_matrix(out, cols, ldo, out_dtype == NVFP4_OUT_F32 ? 4 : 8)) != NVFP4_OK)
        return st;
    if (!aligned4(weights)) return NVFP4_ERR_ALIGN;
    int sms = 0;
    if ((st = current_device(&sms)) != NVFP4_OK) return st;
    CombineArgs a{};
    a.map = row_map(*plan, true, dev_status);
    a.rows = plan->rows;
    a.cols = cols;
    a.y = static_cast<const uint16_t*>(Y_bf16);
    a.ldy = ldy;
    a.weights = weights;
    a.out = out;
    a.ldo = ldo;
    a.dev_status = dev_status;
    return from_cuda(launch_combine(a, out_dtype == NVFP4_OUT_F32, sms,
                                    static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_combine_backward(const void* dout, int dout_dtype, int64_t ldo,
                                    const void* Y_bf16, int64_t cols, int64_t ldy,
                                    const nvfp4_expert_plan* plan, const float* weights,
                                    void* dY_bf16, int64_t lddy, float* dweights, int* dev_status,
                                    void* stream)
{
    nvfp4_status st = check_plan(plan);
    if (st != NVFP4_OK) return st;
    if (dout_dtype != NVFP4_OUT_F32 && dout_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_ARG;
    if (!weights || !dweights) return NVFP4_ERR_NULL;
    if ((st = check_rows_matrix(dout, cols, ldo, dout_dtype == NVFP4_OUT_F32 ? 4 : 8)) != NVFP4_OK)
        return st;
    if ((st = check_rows_matrix(Y_bf16, cols, ldy, 8)) != NVFP4_OK) return st;
    if ((st = check_rows_matrix(dY_bf16, cols, lddy, 8)) != NVFP4_OK) return st;
    if (!aligned4(weights) || !aligned4(dweights)) return NVFP4_ERR_ALIGN;
    int sms = 0;
    if ((st = current_device(&sms)) != NVFP4_OK) return st;
    CombineArgs a{};
    a.map = row_map(*plan, true, dev_status);
    a.rows = plan->rows;
    a.cols = cols;
    a.y = static_cast<const uint16_t*>(Y_bf16);
    a.ldy = ldy;
    a.weights = weights;
    a.dout = dout;
    a.ldo = ldo;
    a.dy = static_cast<uint16_t*>(dY_bf16);
    a.lddy = lddy;
    a.dweights = dweights;
    a.dev_status = dev_status;
    return from_cuda(launch_combine_backward(a, dout_dtype == NVFP4_OUT_F32, sms,
                                             static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
