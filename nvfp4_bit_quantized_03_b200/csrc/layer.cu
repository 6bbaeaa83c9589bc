// C entry points of the operators around a layer's products (include/nvfp4.h): argument checks,
// workspace sizes and dispatch to qk_norm.cu and orthogonalize.cu.  As everywhere in the library: no allocation, no
// synchronization, and nothing queued when an argument is invalid.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_common.h"
#include "heads_overlap.h"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxHeads = 1 << 20;
constexpr int64_t kMaxTokens = 1 << 30;
// beyond any GPU's memory; the output's tensor map takes strides below 2^40 bytes
constexpr int64_t kMaxStride = int64_t(1) << 38;
constexpr int64_t kMaxExtent = int64_t(1) << 48;

bool known_type(int dtype) { return dtype == NVFP4_OUT_F32 || dtype == NVFP4_OUT_BF16; }

bool heads_sizes_ok(int64_t tokens, int64_t heads_q, int64_t heads_k, int64_t head_dim)
{
    return tokens >= 1 && tokens <= kMaxTokens && heads_q >= 1 && heads_q <= kMaxHeads && heads_k >= 0 &&
           heads_k <= kMaxHeads && head_dim >= 16 && head_dim <= kMaxHeadDim && head_dim % 16 == 0;
}

// A view of `heads` heads; `written`: no two of its values share a place.
nvfp4_status check_heads(const nvfp4_heads& v, int64_t heads, int64_t tokens, int64_t D, int dtype,
                         bool written)
{
    if (!v.data) return NVFP4_ERR_NULL;
    if (v.heads != heads || v.token_stride < 0 || v.head_stride < 0 || v.token_stride > kMaxStride ||
        v.head_stride > kMaxStride)
        return NVFP4_ERR_SHAPE;
    // from the first token or head to the last one
    if ((tokens > 1 && v.token_stride > kMaxExtent / (tokens - 1)) || (heads > 1 && v.head_stride > kMaxExtent / (heads - 1)))
        return NVFP4_ERR_SHAPE;
    const int64_t per16 = dtype == NVFP4_OUT_F32 ? 4 : 8;
    if (!aligned16(v.data) || (tokens > 1 && v.token_stride % per16) || (heads > 1 && v.head_stride % per16))
        return NVFP4_ERR_ALIGN;
    if (written) {
        const int64_t across_heads = heads > 1 ? (heads - 1) * v.head_stride + D : D;
        const int64_t across_tokens = tokens > 1 ? (tokens - 1) * v.token_stride + D : D;
        const bool by_token = (heads == 1 || v.head_stride >= D) &&
                              (tokens == 1 || v.token_stride >= across_heads);
        const bool by_head = (tokens == 1 || v.token_stride >= D) &&
                             (heads == 1 || v.head_stride >= across_tokens);
        if (!by_token && !by_head) return NVFP4_ERR_SHAPE;
    }
    return NVFP4_OK;
}

struct HeadsPair {  // a view of the queries' and of the keys' heads
    const nvfp4_heads* q;
    const nvfp4_heads* k;
    int dtype;
    bool written;
};

nvfp4_status take_heads(const HeadsPair& in, int64_t heads_q, int64_t heads_k, int64_t tokens, int64_t D,
                        HeadsView* out)
{
    if (!in.q || (heads_k > 0 && !in.k)) return NVFP4_ERR_NULL;
    if (!known_type(in.dtype)) return NVFP4_ERR_ARG;
    nvfp4_status st = check_heads(*in.q, heads_q, tokens, D, in.dtype, in.written);
    if (st != NVFP4_OK) return st;
    if (heads_k > 0 && (st = check_heads(*in.k, heads_k, tokens, D, in.dtype, in.written)) != NVFP4_OK)
        return st;
    const nvfp4_heads none = {nullptr, 0, 0, 0};
    for (int i = 0; i < 2; ++i) {
        const nvfp4_heads& v = i == 0 ? *in.q : (heads_k > 0 ? *in.k : none);
        // a single token's or head's stride is never used
        out[i] = HeadsView{v.data, v.heads, tokens > 1 ? v.token_stride : 0, v.heads > 1 ? v.head_stride : 0};
    }
    return NVFP4_OK;
}

// No head that is written (views[n - 1]) shares a byte with another one of the call's, except that it may be
// the head of its own that is read, at the same place.
nvfp4_status check_apart(const HeadsPair* in, const HeadsView* const* views, int n, int64_t tokens, int64_t D)
{
    auto runs = [&](int i, int kind) {
        const HeadsView& v = views[i][kind];
        const int64_t size = in[i].dtype == NVFP4_OUT_F32 ? 4 : 2;
        return Runs(v.data, v.heads, tokens, size * D, size * v.head_stride, size * v.token_stride);
    };
    auto same = [&](int i, int j, int kind) {
        const HeadsView &a = views[i][kind], &b = views[j][kind];
        return in[i].dtype == in[j].dtype && a.data == b.data && a.token_stride == b.token_stride &&
               a.head_stride == b.head_stride;
    };
    for (int kind = 0; kind < 2; ++kind) {
        if (views[n - 1][kind].heads == 0) continue;
        const Runs out = runs(n - 1, kind);
        for (int i = 0; i < n; ++i)
            for (int other = 0; other < 2; ++other) {
                if (views[i][other].heads == 0 || (other == kind && (i == n - 1 || same(i, n - 1, kind)))) continue;
                if (runs_meet(out, runs(i, other))) return NVFP4_ERR_SHAPE;
            }
    }
    return NVFP4_OK;
}

// What both directions share; in[0] is x.
nvfp4_status head_args(HeadsArgs& a, const HeadsPair* in, HeadsView* const* views, int n, int64_t tokens,
                       int64_t D, const float* q_weight, const float* k_weight, float eps,
                       const int32_t* positions, const float* table, int64_t table_rows, int64_t rotary,
                       int* dev_status)
{
    if (!in[0].q) return NVFP4_ERR_NULL;
    const int64_t hq = in[0].q->heads, hk = in[0].k ? in[0].k->heads : 0;
    if (!heads_sizes_ok(tokens, hq, hk, D)) return NVFP4_ERR_SHAPE;
    if (rotary < 0 || rotary > D || rotary % 16) return NVFP4_ERR_SHAPE;
    if (rotary > 0 && (table_rows < 1 || table_rows >= kMaxDim)) return NVFP4_ERR_SHAPE;
    if (rotary > 0 && !table) return NVFP4_ERR_NULL;
    if (rotary > 0 && !positions && table_rows < tokens) return NVFP4_ERR_SHAPE;
    // squares below FP32's smallest are zeros, which a smaller eps would show
    if (!(eps >= 1e-30f) || !(eps <= 1e30f)) return NVFP4_ERR_ARG;
    for (int i = 0; i < n; ++i) {
        const nvfp4_status st = take_heads(in[i], hq, hk, tokens, D, views[i]);
        if (st != NVFP4_OK) return st;
    }
    if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned16(table) || !aligned4(positions))
        return NVFP4_ERR_ALIGN;
    a.weight[0] = q_weight;
    a.weight[1] = k_weight;
    a.positions = positions;
    a.table = table;
    a.tokens = tokens;
    a.table_rows = table_rows;
    a.D = static_cast<int>(D);
    a.rotary = static_cast<int>(rotary);
    a.eps = eps;
    a.dev_status = dev_status;
    return NVFP4_OK;
}

constexpr int64_t kMaxSide = 1 << 18;     // FP16 copies times ~ sqrt(side) stay far inside their range
constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxValues = int64_t(1) << 36;

bool matrices_ok(int64_t batch, int64_t rows, int64_t cols)
{
    return batch >= 1 && batch <= kMaxBatch && rows >= 1 && rows <= kMaxSide && cols >= 1 && cols <= kMaxSide &&
           batch * rows * cols <= kMaxValues;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_qk_norm_rope(const nvfp4_heads* q, const nvfp4_heads* k, int in_dtype, int64_t tokens,
                                int64_t head_dim, const float* q_weight, const float* k_weight, float eps,
                                const int32_t* positions, const float* table, int64_t table_rows,
                                int64_t rotary, int interleaved, const nvfp4_heads* q_out,
                                const nvfp4_heads* k_out, int out_dtype, int* dev_status, void* stream)
{
    HeadsArgs a = {};
    const HeadsPair in[2] = {{q, k, in_dtype, false}, {q_out, k_out, out_dtype, true}};
    HeadsView* const views[2] = {a.x, a.z};
    nvfp4_status st = head_args(a, in, views, 2, tokens, head_dim, q_weight, k_weight, eps, positions, table,
                                table_rows, rotary, dev_status);
    if (st != NVFP4_OK) return st;
    int sms = 0;
    if ((st = current_device(&sms)) != NVFP4_OK) return st;
    if ((st = check_apart(in, views, 2, tokens, head_dim)) != NVFP4_OK) return st;
    return from_cuda(launch_qk_norm_rope(a, in_dtype == NVFP4_OUT_F32, out_dtype == NVFP4_OUT_F32,
                                         interleaved != 0, sms, static_cast<cudaStream_t>(stream)));
}

size_t nvfp4_qk_norm_rope_workspace_bytes(int64_t tokens, int64_t heads_q, int64_t heads_k, int64_t head_dim)
{
    if (!heads_sizes_ok(tokens, heads_q, heads_k, head_dim)) return 0;
    return sizeof(float) * static_cast<size_t>(head_dim) *
           static_cast<size_t>(qk_backward_ctas(tokens, heads_q, heads_k, head_dim));
}

nvfp4_status nvfp4_qk_norm_rope_backward(const nvfp4_heads* dq, const nvfp4_heads* dk, int grad_dtype,
                                         const nvfp4_heads* q, const nvfp4_heads* k, int in_dtype,
                                         int64_t tokens, int64_t head_dim, const float* q_weight,
                                         const float* k_weight, float eps, const int32_t* positions,
                                         const float* table, int64_t table_rows, int64_t rotary,
                                         int interleaved, const nvfp4_heads* dq_in, const nvfp4_heads* dk_in,
                                         int dx_dtype, float* dq_weight, float* dk_weight, void* workspace,
                                         int* dev_status, void* stream)
{
    HeadsArgs a = {};
    const HeadsPair in[3] = {{q, k, in_dtype, false}, {dq, dk, grad_dtype, false}, {dq_in, dk_in, dx_dtype, true}};
    HeadsView* const views[3] = {a.x, a.z, a.dx};
    nvfp4_status st = head_args(a, in, views, 3, tokens, head_dim, q_weight, k_weight, eps, positions, table,
                                table_rows, rotary, dev_status);
    if (st != NVFP4_OK) return st;
    if (!workspace) return NVFP4_ERR_NULL;
    if (!aligned16(workspace) || !aligned4(dq_weight) || !aligned4(dk_weight)) return NVFP4_ERR_ALIGN;
    a.partials = static_cast<float*>(workspace);
    a.dweight[0] = dq_weight;
    a.dweight[1] = dk_weight;
    int sms = 0;
    if ((st = current_device(&sms)) != NVFP4_OK) return st;
    if ((st = check_apart(in, views, 3, tokens, head_dim)) != NVFP4_OK) return st;
    return from_cuda(launch_qk_norm_rope_backward(a, in_dtype == NVFP4_OUT_F32, grad_dtype == NVFP4_OUT_F32,
                                                  dx_dtype == NVFP4_OUT_F32, interleaved != 0,
                                                  static_cast<cudaStream_t>(stream)));
}

size_t nvfp4_orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols)
{
    return matrices_ok(batch, rows, cols) ? orthogonalize_workspace(batch, rows, cols) : 0;
}

nvfp4_status nvfp4_selftest_orthogonalize_ways(int64_t batch, int64_t rows, int64_t cols, int* ways)
{
    if (!ways) return NVFP4_ERR_NULL;
    if (!matrices_ok(batch, rows, cols)) return NVFP4_ERR_SHAPE;
    int sms = 0;
    const nvfp4_status st = current_device(&sms);
    return st == NVFP4_OK ? from_cuda(orthogonalize_ways(batch, rows, cols, sms, ways)) : st;
}

nvfp4_status nvfp4_orthogonalize(const void* G, int g_dtype, int64_t batch, int64_t rows, int64_t cols, int64_t ldg,
                                 int64_t g_stride, int steps, const float* coefficients, double eps, void* out_bf16,
                                 int64_t ldo, int64_t out_stride, void* workspace, int* dev_status, void* stream)
{
    if (!G || !coefficients || !out_bf16 || !workspace) return NVFP4_ERR_NULL;
    if (!known_type(g_dtype)) return NVFP4_ERR_ARG;
    if (!matrices_ok(batch, rows, cols)) return NVFP4_ERR_SHAPE;
    if (steps < 1 || steps > kMaxOrthogonalizeSteps || !(eps >= 0.0) || !(eps <= 1e30)) return NVFP4_ERR_ARG;
    for (int i = 0; i < 3 * steps; ++i)
        if (!(std::fabs(coefficients[i]) <= 1e6f)) return NVFP4_ERR_ARG;
    // a single row's or matrix's stride is never used
    if (rows == 1) ldg = cols, ldo = (cols + 7) / 8 * 8;
    if (batch == 1) g_stride = rows * ldg, out_stride = (rows * ldo + 7) / 8 * 8;
    if (ldg < 0 || ldg > kMaxStride || g_stride < 0 || g_stride > kMaxStride) return NVFP4_ERR_SHAPE;
    if (ldo < cols || ldo > kMaxStride || out_stride < (rows - 1) * ldo + cols || out_stride > kMaxStride)
        return NVFP4_ERR_SHAPE;
    const uintptr_t mask = g_dtype == NVFP4_OUT_F32 ? 3u : 1u;
    if ((reinterpret_cast<uintptr_t>(G) & mask) || (reinterpret_cast<uintptr_t>(out_bf16) & 1u) ||
        !aligned16(workspace))
        return NVFP4_ERR_ALIGN;
    int sms = 0;
    const nvfp4_status st = current_device(&sms);
    if (st != NVFP4_OK) return st;
    OrthogonalizeArgs a = {};
    a.g = G;
    a.f32 = g_dtype == NVFP4_OUT_F32;
    a.batch = batch;
    a.rows = rows;
    a.cols = cols;
    a.ldg = ldg;
    a.g_stride = g_stride;
    a.steps = steps;
    a.coefficients = coefficients;
    a.eps = eps;
    a.out = out_bf16;
    a.ldo = ldo;
    a.out_stride = out_stride;
    a.workspace = workspace;
    a.dev_status = dev_status;
    return from_cuda(launch_orthogonalize(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
