// Argument checks and workspace arithmetic shared by the C entry points (api.cu, experts.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4.h"
#include "nvfp4_internal.h"

namespace nvfp4 {

// The current device if it is a compute-capability 10.0 GPU.
nvfp4_status current_device(int* sm_count);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline size_t round256(size_t v) { return (v + 255u) & ~static_cast<size_t>(255u); }

constexpr int64_t kMaxDim = int64_t(1) << 31;

inline nvfp4_status check_operand(const nvfp4_operand* op, int64_t rows, int64_t cols)
{
    if (!op || !op->codes || !op->scales || !op->amax) return NVFP4_ERR_NULL;
    if (op->rows != rows || op->cols != cols) return NVFP4_ERR_SHAPE;
    if (!aligned16(op->codes) || !aligned16(op->scales) || !aligned4(op->amax))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

inline nvfp4_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

inline size_t operand_bytes(int64_t rows, int64_t cols)
{
    return round256(nvfp4_codes_bytes(rows, cols)) + round256(nvfp4_scales_bytes(rows, cols)) + 256;
}

// Cuts a workspace into 256-byte aligned pieces.
struct Carver {
    uint8_t* at;
    uint8_t* take(size_t n)
    {
        uint8_t* q = at;
        at += round256(n);
        return q;
    }
    nvfp4_operand operand(int64_t rows, int64_t cols)
    {
        nvfp4_operand op;
        op.rows = rows;
        op.cols = cols;
        op.codes = take(nvfp4_codes_bytes(rows, cols));
        op.scales = take(nvfp4_scales_bytes(rows, cols));
        op.amax = reinterpret_cast<float*>(take(4));
        return op;
    }
};

}  // namespace nvfp4
