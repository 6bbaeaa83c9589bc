"""NVFP4 training hot path on B200 (sm_100a): quantizers and block-scaled FP4 GEMMs for the
three GEMMs of a linear layer or of a layer of experts, head norms with the position rotation behind
a QKV projection, and the Newton-Schulz update of weight gradients, behind the C ABI of libnvfp4.so
(include/nvfp4.h).

The Python surface is the ctypes binding in ``binding``; it loads the in-tree
``libnvfp4.so`` on first use and raises if the library is missing.
"""
from . import binding
from .binding import (AMAX_GIVEN, BLOCK2D, COLWISE, GATHER, OUT_BF16, OUT_F32, ROWWISE, SR,
                      DEVSTAT_BOUNDS, DEVSTAT_INDEX, DEVSTAT_NONFINITE, DEVSTAT_TIMEOUT,
                      ExpertPlan, NVFP4Error, QuantizedTensor, bounds_checked, combine,
                      combine_backward, expert_plan, experts_dgrad, experts_fprop, experts_wgrad,
                      gemm, gemm_grouped, gemm_grouped_k, linear_dgrad, linear_fprop, linear_wgrad, orthogonalize,
                      qk_norm_rope, qk_norm_rope_backward, quantize, quantize_grouped,
                      rht_quantize, rope_table, route, route_backward, sign_mask_from_seed)

__all__ = ["binding", "AMAX_GIVEN", "BLOCK2D", "COLWISE", "GATHER", "OUT_BF16", "OUT_F32",
           "ROWWISE", "SR", "DEVSTAT_BOUNDS", "DEVSTAT_INDEX", "DEVSTAT_NONFINITE",
           "DEVSTAT_TIMEOUT", "ExpertPlan", "NVFP4Error", "QuantizedTensor", "bounds_checked",
           "combine", "combine_backward", "expert_plan", "experts_dgrad", "experts_fprop",
           "experts_wgrad", "gemm", "gemm_grouped", "gemm_grouped_k", "linear_dgrad",
           "linear_fprop", "linear_wgrad", "orthogonalize", "qk_norm_rope",
           "qk_norm_rope_backward", "quantize", "quantize_grouped", "rht_quantize", "rope_table", "route", "route_backward",
           "sign_mask_from_seed"]
