"""GB300-native block-scaled FP8 GEMM: D = C + A @ B^T with 1x128 (A) and
128x128 (B) scales, FP32 accumulation, bf16 output, plus the M-grouped MoE
variants and the scale-layout transform.  The compute runs in the CUDA
library built from csrc/ (C ABI in include/dg.h); ``binding`` marshals torch
tensors into it.  ``inputs`` generates seeded synthetic problems."""
from . import binding  # noqa: F401  (loading the .so is deferred to the first call)
from .binding import (DGError, dg_fp8_gemm_nt, dg_m_grouped_fp8_gemm_nt_contiguous,  # noqa: F401
                      dg_m_grouped_fp8_gemm_nt_masked, dg_transform_sf, transform_sf,
                      dg_bf16_fp4_gemv_nt, dg_bf16_fp8_gemv_nt, dg_moe_route, dg_moe_fp4_layer, dg_moe_fp8_layer,
                      dg_fp8_gated_gemm_nt, dg_m_grouped_fp8_gated_gemm_nt_contiguous, dg_fp8_gated_gemm_nn_backward,
                      dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous, dg_quantize_fp8, dg_quantize_fp8_blocks,
                      dg_newton_schulz)
