"""MI355X-native DeepSeek-R1-style MoE layer: Python binding of libmoe.so.

The layer's steps are the C-ABI calls declared in include/moe.h
(moe_route, moe_permute, moe_expert_ffn, moe_combine, moe_balanced_partition,
moe_gather_rows, moe_quantize_tokens with moe_expert_ffn_gate_up_tokens,
moe_quantize_mxfp4 for 4-bit experts, moe_layer_few for a few tokens,
moe_pre_norm and moe_combine_norm around the layer, for online rebalancing
moe_count_accumulate, moe_coactivation, moe_affinity_partition, and for training
moe_grouped_gemm, moe_grouped_gemm_dx, moe_grouped_gemm_dw, moe_swiglu,
moe_swiglu_grad, moe_dropout, moe_combine_grad, moe_route_grad), implemented as
HIP kernels for gfx950. This package only marshals arguments; ``build()``
compiles the library with hipcc.
"""
from ._lib import (BF16, F32, FP8_E4M3, MXFP4, SIGMOID, SOFTMAX, EXPORTS, MoEError, dtype_code, lib, make_weights,
                   moe_affinity_partition, moe_balanced_partition, moe_coactivation, moe_combine, moe_combine_grad,
                   moe_combine_norm, moe_count_accumulate, moe_dequantize_mxfp4, moe_dropout, moe_expert_ffn, moe_expert_ffn_down,
                   moe_expert_ffn_gate_up, moe_expert_ffn_gate_up_tokens, moe_expert_ffn_noalloc,
                   NOALLOC_SCRATCH_BYTES, moe_expert_ffn_workspace_size, moe_gather_rows, moe_grouped_gemm,
                   moe_grouped_gemm_dw, moe_grouped_gemm_dx, moe_layer_few,
                   moe_layer_few_workspace_size, moe_layer_fused, moe_layer_fused_workspace_size, moe_permute,
                   moe_permute_workspace_size, moe_pre_norm, moe_quantize_mxfp4, moe_quantize_tokens, moe_route,
                   moe_route_grad, moe_route_select, moe_route_select_workspace_size, moe_swiglu, moe_swiglu_grad)
from .layer import LayerBuffers, LayerGrads, MoELayer, TrainStep, quantize_mxfp4


def build(verbose: bool = False) -> str:
    from .build import build as _build
    return _build(verbose)
