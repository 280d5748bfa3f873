"""MI355X-native single-GPU fine-grained MoE FFN layer forward.

Five steps, five C-ABI entry points in libmoe.so (declared in include/moe.h),
each wrapped here with the same name: moe_route, moe_dispatch,
moe_expert_ffn, moe_combine, moe_load_stats (moe_dispatch_capped is the
dispatch with expert capacities enforced; moe_expert_ffn_gather the FFN
reading token rows through the permutation, with no copy of them); and moe_bias_update, the
dynamic routing-bias step that feeds the next layer call. Around the layer, for
a whole decoder block: moe_norm, moe_norm_residual, moe_route_grouped,
moe_linear and moe_linear_grouped, run together by moe_block_forward and
MoEBlockGraph. In 8 bits: moe_quantize, moe_quantize_weight, moe_linear_fp8 and
moe_linear_grouped_fp8; moe_layer_few is the whole layer for up to 64 tokens in two
or three launches (moe_block_forward takes both as options). Every step runs in the HIP kernels;
this package only marshals tensors, sizes and the current stream.
"""
from .binding import (MoEBlockGraph, MoEError, MoELayerGraph, lib, moe_block_forward, moe_bias_update, moe_capacity, moe_combine,
                      moe_dispatch, moe_dispatch_noalloc, moe_expert_ffn, moe_expert_ffn_gather,
                      moe_layer_few, moe_layer_few_workspace_bytes, moe_layer_forward, moe_linear, moe_linear_fp8, moe_linear_fp8_path,
                      moe_linear_grouped, moe_linear_grouped_fp8, moe_linear_path, moe_load_stats,
                      moe_norm, moe_norm_residual, moe_quantize, moe_quantize_weight, moe_route, moe_route_grouped, moe_status_string,
                      moe_dispatch_workspace_bytes, moe_expert_ffn_workspace_bytes,
                      moe_linear_fp8_workspace_bytes, moe_linear_grouped_fp8_workspace_bytes,
                      moe_linear_grouped_workspace_bytes, moe_linear_workspace_bytes,
                      moe_route_grouped_workspace_bytes, moe_route_workspace_bytes)

__all__ = ["MoEError", "MoELayerGraph", "lib", "moe_route", "moe_dispatch",
           "moe_dispatch_noalloc", "moe_expert_ffn",
           "moe_expert_ffn_gather", "moe_combine",
           "moe_load_stats", "moe_bias_update", "moe_capacity", "moe_layer_forward", "moe_status_string",
           "moe_dispatch_workspace_bytes", "moe_expert_ffn_workspace_bytes",
           "moe_route_workspace_bytes", "moe_norm", "moe_norm_residual", "moe_route_grouped",
           "moe_linear", "moe_linear_grouped", "moe_linear_path", "moe_block_forward", "MoEBlockGraph",
           "moe_route_grouped_workspace_bytes", "moe_linear_workspace_bytes",
           "moe_linear_grouped_workspace_bytes", "moe_quantize", "moe_quantize_weight",
           "moe_linear_fp8", "moe_linear_grouped_fp8", "moe_linear_fp8_path",
           "moe_linear_fp8_workspace_bytes", "moe_linear_grouped_fp8_workspace_bytes", "moe_layer_few",
           "moe_layer_few_workspace_bytes"]
