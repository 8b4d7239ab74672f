"""MI355X (gfx950) scaled FP8 linear layer.

The compute path is ``libfp8lin.so`` (hand-written HIP kernels behind a C ABI,
declared in ``include/fp8lin.h``); this package is its thin Python binding
(``_abi``) plus the host-side delayed-scaling schedule (``state``). PyTorch is
used for device memory and streams only. Importing works without the built
library; calling any entry point without it raises.
"""
from ._abi import (FP8_A_E5M2, FP8_AMAX_ACCUMULATE, FP8_BLOCK_1x128, FP8_E5M2, FP8_BLOCK_128x128, FP8_SCALE_CLEAR_AMAX,
                   FP8_SCALE_FROM_AMAX, FP8_SCALE_RECORD, FP8_SCALE_REFRESH, FP8_TENSORWISE,
                   FP8_LAYOUT_BSHD, FP8_LAYOUT_THD, Fp8Error, Slot, fp8_align_multiple,
                   fp8_bias_grad, fp8_last_error, fp8_pad_varlen, fp8_unpad_varlen,
                   fp8_linear_dgrad, fp8_linear_fwd, fp8_linear_fwd_current, fp8_linear_wgrad,
                   fp8_pad_tokens,
                   fp8_quantize_amax, fp8_scale_update, fp8_version, load,
                   FP8_DT_BF16, FP8_DT_F16, FP8_DT_F32, fp8_layernorm_fwd, fp8_layernorm_bwd,
                   fp8_layernorm_bwd_workspace, fp8_moe_rows, fp8_moe_sort,
                   fp8_moe_sort_workspace, fp8_moe_dispatch, fp8_moe_dispatch_bwd,
                   fp8_moe_combine, fp8_moe_combine_bwd, FP8_ACT_RELU, FP8_ACT_SILU, FP8_ACT_GELU,
                   fp8_moe_route, fp8_moe_route_bwd, fp8_moe_route_workspace, fp8_act_quantize,
                   fp8_act_quantize_bwd, fp8_grouped_linear_fwd, fp8_grouped_linear_dgrad,
                   fp8_grouped_linear_wgrad)
from .autograd import Fp8Linear, fp8_autocast, fp8_state
from .experts import (ExpertBlock, ExpertPlan, GroupedExpertBlock, LayerNorm, Routing,
                      expert_combine, expert_dispatch, expert_mlp, expert_plan, expert_route,
                      layer_norm)
from .state import DelayedScalingLinear

__all__ = ["fp8_quantize_amax", "fp8_scale_update", "fp8_linear_fwd", "fp8_linear_dgrad",
           "fp8_linear_fwd_current",
           "fp8_bias_grad",
           "fp8_linear_wgrad", "fp8_pad_tokens", "fp8_last_error", "fp8_version", "load",
           "Fp8Error", "Slot", "DelayedScalingLinear", "FP8_TENSORWISE", "FP8_BLOCK_1x128",
           "FP8_BLOCK_128x128", "FP8_SCALE_FROM_AMAX", "FP8_SCALE_RECORD", "FP8_SCALE_REFRESH",
           "FP8_AMAX_ACCUMULATE", "FP8_SCALE_CLEAR_AMAX", "FP8_E5M2", "FP8_A_E5M2",
           "Fp8Linear", "fp8_autocast", "fp8_align_multiple", "fp8_pad_varlen",
           "fp8_unpad_varlen", "FP8_LAYOUT_THD", "FP8_LAYOUT_BSHD",
           "fp8_state", "FP8_DT_BF16", "FP8_DT_F16", "FP8_DT_F32",
           "fp8_layernorm_fwd", "fp8_layernorm_bwd", "fp8_layernorm_bwd_workspace",
           "fp8_moe_rows", "fp8_moe_sort", "fp8_moe_sort_workspace", "fp8_moe_dispatch",
           "fp8_moe_dispatch_bwd", "fp8_moe_combine", "fp8_moe_combine_bwd",
           "FP8_ACT_RELU", "FP8_ACT_SILU", "FP8_ACT_GELU", "fp8_moe_route", "fp8_moe_route_bwd",
           "fp8_moe_route_workspace", "fp8_act_quantize", "fp8_act_quantize_bwd",
           "fp8_grouped_linear_fwd", "fp8_grouped_linear_dgrad", "fp8_grouped_linear_wgrad",
           "ExpertBlock", "ExpertPlan", "LayerNorm", "expert_combine", "expert_dispatch",
           "expert_plan", "layer_norm", "GroupedExpertBlock", "Routing", "expert_mlp",
           "expert_route"]
