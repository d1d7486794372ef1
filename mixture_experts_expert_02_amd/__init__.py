"""MoE experts step for MI355X (gfx950): HIP kernels behind a C ABI.

`binding` marshals torch tensors into the C ABI of libmoe_experts.so
(include/moe_experts.h); all computation happens in the HIP library.
"""
from . import binding  # noqa: F401
from .binding import (  # noqa: F401
    GatedGrads, GatedOut, MoeError, NormOut, add_rmsnorm, align, experts_forward, experts_forward_grouped, gated_linear,
    gated_linear_backward, lora_linear, moe_add_rmsnorm, moe_align,
    moe_align_workspace_bytes, moe_device_error, moe_experts_forward, moe_experts_forward_grouped, moe_experts_forward_timed,
    moe_experts_grouped_workspace_bytes, moe_experts_workspace_bytes, moe_experts_workspace_layout,
    moe_gated_linear, moe_gated_linear_backward, moe_gated_linear_backward_workspace_bytes,
    moe_gated_linear_workspace_bytes, moe_lora_linear, moe_lora_linear_workspace_bytes, moe_mx_dequantize, moe_mx_linear, moe_mx_quantize, moe_route, moe_route_topk, moe_strerror, mx_dequantize,
    mx_linear, mx_quantize, problem, route, route_problem, route_topk,
)
