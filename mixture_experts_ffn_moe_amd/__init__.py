"""Routed Mixture-of-Experts FFN layer for MI355X (gfx950).

The compute lives in libmoe_mi355x.so (hand-written HIP kernels behind a C
ABI, declared in include/moe_mi355x.h, moe_shared.h, moe_shared_train.h,
moe_lora.h, moe_q4.h and moe_router_grad.h); this package is its ctypes binding
plus a small tensor-level helper.  PyTorch provides device memory and streams
only.
"""
from __future__ import annotations

from ._lib import (  # noqa: F401
    EXPORTED, LIB_PATH, MOE_BF16, MOE_ERR_HIP, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE,
    MOE_F32, MOE_OK, MOE_Q4_E2M1, MOE_Q4_INT4, NOALLOC_SCRATCH_BYTES, MoeError, MoeLoraSpec, MoeQ4Spec,
    MoeShape, make_lora, make_q4, make_shape, moe_balance_loss, moe_balance_workspace_size, moe_dropout_add,
    moe_dropout_backward, moe_finalize, moe_finalize_backward, moe_finalize_shared, moe_forward,
    moe_forward_noalloc, moe_forward_q4, moe_forward_shared, moe_get_shared_workspace_layout,
    moe_get_workspace_layout, moe_grouped_gemm_down, moe_grouped_gemm_w13_swiglu, moe_lora_down,
    moe_lora_w13_swiglu, moe_lora_workspace_size, moe_permute, moe_probe_mfma_bf16, moe_probe_read,
    moe_q4_down, moe_q4_get_sizes, moe_q4_quantize_down, moe_q4_quantize_w13, moe_q4_w13_swiglu, moe_route,
    moe_route_backward, moe_router_grad_workspace_size, moe_router_weight_grad,
    moe_shared_backward_workspace_size, moe_shared_ffn, moe_shared_ffn_backward, moe_shared_ffn_lora,
    moe_shared_ffn_train, moe_shared_workspace_size, moe_workspace_size, status_string, y_nbytes,
)
from .layer import MoELayerBuffers, SharedTrainBuffers, workspace_views  # noqa: F401
