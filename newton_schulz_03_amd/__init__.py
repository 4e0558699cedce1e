"""Batched Muon optimizer step for AMD MI355X (gfx950).

The computation lives in the HIP library libmuon_mi355x.so (C ABI declared in
include/muon_mi355x.h); this package is its Python binding.
"""
from ._binding import (  # noqa: F401
    CUBIC, EXPORTED, F4_GROUP, F8_BLOCK, F8_MAX_DIM, HEADER_PATH, KERNELS, LIB_PATH, MAX_DIM,
    MUON_BF16, MUON_ERR_HIP, MUON_ERR_INVALID_ARG, MUON_ERR_UNSUPPORTED, MUON_ERR_WORKSPACE,
    MUON_FP32, MUON_OK, MOE_MAX_EXPERTS, MOE_MAX_SLOTS, MOE_MAX_TOP_K, NOALLOC_MAX_WORKSPACE,
    QUINTIC, AdamWParams, DropoutParams, F4Operand, F8Operand, GradNormParams, MoePlan, MuonError,
    NsParams, StepParams, adamw_batched, adamw_workspace_bytes, allocate_workspace, dropout_batched,
    f4_empty, f4_matmul, f4_quantize, f4_workspace_bytes, f8_empty, f8_matmul_batched,
    f8_quantize_batched, f8_workspace_bytes, grad_clip_batched, grad_norm_batched,
    grad_scale_batched, grad_workspace_bytes, hbm_stream, last_error_detail, load_library,
    moe_combine, moe_combine_backward, moe_dispatch, moe_empty_plan, moe_sort, moe_workspace_bytes,
    ns_batched, ns_batched_noalloc, status_string, step_batched, timing_enable, timing_read,
    timing_reset, workspace_bytes,
)
