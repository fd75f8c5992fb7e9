"""libswiglu: the fused SwiGLU gate/up stage on AMD Instinct MI355X (gfx950).

    h = SiLU(x Wg^T) * (x Wu^T)

Python surface (thin marshalling over the C ABI in include/swiglu.h):
    fwd, fwd_fp8, bwd, bwd_noalloc, gemv_fwd, act_fwd, act_quant, act_bwd, swiglu (autograd), probe_read2,
    probe_mfma
and the routed block around the stage:
    route, route_bwd, router (autograd), moe_fwd, block_norm, block_norm_bwd, block_norms (autograd)
over any number of tokens, rows in order of expert:
    expert_plan, expert_gather, expert_combine, expert_combine_bwd, grouped_fwd, grouped_bwd, grouped_mm,
    grouped_mm_bwd; expert_rows, expert_sum, grouped_swiglu, grouped_linear, routed_mlp (autograd)
and the gradients' norm and clipping:
    grad_norm, clip_grads
"""
from ._lib import LIB_PATH, SwigluError, lib  # noqa: F401
from .block_ops import (  # noqa: F401
    BlockNormFunction, RouterFunction, block_norm, block_norm_bwd, block_norm_bwd_workspace_bytes, block_norms, moe_fwd,
    moe_workspace_bytes, route, route_bwd, router,
)
from .group_ops import (  # noqa: F401
    ExpertRowsFunction, ExpertSumFunction, GroupedLinearFunction, GroupedSwiGLUFunction, RoutedMLPFunction, clip_grads,
    expert_combine, expert_combine_bwd, expert_gather, expert_plan, expert_plan_workspace_bytes, expert_rows, expert_sum,
    grad_norm, grad_norm_workspace_bytes, grouped_bwd, grouped_bwd_workspace_bytes, grouped_fwd, grouped_linear,
    grouped_mm, grouped_mm_bwd, grouped_mm_bwd_workspace_bytes, grouped_swiglu, routed_mlp,
)
from .ops import (  # noqa: F401
    SwiGLUFunction, act_bwd, act_bwd_fp8, act_fwd, act_quant, probe_act_quant_stream, bwd, bwd_noalloc, bwd_workspace_bytes, fwd, fwd_fp8, gemv_fwd, probe_gemv_read,
    probe_mfma, probe_read2, swiglu,
)

__all__ = ["fwd", "fwd_fp8", "bwd", "bwd_noalloc", "gemv_fwd", "act_fwd", "act_quant", "act_bwd", "act_bwd_fp8", "swiglu", "SwiGLUFunction", "probe_read2", "probe_gemv_read", "probe_act_quant_stream", "probe_mfma",
           "bwd_workspace_bytes", "route", "route_bwd", "router", "RouterFunction", "moe_fwd", "moe_workspace_bytes", "block_norm", "block_norm_bwd",
           "block_norm_bwd_workspace_bytes", "block_norms", "BlockNormFunction",
           "expert_plan", "expert_plan_workspace_bytes", "expert_gather", "expert_combine", "expert_combine_bwd",
           "grouped_fwd", "grouped_bwd", "grouped_bwd_workspace_bytes", "grouped_mm", "grouped_mm_bwd",
           "grouped_mm_bwd_workspace_bytes",
           "expert_rows", "expert_sum", "grouped_swiglu", "grouped_linear", "routed_mlp", "ExpertRowsFunction",
           "ExpertSumFunction", "GroupedSwiGLUFunction", "GroupedLinearFunction", "RoutedMLPFunction", "grad_norm",
           "grad_norm_workspace_bytes", "clip_grads", "SwigluError", "lib", "LIB_PATH"]
