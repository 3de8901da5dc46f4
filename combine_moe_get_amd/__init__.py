"""MI355X-native MoE expert-parallel dispatch and combine.

The router with its balance losses, the routing layout, the optional int8
quantization, the scatter of routed token copies into expert-major receive rows,
the experts' matrix products over those rows (bf16, int8, microscaled 4-bit; with
their gradients), the gate between them (with its gradient, from bf16 or an 8-bit
checkpoint) and the weighted combine with zero / copy / constant experts (with
its gradient) run in hand-written HIP kernels for gfx950,
behind the C ABI of include/moe_get.h (libmoe_get.so).  This package is the
thin Python binding over that ABI plus seeded input generators.
"""
from .binding import (  # noqa: F401
    DEV_STATUS_BAD_EXPERT_ID, DEV_STATUS_RANK_OVERFLOW, LIB_PATH, QUANT_DYNAMIC_INT8, QUANT_NONE, QUANT_STATIC_INT8,
    Layout, MoeGetError, PreparedCall, Shape, abi_version, alloc_layout, alloc_workspace, check_shape, combine,
    dispatch, layout, layout_dispatch, layout_dispatch_launches, layout_launches, layout_noalloc, lib, make_shape,
    noalloc_scratch_bytes, prepare_layout_dispatch, prepare_combine, prepare_dispatch, prepare_layout,
    prepare_layout_noalloc, rank_capacity, recv_capacity, status_string, workspace_size,
)
from .experts import (  # noqa: F401
    ACT_NONE, ACT_SWIGLU, EXPERTS_DGRAD, EXPERTS_FORWARD, EXPERTS_WGRAD, ROWS_BF16, ROWS_INT8, ROWS_MXFP4,
    CombineGrad, ExpertsCall, ExpertsShape, Swiglu, SwigluGrad, check_experts_shape, combine_grad, experts_matmul,
    experts_matmul_dgrad, experts_matmul_wgrad, experts_tile, make_experts_shape, prepare_combine_grad,
    prepare_experts_matmul, prepare_experts_matmul_dgrad, prepare_experts_matmul_wgrad, prepare_quantize_rows,
    prepare_swiglu, prepare_swiglu_grad, quantize_rows, swiglu, swiglu_grad,
)
from .router import (  # noqa: F401
    GROUP_MAX, GROUP_TOP2, SCORE_SIGMOID, SCORE_SOFTMAX, Balance, BalanceLoss, Route, RouteShape, balance_loss,
    balance_workspace_size, check_route_shape, make_balance, make_route_shape, prepare_balance_loss, prepare_route,
    prepare_route_grad, route, route_grad,
)
