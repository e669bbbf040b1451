"""GB300-native MoonEP layer path: plan, prefetch, permute, grouped GEMM,
combine and reduce_grad as sm_103a CUDA kernels behind a C ABI
(include/moonep.h), and the operators around it (include/moonep_ops.h): the
router with its balance loss and gradient, and the expert product in MXFP4; and
the feed-forward network (include/moonep_ffn.h): products with bias, activation and
residual, their gradients, and the combine with dropout.  ``_lib``, ``_ops`` and
``_ffn`` are the ctypes bindings with the same names."""
from ._lib import (  # noqa: F401
    GEMM_SCRATCH_BYTES, MoonepError, PlanWorkspace, dims, library, moonep_combine, moonep_combine_backward,
    moonep_dispatch, moonep_dispatch_backward, moonep_grouped_gemm_dw, moonep_grouped_gemm_dx,
    moonep_dispatch_send_once,
    moonep_get_plan_layout, moonep_grouped_gemm, moonep_launch_count, moonep_plan,
    moonep_plan_noalloc, moonep_plan_views, moonep_plan_workspace_bytes, moonep_prefetch_weights,
    moonep_read_status,
    moonep_reduce_grad, moonep_selftest_bounded_wait, status_string,
)
from ._ffn import (  # noqa: F401
    linear_dims, moonep_act_backward, moonep_act_backward_workspace_bytes, moonep_combine_dropout,
    moonep_combine_dropout_backward, moonep_grouped_act_backward,
    moonep_grouped_act_backward_workspace_bytes, moonep_grouped_gemm_act, moonep_linear,
    moonep_linear_dw, moonep_linear_dx,
)
from ._ops import (  # noqa: F401
    moonep_mxfp4_dequantize, moonep_mxfp4_dispatch, moonep_mxfp4_grouped_gemm,
    moonep_mxfp4_prefetch_weights, moonep_mxfp4_quantize, moonep_mxfp4_quantize_weights,
    moonep_router_backward, moonep_router_forward, moonep_router_workspace_bytes,
    mxfp4_scale_pitch, router_dims,
)
