"""combine_quant_gb300: GB300-native MoE dispatch / combine with
pre-communication quantisation, and the experts' products between them.

The compute path is libcq.so (hand-written CUDA kernels for sm_103a behind the
C ABI declared in include/cq.h). This package is its thin Python binding:
``api`` marshals torch tensors into the C calls; ``weights`` prepares quantised
expert weights; ``workloads`` draws seeded synthetic inputs; ``build`` compiles
the library in-tree.
"""
from .api import (Config, DispatchResult, ExpertConfig, alloc_dispatch_outputs, alloc_workspace,  # noqa: F401
                  assist_views, check_bounded_meet, check_bounded_wait, combine, combine_q8, combine_quant,
                  combine_ws, cq_check_bounded_meet, cq_check_bounded_wait, cq_combine, cq_combine_q8,
                  cq_combine_quant, cq_combine_ws, cq_dispatch, cq_dispatch_noalloc, cq_dispatch_permute,
                  cq_dispatch_one_kernel, cq_dispatch_route, cq_dispatch_workspace_size,
                  cq_read_combine_status, cq_read_status, dispatch, dispatch_noalloc,
                  dispatch_one_kernel, dispatch_permute, dispatch_route, dispatch_workspace_size,
                  moe_combine, moe_dispatch, read_combine_status, read_status,
                  cq_expert_matmul, cq_expert_matmul_dw, cq_expert_matmul_dx, cq_expert_matmul_w4,
                  cq_read_expert_status, expert_matmul, expert_matmul_dw, expert_matmul_dx,
                  expert_matmul_w4, read_expert_status,
                  MoeConfig, NormConfig, NormResult, alloc_moe_workspace, cq_expert_matmul_b128,
                  cq_expert_matmul_b128_dx, cq_moe_layer, cq_norm_grad, cq_norm_quant, expert_matmul_b128,
                  expert_matmul_b128_dx, moe_layer, norm_grad, norm_quant)
from ._lib import (CQ_ST_BAD_ID, CQ_ST_BAD_MASK, CQ_ST_BAD_ROWS, CQ_ST_INTERNAL, CQ_ST_TIMEOUT,  # noqa: F401
                   CqError)
from .weights import quantize_b128, quantize_mx, quantize_w4  # noqa: F401
